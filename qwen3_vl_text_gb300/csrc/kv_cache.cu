// The paged key/value cache of one decoder layer: filling it (per-head q/k RMSNorm and
// rotation of a packed projection, K and V heads stored in their pages) and evicting from
// it by accumulated attention weight.  Both only move data: a few fp32 operations per
// element, so what bounds them is the bytes (or, for single tokens, the launch).
//
// The norm and rotation restate page "vllm-omni vllm_omni/diffusion/models/minimax_h3/
// encoder.py", MiniMaxH3Qwen3VLTextAttention.forward (q_norm / k_norm over head_dim, then
// _apply_rotary_pos_emb); the pages hold no cache.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace h3 {

namespace {

// Eight values divided by `scale` (IEEE division) and rounded to e4m3, saturating.
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float scale) {
    uint32_t w[2];
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 lo = make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
        const float2 hi = make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
        w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
               ((uint32_t)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(u[i]);
        x[2 * i + 1] = bf16_hi(u[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

constexpr int QK_THREADS = 256;

// D / 8 lanes per head vector, eight elements (16 bytes) each; lane l and lane l ^ (D/16) hold the
// two halves of a rotation pair.  A CTA takes one row and the heads blockIdx.y * 256/(D/8)
// onwards in steps of the grid.
template <int D>
__global__ void __launch_bounds__(QK_THREADS) qk_norm_rope_kernel(const QkNormRope p) {
    pdl_trigger();
    pdl_wait();
    constexpr int LANES = D / 8, HEADS = QK_THREADS / LANES;
    const int t = blockIdx.x;
    const int lane = threadIdx.x % LANES;
    const int heads = p.nq + 2 * p.nkv;
    const int j0 = (8 * lane) % (D / 2);
    const bool upper = lane >= LANES / 2;
    int page = -1, place = 0;
    if (p.has_cache) {
        const int slot = p.slots[t];
        if (slot >= 0) {
            page = slot >> p.cache.page_shift;
            place = slot & ((1 << p.cache.page_shift) - 1);
            if (page >= p.cache.num_pages) {
                if (threadIdx.x == 0 && blockIdx.y == 0) report(p.status, ST_BOUNDS);
                page = -1;
            }
        }
    }
    float cs[8], sn[8];
    if (p.cos_t) {
        #pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const long long at = p.cs_rows ? ((long long)((j0 + i) / 4) * p.cs_rows + t) * 4
                                           : (long long)t * (D / 2) + j0 + i;
            *reinterpret_cast<float4 *>(cs + i) = *reinterpret_cast<const float4 *>(p.cos_t + at);
            *reinterpret_cast<float4 *>(sn + i) = *reinterpret_cast<const float4 *>(p.sin_t + at);
        }
        #pragma unroll
        for (int i = 0; i < 8; ++i) sn[i] = upper ? sn[i] : -sn[i];   // y = x cos + partner * (-+ sin)
    }
    // whole groups of lanes share a head, so the shuffles below stay inside it; the trip count is
    // the same for every lane of a warp
    const int step = HEADS * gridDim.y;
    for (int h0 = blockIdx.y * HEADS; h0 < heads; h0 += step) {
        const int h = h0 + threadIdx.x / LANES;
        const bool in = h < heads;
        const bool is_q = h < p.nq, is_v = h >= p.nq + p.nkv;
        float x[8];
        unpack8(in ? *reinterpret_cast<const uint4 *>(p.qkv + t * p.ld_qkv + (long long)h * D + 8 * lane)
                   : make_uint4(0, 0, 0, 0), x);
        const bf16 *w = is_q ? p.wq : p.wk;
        float ss = 0.f;
        #pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        #pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (in && !is_v && w) {
            const float r = 1.0f / sqrtf(ss / (float)D + p.eps);
            float g[8];
            unpack8(*reinterpret_cast<const uint4 *>(w + 8 * lane), g);
            #pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * g[i];
        }
        if (p.cos_t) {
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = __shfl_xor_sync(0xffffffffu, x[i], LANES / 2);
                if (!is_v) x[i] = fmaf(x[i], cs[i], y * sn[i]);
            }
        }
        if (!in) continue;
        if (is_q) {
            if (p.q_out) *reinterpret_cast<uint4 *>(p.q_out + t * p.ld_q + (long long)h * D + 8 * lane) = pack8(x);
            continue;
        }
        const int g = is_v ? h - p.nq - p.nkv : h - p.nq;
        if (!is_v && p.k_out)
            *reinterpret_cast<uint4 *>(p.k_out + t * p.ld_k + (long long)g * D + 8 * lane) = pack8(x);
        if (page >= 0) {
            const long long at = page * p.cache.page_stride +
                                 ((long long)((g << p.cache.page_shift) + place)) * D + 8 * lane;
            void *dst = is_v ? p.cache.v : p.cache.k;
            if (p.cache.f8)
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(dst) + at) =
                    quant8(x, (is_v ? p.cache.v_scale : p.cache.k_scale)[g]);
            else
                *reinterpret_cast<uint4 *>(static_cast<bf16 *>(dst) + at) = pack8(x);
        }
    }
}

// ---------------------------------------------------------------- eviction

constexpr int SEL_THREADS = 1024;

// Order of the weights as unsigned integers: larger key, larger weight; both zeros alike, NaN lowest.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);   // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int clamped_len(const int32_t *lens, int b, int max_len, int32_t *status, bool say) {
    const int len = lens[b];
    if (len >= 0 && len <= max_len) return len;
    if (say) report(status, ST_BOUNDS);
    return len < 0 ? 0 : max_len;
}

// One CTA per sequence.  Finds the budget-th largest key of the unprotected tokens digit by
// digit (8 bits a pass, a histogram of the tokens that match the digits so far), then walks the
// tokens in order and gives each kept one its new place.
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const CacheEvict p) {
    pdl_trigger();
    pdl_wait();
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_need;
    __shared__ uint32_t wsum[2][32];
    const int b = blockIdx.x, tid = threadIdx.x;
    const int len = clamped_len(p.seq_lens, b, p.max_len, p.status, tid == 0);
    const float *w = p.weight + b * p.ld_weight;
    const int first = min(p.sink, len), last = len - min(p.recent, len);   // candidates [first, last)
    const bool all = len <= p.budget;
    uint32_t prefix = 0, need = 0;
    if (!all) {
        need = (uint32_t)(p.budget - p.sink - p.recent);
        for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
            for (int i = tid; i < 256; i += SEL_THREADS) hist[i] = 0;
            __syncthreads();
            for (int i = first + tid; i < last; i += SEL_THREADS) {
                const uint32_t k = weight_key(w[i]);
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                uint32_t left = need;
                int digit = 255;
                while (digit > 0 && hist[digit] < left) left -= hist[digit--];
                s_prefix = prefix | ((uint32_t)digit << shift);
                s_need = left;
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;   // how many of the tokens that equal the prefix so far are kept
        }
        if (p.budget == p.sink + p.recent) prefix = 0xffffffffu;   // none of the candidates (no key is that large)
    }
    int32_t *kept = p.kept + b * p.ld_kept;
    float *wo = p.weight_out + b * p.ld_weight_out;
    uint32_t base_keep = 0, base_eq = 0;
    for (int i0 = 0; i0 < len; i0 += SEL_THREADS) {
        const int i = i0 + tid;
        float v = 0.f;
        bool sure = false, eq = false;
        if (i < len) {
            v = w[i];
            if (all || i < first || i >= last) sure = true;
            else {
                const uint32_t k = weight_key(v);
                sure = k > prefix;
                eq = k == prefix;
            }
        }
        const uint32_t ms = __ballot_sync(0xffffffffu, sure), me = __ballot_sync(0xffffffffu, eq);
        const int lane = tid & 31, warp = tid >> 5;
        if (lane == 0) {
            wsum[0][warp] = __popc(ms);
            wsum[1][warp] = __popc(me);
        }
        __syncthreads();
        uint32_t ns = 0, ne = 0, ts = 0, te = 0;
        for (int k = 0; k < 32; ++k) {
            if (k < warp) ns += wsum[0][k], ne += wsum[1][k];
            ts += wsum[0][k];
            te += wsum[1][k];
        }
        const uint32_t below = (1u << lane) - 1;
        ns += __popc(ms & below);
        ne += base_eq + __popc(me & below);
        const uint32_t at = base_keep + ns + (min(ne, need) - min(base_eq, need));
        if (sure || (eq && ne < need)) {
            kept[at] = i;
            wo[at] = v;
        }
        base_keep += ts + (min(base_eq + te, need) - min(base_eq, need));
        base_eq += te;
        __syncthreads();
    }
    for (int i = (int)base_keep + tid; i < p.budget; i += SEL_THREADS) kept[i] = -1;
    for (int i = (int)base_keep + tid; i < p.max_len; i += SEL_THREADS) wo[i] = 0.f;
    if (tid == 0) p.new_lens[b] = (int32_t)base_keep;
}

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_VECS = 8;   // 16-byte vectors in flight per thread

// Moves the kept rows of one kv head's K (blockIdx.y even) or V (odd) of one sequence.  A CTA
// takes chunks of rows blockIdx.x, + gridDim.x, ...; in place (gridDim.x = 1) the chunks go in
// order: a row moves to its own index or a smaller one, so a chunk's sources are never behind its
// own first row, and no store of an earlier chunk reaches them; the barrier keeps a chunk's
// stores behind its own loads.
__global__ void __launch_bounds__(MOVE_THREADS) evict_move_kernel(const CacheEvict p) {
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.z, g = blockIdx.y >> 1;
    const int row_vecs = p.cache.d * (p.cache.f8 ? 1 : 2) / 16;   // 4, 8 or 16
    char *pool = static_cast<char *>((blockIdx.y & 1) ? p.cache.v : p.cache.k);
    const long long page_bytes = p.cache.page_stride * (p.cache.f8 ? 1 : 2);
    const int rows = MOVE_THREADS * MOVE_VECS / row_vecs, per = MOVE_THREADS / row_vecs;
    const int n = p.new_lens[b];
    const int32_t *kept = p.kept + b * p.ld_kept;
    const int32_t *ti = p.table + (long long)b * p.ld_table;
    const int32_t *to = p.table_out ? p.table_out + (long long)b * p.ld_table_out : ti;
    const int vec = threadIdx.x % row_vecs;
    const int mask = (1 << p.cache.page_shift) - 1;
    const auto place = [&](const int32_t *table, int i) -> char * {
        const int page = table[i >> p.cache.page_shift];
        if (page < 0 || page >= p.cache.num_pages) return nullptr;
        return pool + page * page_bytes + ((long long)((g << p.cache.page_shift) + (i & mask)) * row_vecs + vec) * 16;
    };
    for (int r0 = blockIdx.x * rows; r0 < n; r0 += rows * gridDim.x) {
        uint4 v[MOVE_VECS];
        char *dst[MOVE_VECS];
        #pragma unroll
        for (int k = 0; k < MOVE_VECS; ++k) {
            const int r = r0 + k * per + threadIdx.x / row_vecs;
            dst[k] = nullptr;
            if (r < n) {
                const char *src = place(ti, kept[r]);
                dst[k] = place(to, r);
                if (!src || !dst[k]) {
                    report(p.status, ST_BOUNDS);
                    dst[k] = nullptr;
                } else if (src == dst[k]) {
                    dst[k] = nullptr;   // already in its place
                } else {
                    v[k] = *reinterpret_cast<const uint4 *>(src);
                }
            }
        }
        if (!p.table_out) __syncthreads();
        #pragma unroll
        for (int k = 0; k < MOVE_VECS; ++k)
            if (dst[k]) *reinterpret_cast<uint4 *>(dst[k]) = v[k];
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRope &p, cudaStream_t st) {
    if (p.T <= 0) return cudaSuccess;
    const int per = QK_THREADS / (p.d / 8), groups = (p.nq + 2 * p.nkv + per - 1) / per;
    // few rows: the heads of a row over several CTAs
    const int sms = device_num_sms();
    int gy = 1;
    if (p.T < 2 * sms) gy = (2 * sms + p.T - 1) / p.T;
    if (gy > groups) gy = groups;
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3(p.T, gy), dim3(QK_THREADS), 0, st, at);
    return cudaLaunchKernelEx(&cfg, p.d == 128 ? qk_norm_rope_kernel<128> : qk_norm_rope_kernel<64>, p);
}

cudaError_t launch_cache_evict(const CacheEvict &p, cudaStream_t st) {
    if (p.n_seqs <= 0) return cudaSuccess;
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3(p.n_seqs), dim3(SEL_THREADS), 0, st, at);
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
    if (e != cudaSuccess || p.max_len == 0) return e;
    const int most = p.budget < p.max_len ? p.budget : p.max_len;
    const int rows = MOVE_THREADS * MOVE_VECS / (p.cache.d * (p.cache.f8 ? 1 : 2) / 16);
    cfg = pdl_config(dim3(p.table_out ? (most + rows - 1) / rows : 1, 2 * p.cache.nkv, p.n_seqs), dim3(MOVE_THREADS), 0,
                     st, at);
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

}  // namespace h3
