// The paged key/value cache of one decoder layer: filling it (per-head q/k RMSNorm and
// rotation of a packed projection, K and V heads stored in their pages) and evicting from
// it by accumulated attention weight.  Both only move data: a few fp32 operations per
// element, so what bounds them is the bytes (or, for single tokens, the launch).
//
// The norm and rotation restate page "vllm-omni vllm_omni/diffusion/models/minimax_h3/
// encoder.py", MiniMaxH3Qwen3VLTextAttention.forward (q_norm / k_norm over head_dim, then
// _apply_rotary_pos_emb); the pages hold no cache.
#include <algorithm>
#include <atomic>

#include "cache_rows.cuh"
#include "common.cuh"
#include "kernels.h"

namespace h3 {

namespace {

constexpr int QK_THREADS = 256;

// D / 16 lanes (a group) per head vector; lane l holds the elements 8l .. 8l + 7 of both halves, so
// that a rotation pair never leaves its lane.  Each row has 1 << gshift groups of a CTA, which take
// its heads in turn (blockIdx.y: every gridDim.y-th turn), so the row's rotary factors stay in
// registers; a CTA takes as many rows as it has groups for.  BATCH: head vectors a group loads before it works on
// the first; 3 where a group has several turns (8192 rows of 80 heads of 128: 61.7 us = 5.8 TB/s, with
// 1, 2 and 5: 71.8, 65.3 and 64.9), else 1 (4595 rows of 8 heads of 64: 3.5 us, with 3: 4.2).  Bound by the
// bytes, closely followed by the issue of instructions: 8 bytes per lane and shuffled rotation partners took 93 us.
template <int D, int BATCH>
__global__ void __launch_bounds__(QK_THREADS) qk_norm_rope_kernel(const QkNormRope p, int gshift) {
    constexpr int LANES = D / 16, GROUPS = QK_THREADS / LANES;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const int t = blockIdx.x * (GROUPS >> gshift) + (group >> gshift);
    const bool row = t < p.T;
    const int heads = row ? p.nq + 2 * p.nkv : 0;
    const int step = gridDim.y << gshift;
    const int first = (blockIdx.y << gshift) + (group & ((1 << gshift) - 1));
    const bf16 *src = p.qkv + t * p.ld_qkv + 8 * lane;
    float cs[8], sn[8];
    int slot = -1;
    const bool rotate = p.cos_t != nullptr;
    // the same number of turns for every lane of a warp (the shuffles below need them all)
    for (int h0 = 0; h0 < p.nq + 2 * p.nkv; h0 += BATCH * step) {
        uint4 raw[BATCH][2];
        #pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int h = h0 + first + u * step;
            raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
            if (h < heads) {
                const uint4 *v = reinterpret_cast<const uint4 *>(src + (long long)h * D);
                raw[u][0] = v[0];
                raw[u][1] = v[D / 16];
            }
        }
        if (h0 == 0) {   // behind the first loads: what the row's heads share
            if (p.has_cache && row) slot = p.slots[t];
            if (rotate && row) {
                #pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const long long at = p.cs_rows ? ((long long)(2 * lane + i / 4) * p.cs_rows + t) * 4
                                                   : (long long)t * (D / 2) + 8 * lane + i;
                    *reinterpret_cast<float4 *>(cs + i) = *reinterpret_cast<const float4 *>(p.cos_t + at);
                    *reinterpret_cast<float4 *>(sn + i) = *reinterpret_cast<const float4 *>(p.sin_t + at);
                }
            }
        }
        #pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int h = h0 + first + u * step;
            const bool in = h < heads, is_q = h < p.nq, is_v = h >= p.nq + p.nkv;
            float x[8], y[8];
            unpack8(raw[u][0], x);
            unpack8(raw[u][1], y);
            const bf16 *w = is_q ? p.wq : p.wk;
            float ss = 0.f;
            #pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
            #pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!in) continue;
            if (!is_v) {
                if (w) {
                    const float r = rsqrtf(ss / (float)D + p.eps);   // within 2 ulp
                    float g[8];
                    unpack8(*reinterpret_cast<const uint4 *>(w + 8 * lane), g);
                    #pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] *= r * g[i];
                    unpack8(*reinterpret_cast<const uint4 *>(w + D / 2 + 8 * lane), g);
                    #pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] *= r * g[i];
                }
                if (rotate) {
                    #pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a = x[i];
                        x[i] = fmaf(a, cs[i], -(y[i] * sn[i]));
                        y[i] = fmaf(y[i], cs[i], a * sn[i]);
                    }
                }
                raw[u][0] = pack8(x);
                raw[u][1] = pack8(y);
            }
            if (is_q) {
                if (p.q_out) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + t * p.ld_q + (long long)h * D + 8 * lane);
                    dst[0] = raw[u][0];
                    dst[D / 16] = raw[u][1];
                }
                continue;
            }
            const int g = is_v ? h - p.nq - p.nkv : h - p.nq;
            if (!is_v && p.k_out) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.k_out + t * p.ld_k + (long long)g * D + 8 * lane);
                dst[0] = raw[u][0];
                dst[D / 16] = raw[u][1];
            }
            if (slot < 0) continue;
            const int page = slot >> p.cache.page_shift, place = slot & ((1 << p.cache.page_shift) - 1);
            if (page >= p.cache.num_pages) {
                if (lane == 0) report(p.status, ST_BOUNDS);
                continue;
            }
            const long long at = page * p.cache.page_stride +
                                 ((long long)((g << p.cache.page_shift) + place)) * D + 8 * lane;
            void *dst = is_v ? p.cache.v : p.cache.k;
            if (p.cache.f8) {
                const float scale = (is_v ? p.cache.v_scale : p.cache.k_scale)[g];
                uint2 *out = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(dst) + at);
                out[0] = quant8(x, scale);
                out[D / 16] = quant8(y, scale);
            } else {
                uint4 *out = reinterpret_cast<uint4 *>(static_cast<bf16 *>(dst) + at);
                out[0] = raw[u][0];
                out[D / 16] = raw[u][1];
            }
        }
    }
}

// ---------------------------------------------------------------- eviction

constexpr int SEL_THREADS = 1024;
constexpr int SEL_BLOCK = 32 * SEL_THREADS;   // tokens of one block of the placing pass
constexpr int SEL_CACHE = 45056;              // weights a CTA holds in shared memory (176 KB)
constexpr int SEL_PER_CTA = 4096;             // tokens per CTA from which the cluster grows
constexpr int BINS = 2048;

// Order of the weights as unsigned integers: larger key, larger weight; both zeros alike, NaN lowest.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);   // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Inclusive scan over the block (1024 threads); sums [32] shared.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();   // the last use of sums is over
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    uint32_t w = sums[lane];
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);   // sum of the warps before this one
    return v + (warp ? before : 0u);
}

// Adds to the word at this shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ void add_cluster(uint32_t *p, uint32_t rank, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "r"(v)
                 : "memory");
}
__device__ __forceinline__ void set_cluster(uint32_t *p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// One CTA, or a cluster of up to 16, per sequence, each with a contiguous part of its tokens, whose weights
// it holds in shared memory (what does not fit is read again).  The budget-th largest key of the
// unprotected tokens is found in up to three digits (11, 11 and 10 bits): a histogram of the tokens that
// match the digits so far, scanned from the top by all threads; it ends early when the digit's whole bin is
// kept, which two digits almost always reach unless weights are equal.  In a cluster every CTA adds the bins
// that it has anything in to the first one's sums, which finds the digit for all.
// Then the tokens are counted in order, as bit masks of 32, and each kept one is written to its place.
// What bounds it is the chain of these steps, not the 4 bytes per token: back to back 8.1 us for 32 sequences of 4608 tokens,
// 10.8 us for one of 65,537 (the first with cold caches, under ncu: 12.4).
template <bool CLUSTER>
__global__ void __launch_bounds__(SEL_THREADS, 1) evict_select_kernel(const CacheEvict p, int cached) {
    extern __shared__ float held[];               // [cached] weights
    __shared__ __align__(8) uint32_t hist[BINS];
    __shared__ __align__(8) uint32_t sum[CLUSTER ? 3 : 1][BINS];   // over the cluster, one per digit
    __shared__ uint32_t mask_sure[SEL_BLOCK / 32], mask_eq[SEL_BLOCK / 32];
    __shared__ uint32_t sums[32], s_base[2], s_total;
    __shared__ uint32_t s_found[3];   // the digit, how many of its bin are kept, how many it holds
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < BINS; i += SEL_THREADS) {
        hist[i] = 0;
        #pragma unroll
        for (int k = 0; k < (CLUSTER ? 3 : 1); ++k) sum[k][i] = 0;
    }
    if (tid < 2) s_base[tid] = 0;
    if (CLUSTER) cluster_arrive();   // the sums may be added to once all CTAs have cleared theirs
    pdl_wait();
    const uint32_t rank = CLUSTER ? cluster_ctarank() : 0u;
    const int ranks = CLUSTER ? (int)gridDim.x : 1, b = blockIdx.y;
    int len = p.seq_lens[b];
    if (len < 0 || len > p.max_len) {
        if (tid == 0 && rank == 0) report(p.status, ST_BOUNDS);
        len = len < 0 ? 0 : p.max_len;
    }
    const int per = (len + ranks - 1) / ranks;                 // this CTA's tokens [begin, begin + n)
    const int begin = min((int)rank * per, len), n = min(per, len - begin);
    const float *w = p.weight + b * p.ld_weight + begin;
    const int first = min(p.sink, len) - begin, last = len - min(p.recent, len) - begin;   // candidates [first, last)
    const bool all = len <= p.budget;
    const uint32_t wanted = all ? 0u : (uint32_t)(p.budget - p.sink - p.recent);   // of the candidates
    uint32_t prefix = 0, need = wanted;
    int cut = 0;   // keys are compared without their lowest `cut` bits
    #pragma unroll 4
    for (int i = tid; i < min(n, cached); i += SEL_THREADS) held[i] = w[i];
    const auto weight_of = [&](int i) { return i < cached ? held[i] : w[i]; };
    if (CLUSTER) cluster_wait();
    __syncthreads();
    for (int pass = 0; pass < 3 && wanted; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
        const uint32_t mask = (1u << bits) - 1, high = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
        #pragma unroll 4
        for (int i = max(first, 0) + tid; i < min(last, n); i += SEL_THREADS) {
            const uint32_t k = weight_key(weight_of(i));
            if (((k ^ prefix) & high) == 0) atomicAdd(&hist[(k >> shift) & mask], 1u);
        }
        __syncthreads();
        // thread t: the bins 2047 - 2t and 2046 - 2t, so that the scan runs from the largest down
        const int low = BINS - 2 - 2 * tid;
        uint2 c = *reinterpret_cast<const uint2 *>(hist + low);
        *reinterpret_cast<uint2 *>(hist + low) = make_uint2(0, 0);   // for the next digit
        if (CLUSTER) {
            if (c.x) add_cluster(&sum[pass][low], 0, c.x);
            if (c.y) add_cluster(&sum[pass][low + 1], 0, c.y);
            cluster_sync();
            c = *reinterpret_cast<const uint2 *>(sum[pass] + low);
        }
        if (rank == 0) {
            const uint32_t upto = block_scan(c.x + c.y, sums), before = upto - c.x - c.y;
            if (before < need && need <= upto) {   // exactly one thread
                const bool in_high = need <= before + c.y;
                s_found[0] = in_high ? low + 1 : low;
                s_found[1] = need - before - (in_high ? 0u : c.y);
                s_found[2] = in_high ? c.y : c.x;
            }
            __syncthreads();
            if (CLUSTER && tid > 0 && tid < ranks)
                #pragma unroll
                for (int i = 0; i < 3; ++i) set_cluster(&s_found[i], tid, s_found[i]);
        }
        if (CLUSTER) cluster_sync();
        prefix |= s_found[0] << shift;
        need = s_found[1];   // of the tokens that match the digits so far, this many are kept
        cut = shift;
        if (s_found[2] == need) break;
    }
    // kept for certain: protected tokens and larger keys; of the equal ones the first `need`
    const auto sort_of = [&](int i, bool &sure, bool &eq) {
        sure = all || i < first || i >= last;
        eq = false;
        if (!sure && wanted) {
            const uint32_t k = weight_key(weight_of(i)) >> cut;
            sure = k > prefix >> cut;
            eq = k == prefix >> cut;
        }
    };
    // The masks of a block of 32 rows of 1024 tokens, and thread t's count of both kinds before mask t, in one word
    // (a block holds at most 32768 of each); s_total: the block's.
    const auto mark = [&](int i0, int rows) {
        __syncthreads();
        #pragma unroll 4
        for (int r = 0; r < rows; ++r) {
            const int i = i0 + r * SEL_THREADS + tid;
            bool sure = false, eq = false;
            if (i < n) sort_of(i, sure, eq);
            const uint32_t ms = __ballot_sync(0xffffffffu, sure), me = __ballot_sync(0xffffffffu, eq);
            if (lane == 0) {
                mask_sure[r * 32 + warp] = ms;
                mask_eq[r * 32 + warp] = me;
            }
        }
        __syncthreads();
        const uint32_t own = tid < 32 * rows ? (uint32_t)__popc(mask_sure[tid]) << 16 | (uint32_t)__popc(mask_eq[tid]) : 0u;
        const uint32_t inc = block_scan(own, sums);
        hist[tid] = inc - own;   // (the digits are done with the histogram)
        if (tid == SEL_THREADS - 1) s_total = inc;
        __syncthreads();
    };
    const auto rows_of = [&](int i0) { return (min(n - i0, SEL_BLOCK) + SEL_THREADS - 1) / SEL_THREADS; };
    uint32_t base_sure = 0, base_eq = 0;   // of the tokens before this CTA's (before this block's)
    if (CLUSTER) {
        uint32_t cs, ce;
        if (n <= SEL_BLOCK) {
            mark(0, rows_of(0));
            cs = s_total >> 16;
            ce = s_total & 0xffffu;
        } else {   // more than a block: counted first, marked again below
            cs = ce = 0;
            for (int i0 = 0; i0 < n; i0 += SEL_BLOCK) {
                mark(i0, rows_of(i0));
                cs += s_total >> 16;
                ce += s_total & 0xffffu;
            }
        }
        if (tid < ranks && tid > (int)rank) {
            add_cluster(&s_base[0], tid, cs);
            add_cluster(&s_base[1], tid, ce);
        }
        cluster_sync();   // (the last access to another CTA's memory is before it)
        base_sure = s_base[0];
        base_eq = s_base[1];
    }
    int32_t *kept = p.kept + b * p.ld_kept;
    float *wo = p.weight_out + b * p.ld_weight_out;
    for (int i0 = 0; i0 < n; i0 += SEL_BLOCK) {
        const int rows = rows_of(i0);
        if (!CLUSTER || n > SEL_BLOCK) mark(i0, rows);
        const uint32_t below = (1u << lane) - 1;
        #pragma unroll 4
        for (int r = 0; r < rows; ++r) {
            const uint32_t ms = mask_sure[r * 32 + warp], me = mask_eq[r * 32 + warp], at = hist[r * 32 + warp];
            const uint32_t ns = base_sure + (at >> 16) + __popc(ms & below);
            const uint32_t ne = base_eq + (at & 0xffffu) + __popc(me & below);
            if ((ms >> lane & 1) || ((me >> lane & 1) && ne < need)) {
                const int i = i0 + r * SEL_THREADS + tid;
                const uint32_t to = ns + min(ne, need);
                kept[to] = begin + i;
                wo[to] = weight_of(i);
            }
        }
        base_sure += s_total >> 16;
        base_eq += s_total & 0xffffu;
    }
    // the rest of the rows, by all CTAs of the cluster
    const int total = all ? len : p.budget;
    for (int i = total + (int)rank * SEL_THREADS + tid; i < p.max_len; i += ranks * SEL_THREADS) wo[i] = 0.f;
    for (long long i = total + (int)rank * SEL_THREADS + tid; i < p.budget; i += ranks * SEL_THREADS) kept[i] = -1;
    // new_lens may be seq_lens: every thread of the sequence has read the length (in a cluster: before the
    // barrier above)
    __syncthreads();
    if (tid == 0 && rank == 0) p.new_lens[b] = total;
}

constexpr int MOVE_THREADS = 256;

// Where the rows (of kv head 0) of the kept tokens i0 + r were and go, r = tid, tid + MOVE_THREADS, ... < rows, as byte
// offsets in the pool; to: -1 if the token does not move.  All loads of a step are in flight together.
template <int MAX_ROWS>
__device__ __forceinline__ void look_up(const CacheEvict &p, int b, int i0, int rows, int n, const int32_t *table_out,
                                        long long *from, long long *to) {
    constexpr int N = (MAX_ROWS + MOVE_THREADS - 1) / MOVE_THREADS;
    const int shift = p.cache.page_shift, mask = (1 << shift) - 1;
    const int row_bytes = p.cache.d * (p.cache.f8 ? 1 : 2);
    const long long page_bytes = p.cache.page_stride * (p.cache.f8 ? 1 : 2);
    int k[N], src[N], dst[N];
    #pragma unroll
    for (int j = 0; j < N; ++j) {
        const int r = threadIdx.x + j * MOVE_THREADS;
        k[j] = r < rows && i0 + r < n ? p.kept[b * p.ld_kept + i0 + r] : -1;
    }
    #pragma unroll
    for (int j = 0; j < N; ++j) {
        src[j] = k[j] >= 0 ? p.table[(long long)b * p.ld_table + (k[j] >> shift)] : -1;
        dst[j] = k[j] >= 0 ? table_out[(i0 + (int)threadIdx.x + j * MOVE_THREADS) >> shift] : -1;
    }
    #pragma unroll
    for (int j = 0; j < N; ++j) {
        const int r = threadIdx.x + j * MOVE_THREADS;
        long long f = -1, t = -1;
        if (k[j] >= 0) {
            if (src[j] < 0 || src[j] >= p.cache.num_pages || dst[j] < 0 || dst[j] >= p.cache.num_pages) {
                report(p.status, ST_BOUNDS);
            } else {
                f = src[j] * page_bytes + (long long)(k[j] & mask) * row_bytes;
                t = dst[j] * page_bytes + (long long)((i0 + r) & mask) * row_bytes;
                if (f == t) t = -1;   // already there
            }
        }
        if (r < rows) {
            from[r] = f;
            to[r] = t;
        }
    }
}

// Copies the kept tokens into other pages: a CTA looks up the places of a chunk of tokens once and moves the
// chunk's rows of K and V of the kv heads (planes blockIdx.y, + gridDim.y, ...).  Bound by the bytes: every row is
// read and written once (32 sequences of 4096 tokens of 4 KB: 158 us, 6.8 TB/s).
__global__ void __launch_bounds__(MOVE_THREADS) evict_copy_kernel(const CacheEvict p) {
    constexpr int VECS = 4, MAX_ROWS = MOVE_THREADS * VECS / 4;   // 16-byte vectors of a plane per thread; rows of 4 vectors
    __shared__ long long s_src[MAX_ROWS], s_dst[MAX_ROWS];
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.z, tid = threadIdx.x;
    const int row_bytes = p.cache.d * (p.cache.f8 ? 1 : 2), vec_shift = 31 - __clz(row_bytes / 16);
    const long long head_bytes = (long long)row_bytes << p.cache.page_shift;
    const int rows = (MOVE_THREADS * VECS) >> vec_shift, r0 = blockIdx.x * rows, n = p.new_lens[b];
    if (r0 >= n) return;
    look_up<MAX_ROWS>(p, b, r0, rows, n, p.table_out + (long long)b * p.ld_table_out, s_src, s_dst);
    __syncthreads();
    for (int q = blockIdx.y; q < 2 * p.cache.nkv; q += gridDim.y) {
        char *pool = static_cast<char *>((q & 1) ? p.cache.v : p.cache.k) + (q >> 1) * head_bytes +
                     (tid & ((1 << vec_shift) - 1)) * 16;
        uint4 v[VECS];
        #pragma unroll
        for (int k = 0; k < VECS; ++k) {
            const int r = (k * MOVE_THREADS + tid) >> vec_shift;
            if (s_dst[r] >= 0) v[k] = *reinterpret_cast<const uint4 *>(pool + s_src[r]);
        }
        #pragma unroll
        for (int k = 0; k < VECS; ++k) {
            const int r = (k * MOVE_THREADS + tid) >> vec_shift;
            if (s_dst[r] >= 0) *reinterpret_cast<uint4 *>(pool + s_dst[r]) = v[k];
        }
    }
}

// Packs the kept tokens in place.  A CTA takes a slice (2^slice_shift 16-byte vectors) of one plane's rows through
// all chunks of tokens in order: a token moves to its own index or a smaller one, so no source of a chunk lies
// before the chunk's first token, where the stores of earlier chunks end; the barrier keeps a chunk's own
// stores behind its loads, and the one behind the stores keeps the places they go by until all warps have used
// them (a third buffer of places instead: 159 against 148 us for the 32 sequences below).  With few sequences the chain of
// chunks bounds it, so the slices are then narrow, the chunks long, and the places of the next chunk looked up
// while this one's rows are loaded (one sequence of 4608 tokens cut to 4096, both launches: 23 us, with whole rows
// and nothing ahead 52 us; 32 of them 148 us).
__global__ void __launch_bounds__(MOVE_THREADS, 4) evict_pack_kernel(const CacheEvict p, int slice_shift) {
    constexpr int VECS = 8, MAX_ROWS = MOVE_THREADS * VECS / 2;
    __shared__ long long s_src[2][MAX_ROWS], s_dst[2][MAX_ROWS];
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.z, tid = threadIdx.x;
    const int row_bytes = p.cache.d * (p.cache.f8 ? 1 : 2), slices = (row_bytes / 16) >> slice_shift;
    const long long head_bytes = (long long)row_bytes << p.cache.page_shift;
    const int rows = (MOVE_THREADS * VECS) >> slice_shift, n = p.new_lens[b];
    const auto next = [&](int r0, int buf) {
        look_up<MAX_ROWS>(p, b, r0, rows, n, p.table + (long long)b * p.ld_table, s_src[buf], s_dst[buf]);
    };
    for (int q = blockIdx.y; q < 2 * p.cache.nkv * slices; q += gridDim.y) {
        const int slice = q % slices, plane = q / slices;
        char *pool = static_cast<char *>((plane & 1) ? p.cache.v : p.cache.k) + (plane >> 1) * head_bytes +
                     ((slice << slice_shift) + (tid & ((1 << slice_shift) - 1))) * 16;
        __syncthreads();
        next(0, 0);
        __syncthreads();
        for (int r0 = 0, buf = 0; r0 < n; r0 += rows, buf ^= 1) {
            uint4 v[VECS];
            #pragma unroll
            for (int k = 0; k < VECS; ++k) {
                const int r = (k * MOVE_THREADS + tid) >> slice_shift;
                if (s_dst[buf][r] >= 0) v[k] = *reinterpret_cast<const uint4 *>(pool + s_src[buf][r]);
            }
            if (r0 + rows < n) next(r0 + rows, buf ^ 1);
            __syncthreads();
            #pragma unroll
            for (int k = 0; k < VECS; ++k) {
                const int r = (k * MOVE_THREADS + tid) >> slice_shift;
                if (s_dst[buf][r] >= 0) *reinterpret_cast<uint4 *>(pool + s_dst[buf][r]) = v[k];
            }
            __syncthreads();
        }
    }
}

constexpr int SEL_RANKS = 16;   // CTAs of a cluster, at most; more than 8 where the device can place such a cluster

template <bool CLUSTER>
cudaError_t launch_select(const CacheEvict &p, int ranks, cudaStream_t st) {
    static std::atomic<int> most[kMaxDevices];   // per device, once its shared memory is opted in: the largest cluster
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    cudaLaunchAttribute at[2];
    const auto config = [&](int r, size_t bytes) {
        cudaLaunchConfig_t cfg = pdl_config(dim3(r, p.n_seqs), dim3(SEL_THREADS), bytes, st, at);
        if (CLUSTER) {
            at[1].id = cudaLaunchAttributeClusterDimension;
            at[1].val.clusterDim.x = r;
            at[1].val.clusterDim.y = 1;
            at[1].val.clusterDim.z = 1;
            cfg.numAttrs = 2;
        }
        return cfg;
    };
    if (most[dev].load() == 0) {
        cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             SEL_CACHE * 4);
        if (e != cudaSuccess) return e;
        int found = 8;
        if (CLUSTER && cudaFuncSetAttribute(evict_select_kernel<CLUSTER>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                            1) == cudaSuccess) {
            int clusters = 0;
            const cudaLaunchConfig_t cfg = config(SEL_RANKS, SEL_CACHE * 4);
            if (cudaOccupancyMaxActiveClusters(&clusters, evict_select_kernel<CLUSTER>, &cfg) == cudaSuccess && clusters > 0)
                found = SEL_RANKS;
        }
        cudaGetLastError();   // a refused size leaves an error behind
        most[dev].store(found);
    }
    if (ranks > most[dev].load()) ranks = most[dev].load();
    const int per = (p.max_len + ranks - 1) / ranks, cached = per < SEL_CACHE ? per : SEL_CACHE;
    const cudaLaunchConfig_t cfg = config(ranks, (size_t)cached * 4);
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<CLUSTER>, p, cached);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRope &p, cudaStream_t st) {
    if (p.T <= 0) return cudaSuccess;
    // groups of a row: the power of two, up to a whole CTA's, that leaves the fewest of them idle in
    // the last turn (the largest of such); for few rows the largest, as it has the fewest turns
    const int groups = QK_THREADS / (p.d / 16), heads = p.nq + 2 * p.nkv, sms = device_num_sms();
    int gshift = 0, waste = 0;
    for (int g = 1; (1 << g) <= groups && (1 << (g - 1)) < heads; ++g) {
        const int idle = ((heads + (1 << g) - 1) >> g << g) - heads;
        if (idle <= waste || p.T < sms) gshift = g, waste = idle;
    }
    const int per_cta = groups >> gshift, rows = (p.T + per_cta - 1) / per_cta;
    // few rows: the turns of a row's heads over several CTAs
    const int turns = (heads + (1 << gshift) - 1) >> gshift;
    int gy = rows < 4 * sms ? (4 * sms + rows - 1) / rows : 1;
    if (gy > turns) gy = turns;
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3(rows, gy), dim3(QK_THREADS), 0, st, at);
    if (turns > gy)
        return cudaLaunchKernelEx(&cfg, p.d == 128 ? qk_norm_rope_kernel<128, 3> : qk_norm_rope_kernel<64, 3>, p, gshift);
    return cudaLaunchKernelEx(&cfg, p.d == 128 ? qk_norm_rope_kernel<128, 1> : qk_norm_rope_kernel<64, 1>, p, gshift);
}

cudaError_t launch_cache_evict(const CacheEvict &p, cudaStream_t st) {
    if (p.n_seqs <= 0) return cudaSuccess;
    int ranks = 1;
    while (ranks < SEL_RANKS && p.max_len > ranks * SEL_PER_CTA) ranks *= 2;
    cudaError_t e = ranks > 1 ? launch_select<true>(p, ranks, st) : launch_select<false>(p, 1, st);
    if (e != cudaSuccess || p.max_len == 0) return e;
    const int row_vecs = p.cache.d * (p.cache.f8 ? 1 : 2) / 16, sms = device_num_sms();   // 4, 8 or 16
    const int most = p.budget < p.max_len ? p.budget : p.max_len;
    const int vec_shift = 31 - __builtin_clz((unsigned)row_vecs);
    const long long planes = 2LL * p.cache.nkv;
    cudaLaunchAttribute at[1];
    if (p.table_out) {
        // the planes of a chunk over several CTAs where the chunks alone are too few to fill the SMs
        const int rows = (MOVE_THREADS * 4) >> vec_shift, chunks = (most + rows - 1) / rows;
        const long long ctas = (long long)chunks * p.n_seqs, want = 8LL * sms;
        const long long gy = std::min(planes, ctas >= want ? 1 : (want + ctas - 1) / ctas);
        cudaLaunchConfig_t cfg = pdl_config(dim3(chunks, (unsigned)gy, p.n_seqs), dim3(MOVE_THREADS), 0, st, at);
        return cudaLaunchKernelEx(&cfg, evict_copy_kernel, p);
    }
    // slices down to a sector of 32 bytes where the planes alone are too few
    int slice_shift = vec_shift;
    while (slice_shift > 1 && (planes << (vec_shift - slice_shift)) * p.n_seqs < 2 * sms) --slice_shift;
    const long long gy = std::min(planes << (vec_shift - slice_shift), 65535LL);
    cudaLaunchConfig_t cfg = pdl_config(dim3(1, (unsigned)gy, p.n_seqs), dim3(MOVE_THREADS), 0, st, at);
    return cudaLaunchKernelEx(&cfg, evict_pack_kernel, p, slice_shift);
}

}  // namespace h3
