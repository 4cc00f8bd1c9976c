// Attention of one new token of each sequence over a paged key/value cache.
//
// For q head h of kv group g: s_i = q . k_i / sqrt(d), o = sum_i softmax(s)_i v_i over the i < len
// tokens of the sequence, in one pass over the keys with the running maximum m and sum l of the
// softmax (scores in log2 units: p = 2^(s log2e - m)).
#include <cuda_fp8.h>

#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace h3 {

namespace {

constexpr int AD_WARPS = 8;

__device__ __forceinline__ float load_elem(const void *base, long long at, bool f8) {
    if (f8) {
        __nv_fp8_e4m3 x;
        x.__x = static_cast<const uint8_t *>(base)[at];
        return (float)x;
    }
    return __bfloat162float(static_cast<const bf16 *>(base)[at]);
}

// One CTA per (q head, sequence); its warps take the keys in turn, D / 32 elements per lane.
template <int D>
__global__ void __launch_bounds__(AD_WARPS * 32) attention_decode_kernel(const AttentionDecode p, float *scores,
                                                                          float2 *stat, long long ld_scores) {
    pdl_trigger();
    pdl_wait();
    constexpr int E = D / 32;
    __shared__ float sm_o[AD_WARPS][D], sm_m[AD_WARPS], sm_l[AD_WARPS];
    const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = h / (p.nq / p.cache.nkv);
    int len = p.seq_lens[b];
    if (len < 0 || len > p.max_len) {
        if (threadIdx.x == 0) report(p.status, ST_BOUNDS);
        len = len < 0 ? 0 : p.max_len;
    }
    const float ks = p.cache.f8 ? p.cache.k_scale[g] : 1.f, vs = p.cache.f8 ? p.cache.v_scale[g] : 1.f;
    const float scale = 1.4426950408889634f / sqrtf((float)D) * ks;
    float q[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(p.q[b * p.ld_q + h * D + lane + 32 * e]);
        o[e] = 0.f;
    }
    const int mask = (1 << p.cache.page_shift) - 1;
    for (int i = warp; i < len; i += AD_WARPS) {
        const int page = p.table[(long long)b * p.ld_table + (i >> p.cache.page_shift)];
        const bool ok = page >= 0 && page < p.cache.num_pages;
        if (!ok && lane == 0) report(p.status, ST_BOUNDS);
        const long long at =
            page * p.cache.page_stride + (long long)((g << p.cache.page_shift) + (i & mask)) * D + lane;
        float s = 0.f;
        if (ok)
            for (int e = 0; e < E; ++e) s = fmaf(q[e], load_elem(p.cache.k, at + 32 * e, p.cache.f8), s);
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= scale;
        if (scores && lane == 0) scores[((long long)b * p.nq + h) * ld_scores + i] = s;
        const float mn = fmaxf(m, s), c = exp2f(m - mn), pr = exp2f(s - mn);
        m = mn;
        l = l * c + pr;
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * c + (ok ? pr * load_elem(p.cache.v, at + 32 * e, p.cache.f8) : 0.f);
    }
    for (int e = 0; e < E; ++e) sm_o[warp][lane + 32 * e] = o[e];
    if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
    __syncthreads();
    float mm = -INFINITY;
    for (int w = 0; w < AD_WARPS; ++w) mm = fmaxf(mm, sm_m[w]);
    float ll = 0.f;
    for (int w = 0; w < AD_WARPS; ++w) ll += len ? sm_l[w] * exp2f(sm_m[w] - mm) : 0.f;
    for (int e = threadIdx.x; e < D; e += blockDim.x) {
        float acc = 0.f;
        for (int w = 0; w < AD_WARPS; ++w) acc += len ? sm_o[w][e] * exp2f(sm_m[w] - mm) : 0.f;
        p.o[b * p.ld_o + h * D + e] = __float2bfloat16_rn(len ? acc / ll * vs : 0.f);
    }
    if (stat && threadIdx.x == 0) stat[b * p.nq + h] = make_float2(mm, 1.f / ll);
}

// weight_out[b][i] = weight_in[b][i] + sum over the q heads, in order, of their p_i.
__global__ void __launch_bounds__(256) attention_weight_kernel(const AttentionDecode p, const float *scores,
                                                               const float2 *stat, long long ld_scores) {
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.y, i = blockIdx.x * blockDim.x + threadIdx.x;
    const int len = min(max(p.seq_lens[b], 0), p.max_len);
    if (i >= len) return;
    float acc = 0.f;
    for (int h = 0; h < p.nq; ++h) {
        const float2 ml = stat[b * p.nq + h];
        acc += exp2f(scores[((long long)b * p.nq + h) * ld_scores + i] - ml.x) * ml.y;
    }
    p.weight_out[b * p.ld_weight + i] = (p.weight_in ? p.weight_in[b * p.ld_weight + i] : 0.f) + acc;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t attention_decode_workspace_bytes(int num_sms, int n_seqs, int nq, int max_len, bool weights) {
    if (num_sms <= 0 || n_seqs < 0 || n_seqs > kMaxSeqs || nq < 1 || nq > 65536 || max_len < 0) return 0;
    size_t n = 256;
    if (weights)
        n += up256((size_t)n_seqs * nq * sizeof(float2)) + (size_t)n_seqs * nq * up256((size_t)max_len * 4);
    return n;
}

cudaError_t launch_attention_decode(const AttentionDecode &p, cudaStream_t st) {
    if (p.n_seqs <= 0) return cudaSuccess;
    char *ws = static_cast<char *>(p.workspace) + 256;
    float2 *stat = p.weight_out ? reinterpret_cast<float2 *>(ws) : nullptr;
    float *scores = p.weight_out ? reinterpret_cast<float *>(ws + up256((size_t)p.n_seqs * p.nq * sizeof(float2)))
                                 : nullptr;
    const long long ld = (long long)up256((size_t)p.max_len * 4) / 4;
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3(p.nq, p.n_seqs), dim3(AD_WARPS * 32), 0, st, at);
    cudaError_t e = cudaLaunchKernelEx(&cfg, p.cache.d == 128 ? attention_decode_kernel<128> : attention_decode_kernel<64>,
                                       p, scores, stat, ld);
    if (e != cudaSuccess || !p.weight_out || p.max_len == 0) return e;
    cfg = pdl_config(dim3((p.max_len + 255) / 256, p.n_seqs), dim3(256), 0, st, at);
    return cudaLaunchKernelEx(&cfg, attention_weight_kernel, p, (const float *)scores, (const float2 *)stat, ld);
}

}  // namespace h3
