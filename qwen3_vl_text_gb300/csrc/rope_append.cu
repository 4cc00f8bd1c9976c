// New rows of a packed projection: per-head q/k RMSNorm, rotation by positions that the kernel turns into angles
// itself, and the K and V heads appended to their sequences in a paged cache.
//
//   y = R(pos * w) (x / rms(x) * weight),  R: rotation of rotary_dim / 2 pairs, w_j = theta^(-2j / rotary_dim), scaled
//
// Angles.  cos and sin of pos * w_j need pos * w_j modulo a turn; as an fp32 product it is off by 2^-25 of the angle,
// which is 0.03 radians at position 10^6.  The host passes w_j / 2 pi as a 64-bit fraction f_j of a turn, and pos * f_j
// in 64-bit integers wraps by itself: the only errors are f_j's own 2^-53 of w_j (times the position) and fp32's
// 2^-24 of the result, at any position.  cos and sin are taken once per row and frequency of a CTA, in shared memory.
//
// What bounds it: the bytes, read once and written once, or for a few rows the chain of dependent loads row -> sequence ->
// length -> page -> store.  The rows' own loads go out before that chain.
#include <algorithm>
#include <cstdint>

#include "cache_rows.cuh"
#include "common.cuh"
#include "kernels.h"

namespace h3 {

namespace {

constexpr int THREADS = 256;

// The sequence whose rows [cu[b], cu[b + 1]) hold row t, by a whole warp: n_seqs <= 1024, so two loads at most, one
// after the other.  -1: none.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int n_seqs, int t, int lane) {
    int base = 0;
    if (n_seqs > 32) {
        const bool past = cu[min(32 * (lane + 1), n_seqs)] <= t;   // (the last of the blocks end at n_seqs)
        base = 32 * __popc(__ballot_sync(0xffffffffu, past));
        if (base >= n_seqs) return -1;
    }
    const int at = min(base + lane + 1, n_seqs);
    const bool past = base + lane + 1 <= n_seqs && cu[at] <= t;
    const int b = base + __popc(__ballot_sync(0xffffffffu, past));
    return b < n_seqs && cu[b] <= t && t < cu[b + 1] ? b : -1;
}

// D / 16 lanes (a group) per head vector, each with two chunks of eight elements, chosen so that no rotation pair leaves its lane:
// with R = rotary_dim / 16, lane l < R holds chunks l and l + R (with pairs (j, j + rotary_dim / 2) these are the two
// halves of eight pairs, with pairs (2j, 2j + 1) any chunk holds whole pairs), the others hold the chunks that are not rotated.
// Each row has 1 << gshift groups of a CTA, which take its heads in turn (blockIdx.y: every gridDim.y-th turn).
// A CTA takes `share` rows, GROUPS >> gshift at a time, and finds places and angles of all of them at its beginning: with
// that chain in front of every two rows of 80 heads of 128, 5600 rows took 63 us instead of 53 (4.5 TB/s; 8192 rows 68 us, 5.2).  Not
// HBM's limit: kv_cache.cu's kernel, which is given slots and tables, takes 61.7 us for those 8192 rows.
// BATCH: head vectors a group loads before it works on the first.
template <int D, int BATCH>
__global__ void __launch_bounds__(THREADS, BATCH == 1 ? 4 : 3)
    rope_append_kernel(const __grid_constant__ RopeAppend p, int gshift, int share) {
    constexpr int LANES = D / 16, GROUPS = THREADS / LANES;
    __shared__ float2 turn[GROUPS][D / 2];      // (cos, sin) of a row's frequencies
    __shared__ long long s_at[GROUPS];          // element offset of the row's place in the cache (head 0); -1: not stored
    __shared__ int s_pos[GROUPS][3];
    __shared__ bool s_live[GROUPS];             // the row belongs to a sequence
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const int rows = GROUPS >> gshift, t0 = blockIdx.x * share, t_end = min(t0 + share, p.T);
    const int heads = p.nq + 2 * p.nkv;
    const int step = gridDim.y << gshift;
    const int first = (blockIdx.y << gshift) + (group & ((1 << gshift) - 1));
    const int R = p.rot >> 4;
    const bool turned = lane < R;
    const int c0 = turned ? lane : 2 * R + lane - R, c1 = turned ? lane + R : c0 + D / 16 - R;
    bool found = false;
    float2 cs[8];
    long long at = -1;
    bool live = false;
    // (row, turn of its heads), the same number for every lane of a warp (the shuffles below need them all)
    int t_base = t0, h0 = 0;
    #pragma unroll 1
    while (t_base < t_end) {
        const int r = t_base - t0 + (group >> gshift), t = t0 + r;
        const bf16 *src = p.qkv + t * p.ld_qkv;
        const int in_row = t < t_end ? heads : 0;
        uint4 raw[BATCH][2];
        #pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int h = h0 + first + u * step;
            raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
            if (h < in_row) {
                const uint4 *v = reinterpret_cast<const uint4 *>(src + (long long)h * D);
                raw[u][0] = v[c0];
                raw[u][1] = v[c1];
            }
        }
        if (!found) {   // behind the first loads: what the rows' heads share
            found = true;
            const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
            for (int i = warp; i < t_end - t0; i += THREADS / 32) {
                const int row = t0 + i;
                const int b = !p.seq_lens ? 0 : p.cu_rows ? sequence_of(p.cu_rows, p.n_seqs, row, wl) : row < p.n_seqs ? row : -1;
                long long to = -1;
                int place = 0;
                if (b >= 0 && p.seq_lens) {
                    place = p.seq_lens[b] - (p.cu_rows ? p.cu_rows[b + 1] - row : 1);
                    if (p.has_cache) {
                        bool good = place >= 0 && place < p.max_len;
                        if (good) {
                            const int page = p.table[(long long)b * p.ld_table + (place >> p.cache.page_shift)];
                            good = page >= 0 && page < p.cache.num_pages;
                            to = page * p.cache.page_stride + (long long)(place & ((1 << p.cache.page_shift) - 1)) * D;
                        }
                        if (!good) {
                            to = -1;
                            if (wl == 0) report(p.status, ST_BOUNDS);
                        }
                    }
                }
                if (wl == 0) {
                    s_live[i] = b >= 0;
                    s_at[i] = to;
                }
                if (wl < 3)
                    s_pos[i][wl] = p.positions ? p.positions[(wl < p.axes ? wl : 0) * p.ld_pos + row] : place;
            }
            __syncthreads();
            for (int i = threadIdx.x; i < (t_end - t0) * (p.rot >> 1); i += THREADS) {
                const int row = i / (p.rot >> 1), j = i - row * (p.rot >> 1);
                const int axis = (int)(p.axis1 >> j & 1) + 2 * (int)(p.axis2 >> j & 1);
                // a signed 64-bit fraction of a turn, in halves of a turn
                const long long f = (long long)((unsigned long long)(long long)s_pos[row][axis] * p.turns[j]);
                float s, c;
                sincospif(__ll2float_rn(f) * 0x1p-63f, &s, &c);
                turn[row][j] = make_float2(c * p.magnitude, s * p.magnitude);
            }
            __syncthreads();
        }
        if (h0 == 0 && in_row) {
            live = s_live[r];
            at = s_at[r];
            if (turned) {
                #pragma unroll
                for (int i = 0; i < 8; ++i)
                    cs[i] = turn[r][p.interleaved ? 4 * (i < 4 ? c0 : c1) + (i & 3) : 8 * lane + i];
            }
        }
        #pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int h = h0 + first + u * step;
            const bool is_q = h < p.nq, is_v = h >= p.nq + p.nkv;
            float x[8], y[8];
            unpack8(raw[u][0], x);
            unpack8(raw[u][1], y);
            const bf16 *w = is_q ? p.wq : p.wk;
            float ss = 0.f;
            #pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
            #pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (h >= in_row || !live) continue;
            if (!is_v) {
                if (w) {
                    const float inv = rsqrtf(ss / (float)D + p.eps);   // within 2 ulp
                    float g[8];
                    unpack8(reinterpret_cast<const uint4 *>(w)[c0], g);
                    #pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] *= inv * g[i];
                    unpack8(reinterpret_cast<const uint4 *>(w)[c1], g);
                    #pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] *= inv * g[i];
                }
                if (turned) {
                    if (p.interleaved) {
                        #pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float a = x[2 * i], b = y[2 * i];
                            x[2 * i] = fmaf(a, cs[i].x, -(x[2 * i + 1] * cs[i].y));
                            x[2 * i + 1] = fmaf(x[2 * i + 1], cs[i].x, a * cs[i].y);
                            y[2 * i] = fmaf(b, cs[4 + i].x, -(y[2 * i + 1] * cs[4 + i].y));
                            y[2 * i + 1] = fmaf(y[2 * i + 1], cs[4 + i].x, b * cs[4 + i].y);
                        }
                    } else {
                        #pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float a = x[i];
                            x[i] = fmaf(a, cs[i].x, -(y[i] * cs[i].y));
                            y[i] = fmaf(y[i], cs[i].x, a * cs[i].y);
                        }
                    }
                }
                raw[u][0] = pack8(x);
                raw[u][1] = pack8(y);
            }
            if (is_q) {
                if (p.q_out) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + t * p.ld_q + (long long)h * D);
                    dst[c0] = raw[u][0];
                    dst[c1] = raw[u][1];
                }
                continue;
            }
            const int g = is_v ? h - p.nq - p.nkv : h - p.nq;
            if (!is_v && p.k_out) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.k_out + t * p.ld_k + (long long)g * D);
                dst[c0] = raw[u][0];
                dst[c1] = raw[u][1];
            }
            if (at < 0) continue;
            const long long to = at + ((long long)g << p.cache.page_shift) * D;
            void *dst = is_v ? p.cache.v : p.cache.k;
            if (p.cache.f8) {
                const float scale = (is_v ? p.cache.v_scale : p.cache.k_scale)[g];
                uint2 *out = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(dst) + to);
                out[c0] = quant8(x, scale);
                out[c1] = quant8(y, scale);
            } else {
                uint4 *out = reinterpret_cast<uint4 *>(static_cast<bf16 *>(dst) + to);
                out[c0] = raw[u][0];
                out[c1] = raw[u][1];
            }
        }
        h0 += BATCH * step;
        if (h0 >= heads) h0 = 0, t_base += rows;
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppend &p, cudaStream_t st) {
    if (p.T <= 0) return cudaSuccess;
    // groups of a row: the power of two, up to a whole CTA's, that leaves the fewest of them idle in
    // the last turn (the largest of such); for few rows the largest, as it has the fewest turns
    const int groups = THREADS / (p.d / 16), heads = p.nq + 2 * p.nkv, sms = device_num_sms();
    if (sms <= 0) return cudaErrorNoDevice;
    int gshift = 0, waste = 0;
    for (int g = 1; (1 << g) <= groups && (1 << (g - 1)) < heads; ++g) {
        const int idle = ((heads + (1 << g) - 1) >> g << g) - heads;
        if (idle <= waste || p.T < sms) gshift = g, waste = idle;
    }
    const int per_cta = groups >> gshift;
    // rows of a CTA: up to four rounds of the three resident CTAs per SM (one, two and three rounds: 55.6, 54.9 and 56.1 us in that
    // case; 8192 rows 73.1, 71.9 and 67.8 against 67.9), in whole groups of rows and up to what a CTA has places for: 5580 rows are
    // 1395 CTAs, 3.06 rounds, 8192 are 1366
    int share = (p.T + 12 * sms - 1) / (12 * sms);
    share = std::min((share + per_cta - 1) / per_cta * per_cta, groups);
    const int rows = (p.T + share - 1) / share;
    // few rows: the turns of a row's heads over several CTAs
    const int turns = (heads + (1 << gshift) - 1) >> gshift;
    int gy = rows < 4 * sms ? (4 * sms + rows - 1) / rows : 1;
    if (gy > turns) gy = turns;
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3(rows, gy), dim3(THREADS), 0, st, at);
    if (turns > gy)
        return cudaLaunchKernelEx(&cfg, p.d == 128 ? rope_append_kernel<128, 3> : rope_append_kernel<64, 3>, p, gshift, share);
    return cudaLaunchKernelEx(&cfg, p.d == 128 ? rope_append_kernel<128, 1> : rope_append_kernel<64, 1>, p, gshift, share);
}

}  // namespace h3
