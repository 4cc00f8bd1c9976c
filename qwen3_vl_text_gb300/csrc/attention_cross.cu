// Attention of packed query rows over keys and values of another length, on the tcgen05 tensor cores: cross attention
// to an encoder's states, and the part of a shared prefix in the attention of one new token (attention_decode.cu
// adds each sequence's own tokens).
//
//   o[t, h] = sum_i p_i v_i,  p = softmax_i(q[t, h] . k_i / sqrt(d)) over all keys i of t's segment, kv head h / (nq / nkv)
//
// No mask but the segment's end, so the rows of a kv head's whole group of q heads share every key: a tile's 128 rows are
// (token, head of the group) pairs, 128 / group tokens at a time, fetched as one box of a tensor map of q as [token][kv
// head][head of the group][element].  One token of a group of 8 heads is 8 rows of one tile, 4096 tokens are 256 full ones.
//
// Work: an item is a pair of row tiles A and B, or a last single one, of one kv head of one segment, in steps of 128 keys.  A
// pair shares every step; a single tile is run as A and B too, A on the even steps and B on the odd ones, and their
// results are merged at the end.  Items weigh 2 per step (single 1), and FIXED for their beginning and end; their weights are laid end
// to end and cut into one equal run per CTA, one CTA per SM, whatever the lengths are (read on the device); a step goes to the run
// that holds its first weight, or, where that is about as even, an item to the run that holds its first.  A run may end inside an item, whose parts (unnormalised output, running
// maximum and sum, fp32) go to the workspace and are joined in key order by a second launch: the result does not depend
// on timing.
//   warps 0-3    softmax of tile A, 4-7 of tile B: a thread per row; the running maximum is raised lazily; an item's end:
//                O / l -> bf16 -> global, or the part
//   warp 8       TMA: K, Q_A, Q_B, V, K, V, ... (page numbers looked up a batch of tiles ahead)
//   warps 9, 10  tcgen05.mma, from one thread each: S_t = Q_t K_j^T and O_t += P_t V_j of tile A and of tile B; the tensor
//                cores work on one tile while the other's softmax runs; P is read from TMEM (allocated by warp 8)
//   warp 11      finds the items of the run and hands them to the others through a ring
//   warps 12-15  (e4m3 pages) convert raw tiles to f16 ones
// P enters the value product in bf16 (packed rows: off by up to 2^-8 of each weight, as the rounded output is of itself) or as two halves of bf16
// (bf16 pages: 2^-16); e4m3 pages: in f16 (2^-11), times 2^13, as f16 ends at 2^-24.  Shape::SPLIT has what each costs.  Rows of
// no token are computed on what lies in shared memory and never stored.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "cross_walk.h"
#include "kernels.h"

namespace h3 {

using namespace cross;

namespace {

// mbar_wait in fewer instructions: the code of this kernel's roles competes for the SM's instruction cache (with waits, masks and
// copies of loops written out at every place, 96 KB, every role waited for instructions).
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, const volatile int *abort) {
    const uint32_t a = smem_u32(bar);
    bool done = mbar_try_wait(a, parity);
    if (__builtin_expect(done, 1)) return true;
    const long long t0 = clock64();
    #pragma unroll 1
    while (!done) {
        if (*abort || clock64() - t0 > kSpinLimitCycles) break;
        done = mbar_try_wait(a, parity);
    }
    return done;
}

// An item as one warp hands it to the others.
struct __align__(16) Item {
    int row0, n_a, n_b;     // row of its first token, tokens of its tiles (n_b 0: single)
    int head, chunk;        // kv head and share of its group
    int j0, j1, len, key0;  // steps of this run [j0, j1) (none: the run is over), keys; their first row, or the segment
    int parts, owner;       // parts of the item (0: all of its steps are this run's) and the CTA that has the first
    int pos;                // key tiles of the run before it
    // steps of row tile t: the first, and the distance of the next
    __device__ __forceinline__ int first(int t) const { return j0 + (n_b ? 0 : t); }
    __device__ __forceinline__ int stride() const { return n_b ? 1 : 2; }
    __device__ __forceinline__ bool active(int t) const { return first(t) < j1; }
};
constexpr int ITEMS = 8;

template <int D, int MODE>
struct Shape {
    static constexpr bool F8 = MODE == PAGES8;
    static constexpr int THREADS = F8 ? 512 : 384;
    static constexpr int ATOM = TQ * 128;                  // 64 columns of a 128-row tile
    static constexpr int TILE = TK * D * 2;                // one operand tile
    static constexpr int NSK = D == 128 ? 2 : F8 ? 3 : 4, NSV = NSK;   // K tiles, and V tiles, held
    // An e4m3 tile arrives in the second half of its place, where (128 columns) a row's 128 bytes are those of the f16 row's own second
    // half, so that a warp can convert its rows in place; 64 columns: beside the places.
    static constexpr int RAW = TK * D;
    static constexpr int RAWS = F8 && D == 64 ? NSK + NSV : 0;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * TILE;
    static constexpr int OFF_V = OFF_K + NSK * TILE;
    static constexpr int OFF_RAW = OFF_V + NSV * TILE;
    static constexpr int OFF_SEG = OFF_RAW + RAWS * RAW;   // pre, cq, ck
    static constexpr int OFF_ITEM = OFF_SEG + 3 * 4 * (kMaxSeqs + 4);  // ring of items
    static constexpr int OFF_ML = OFF_ITEM + ITEMS * (int)sizeof(Item);   // [128] (m, l) of tile B's share of a single tile's rows
    static constexpr int OFF_OUT = OFF_ML + 128 * 8;       // 32 rows x 64 bytes of output per softmax warp
    static constexpr int OFF_BAR = OFF_OUT + (MODE == ROWS ? 8 * 2048 : 0);
    static constexpr int BARS = 2 * NSK + 2 * NSV + 18 + 2 * ITEMS + (F8 ? NSK + NSV : 0);
    static constexpr int READERS = 11 + (F8 ? 4 : 0);      // warps that read an item
    static constexpr int BYTES = OFF_BAR + BARS * 8 + 128 + 1024;   // + alignment of the base
    // bf16 pages: P as two bf16 halves, as the decoding kernel has it, so that a prefix's weights keep 16 bits whichever kernel reads it.
    // 64 sequences behind 8192 tokens 71.2 -> 74.9 us; error against 64 bits 2.20e-3 -> 1.66e-3, that of the output's rounding alone.
    // Packed rows, which the tensor core bounds, would pay 37% (4096 queries over 1024 keys 119 -> 165 us, over 4096 406 -> 567, 16
    // ragged prompts 175 -> 238; 2.28e-3 -> 1.66e-3), e4m3 pages 9% for an error that stays 1.66e-3.
    static constexpr bool SPLIT = MODE == PAGES;
    // Scores held at a time: with e4m3 or split weights too few registers for a row, S is read twice (a whole row: 81 us in that case).
    static constexpr int HELD = MODE == ROWS ? TK : 64;
    // Column behind the tile's first score of the weights of keys 16 kk to 16 kk + 15; their second halves lie HELD / 2 further.
    static constexpr __device__ int p_at(int kk) { return kk * 16 / HELD * HELD + kk * 16 % HELD / 2; }
    static constexpr float UP = F8 ? 8192.f : 1.f;         // weights, and so l and o, are held times this
    static constexpr float UP_LOG2 = F8 ? 13.f : 0.f;
    // the maximum is raised when it grew by more than this (log2): weights reach 2^8, f16 ones 2^15 with UP
    static constexpr float RAISE = F8 ? 2.f : 8.f;
};

struct Args {
    AttentionCross p;
    int group, gc, chunks, tok;   // q heads per kv head; rows of a token in a tile, tiles' shares of a group; tokens of a tile
    unsigned inv_gc;              // ceil(2^16 / gc): row * inv_gc >> 16 = row / gc for row < 128
    int box_shift;                // log2 of the places of a page that one box covers
    float scale_log2;
    float *part;                  // [cta][slot][tile][D][128] partial outputs, unnormalised
    float2 *ml;                   // [cta][slot][tile][128] their running maximum and sum
    int4 *desc;                   // [cta][slot][2] the item of that part: (row of its first token, tokens of A, tokens of B,
                                  // unit), (parts, CTA of the first, -, -); parts 0: no part
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t r, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two values of 0 or more cut to bf16, and the negative of one.
__device__ __forceinline__ uint32_t cut_bf16x2(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ float minus_cut(float x) { return __uint_as_float((__float_as_uint(x) & 0xffff0000u) | 0x80000000u); }
// Two e4m3 bytes -> two f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *m, uint64_t *bar, int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Hint: bring the box at these element coordinates into L2.
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap *m, int32_t x, int32_t y, int32_t z, int32_t w) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
// tcgen05.mma with descriptors given by their low words (address and leading offset); the high words are constant.
// One addition per operand (with whole descriptors 2% slower).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // stride 1024 bytes, version 1, 128-byte swizzle
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "n"(kDescHi)
        : "memory");
}

// Weight that parts and their join cost (where there are pairs, and where not): packed rows' runs end between items where that makes
// none longer by more than this.  64 q heads over 8 of 128, runs that cut items against whole ones, and the weight added: 4096 queries
// over 1024 keys 131 and 118 us (5), 512 over 1024 37.3 and 24.3 (3), 512 over 4096 73 and 64 (10), 16 ragged prompts 181 and 173 (10);
// 64 over 1024 16.9 and 23.5 (16), 256 over 4096 45 and 64 (38).  Single tiles, 16 queries each over 500 keys, 16 sequences 21.3 and
// 15.6 (1), 30 over 1000 40.1 and 36.2 (5); 1 over 1000 13.3 and 17.4 (8), 4 of 100 queries of 10 heads over 4096 26.1 and 40.0 (26);
// 9 of 64 queries of 10 heads over 2000 28.3 and 27.1 (8: the rule misses it).
constexpr int JOIN_PAIRS = 12, JOIN_SINGLES = 6;

template <int D, int MODE>
__global__ void __launch_bounds__(Shape<D, MODE>::THREADS, 1)
    attention_cross_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Args a) {
    using S = Shape<D, MODE>;
    constexpr bool F8 = S::F8;
    constexpr int NSK = S::NSK, NSV = S::NSV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *sQ = smem + S::OFF_Q, *sK = smem + S::OFF_K, *sV = smem + S::OFF_V;
    int *pre = reinterpret_cast<int *>(smem + S::OFF_SEG), *cq = pre + kMaxSeqs + 4, *ck = cq + kMaxSeqs + 4;
    Item *ring = reinterpret_cast<Item *>(smem + S::OFF_ITEM);
    float2 *ml_s = reinterpret_cast<float2 *>(smem + S::OFF_ML);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::OFF_BAR);
    uint64_t *k_full = bars, *v_full = k_full + NSK, *k_empty = v_full + NSV, *v_empty = k_empty + NSK;
    uint64_t *q_full = v_empty + NSV, *q_ready = q_full + 2, *q_empty = q_ready + 2;   // [2] row tile, from here on
    uint64_t *s_full = q_empty + 2, *p_full = s_full + 2, *pv_done = p_full + 2, *l_full = pv_done + 2, *o_free = l_full + 1;   // [1], [1]
    uint64_t *turn = o_free + 1, *drain = turn + 2, *item_full = drain + 2, *item_empty = item_full + ITEMS;
    uint64_t *k_raw = F8 ? item_empty + ITEMS : k_full, *v_raw = F8 ? k_raw + NSK : v_full;   // where TMA arrives
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(F8 ? v_raw + NSV : item_empty + ITEMS);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *s_warp = reinterpret_cast<int *>(tmem_slot + 2);   // [16] scan of the warps' sums
    int *s_items = s_warp + 16, *s_most = s_items + 1;      // items, the largest weight

    const AttentionCross &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_trigger();
    if (tid == 0) {
        for (int i = 0; i < NSK; ++i) {
            mbar_init(k_full + i, F8 ? 4 : 1);
            mbar_init(k_empty + i, 2);
        }
        for (int i = 0; i < NSV; ++i) {
            mbar_init(v_full + i, F8 ? 4 : 1);
            mbar_init(v_empty + i, 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(q_ready + i, 4);
            mbar_init(q_empty + i, 1);
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(pv_done + i, 1);
            mbar_init(turn + i, 1);
            mbar_init(drain + i, 1);
        }
        mbar_init(l_full, 4);
        mbar_init(o_free, 4);
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(item_full + i, 1);
            mbar_init(item_empty + i, S::READERS);
        }
        for (int i = 0; F8 && i < NSK; ++i) {
            mbar_init(k_raw + i, 1);
            mbar_init(v_raw + i, 1);
        }
        *abort = 0;
        *s_items = *s_most = 0;
        fence_barrier_init();
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    if (warp == 8) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_wait();

    // the segments, clamped into what the call covers, and their weights: four per thread, scanned over the block
    bool any_empty = false;
    const int units = p.nkv * a.chunks;
    {
        bool bad = false, back = false;
        for (int i = tid; i <= p.n_segs; i += S::THREADS) {
            const int q = p.cu_q ? p.cu_q[i] : i ? p.Tq : 0;
            cq[i] = clamped(q, p.Tq);
            bad |= q != cq[i];
            back |= p.cu_q && i < p.n_segs && p.cu_q[i + 1] < q;
            if (MODE == ROWS || i < p.n_segs) {
                const int k = MODE != ROWS ? p.key_lens[i] : p.cu_k ? p.cu_k[i] : i ? p.max_keys : 0;
                ck[i] = clamped(k, p.max_keys);
                bad |= k != ck[i];
            }
        }
        if (__builtin_expect(__syncthreads_or(back), 0)) {
            if (tid == 0) ascend(cq, p.n_segs + 1);
            bad = true;
            __syncthreads();
        }
        const Segments g{pre, cq, ck};
        int n[4], sum = 0, items = 0, most = 0;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = 4 * tid + i;
            n[i] = 0;
            if (s < p.n_segs) {
                const int tokens = seg_tokens(g, s), tiles = (tokens + a.tok - 1) / a.tok, keys = seg_keys<MODE>(g, s);
                const int steps = (keys + TK - 1) / TK;
                if (keys > 0) {
                    n[i] = units * unit_weight(tiles, steps);
                    items += units * ((tiles + 1) >> 1);
                    if (tiles > 0) most = max(most, (tiles > 1 ? 2 * steps : steps) + FIXED + (tiles > 1 ? 1 << 30 : 0));
                }
                any_empty |= tokens > 0 && keys == 0;
                bad |= MODE == ROWS && ck[s + 1] < ck[s];
            }
            sum += n[i];
        }
        if (MODE != ROWS) any_empty |= cq[0] > 0 || cq[p.n_segs] < p.Tq;
        if (bad && blockIdx.x == 0) report(p.status, ST_BOUNDS);
        int inc = sum;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (MODE == ROWS) {
            items = __reduce_add_sync(0xffffffffu, items);
            most = __reduce_max_sync(0xffffffffu, most);
        }
        if (lane == 31) {
            s_warp[warp] = inc;
            if (MODE == ROWS && items > 0) {
                atomicAdd(s_items, items);
                atomicMax(s_most, most);   // (bit 30: there are pairs)
            }
        }
        __syncthreads();
        int at = inc - sum;
        for (int w = 0; w < warp; ++w) at += s_warp[w];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = 4 * tid + i;
            if (s <= p.n_segs) pre[s] = at;
            at += n[i];
        }
        tc_fence_before();
        any_empty = __syncthreads_or(any_empty);
        tc_fence_after();
    }
    const uint32_t tmem_base = *tmem_slot;
    const Segments g{pre, cq, ck};
    // A run has a step's weight at least: the parts of an item are then those of consecutive CTAs.
    const unsigned T = (unsigned)pre[p.n_segs], G = min(T / 2, gridDim.x);
    const Runs runs(T, G);
    bool snap = false;
    if (MODE == ROWS && G > 0) {
        const int items = *s_items, most = *s_most & ~(1 << 30), run = (int)(T / G);
        // what the longest run has more than its share if runs take whole items (all alike, at most one each, or any)
        const int more = (long long)most * items == (long long)T ? (run / most + (run % most ? 1 : 0)) * most - run
                                                                 : items <= (int)G ? most - run : most;
        snap = more <= (*s_most >> 30 ? JOIN_PAIRS : JOIN_SINGLES);
    }

    // rows without any key: zeros, or (prefixes) an empty part
    if (__builtin_expect(any_empty, 0)) {
        const auto fill = [&](int t0, int t1) {
            const int step = gridDim.x * S::THREADS / 32, at = blockIdx.x * (S::THREADS / 32) + warp;
            for (int r = t0 + at; r < t1; r += step) {   // a row of every head per warp
                if (MODE == ROWS) {
                    for (int i = lane; i < p.nq * D / 8; i += 32)
                        *reinterpret_cast<uint4 *>(p.o + r * p.ld_o + i * 8) = make_uint4(0, 0, 0, 0);
                } else {
                    for (int i = lane; i < p.nq; i += 32) p.pre_ml[(long long)r * p.nq + i] = make_float2(-INFINITY, 0.f);
                }
            }
        };
        for (int s = 0; s < p.n_segs; ++s)
            if (seg_keys<MODE>(g, s) == 0 && seg_tokens(g, s) > 0) fill(cq[s], cq[s + 1]);
        if (MODE != ROWS) {
            if (cq[0] > 0) fill(0, cq[0]);
            if (cq[p.n_segs] < p.Tq) fill(cq[p.n_segs], p.Tq);
        }
    }

    const auto raw_k = [&](uint32_t s) { return D == 128 ? sK + s * S::TILE + S::RAW : smem + S::OFF_RAW + s * S::RAW; };
    const auto raw_v = [&](uint32_t s) { return D == 128 ? sV + s * S::TILE + S::RAW : smem + S::OFF_RAW + (NSK + s) * S::RAW; };
    // A wait that runs out, in any warp, ends the CTA: *abort lets all other waits return, and no warp waits otherwise.
    const auto wait_on = [&](uint64_t *bar, uint32_t parity) {   // by a whole warp
        const bool good = __all_sync(0xffffffffu, wait_bar(bar, parity, abort));
        if (__builtin_expect(!good, 0) && lane == 0) {
            report(p.status, ST_TIMEOUT);
            *abort = 1;
        }
        return good;
    };
    // Items are read in the ring, where they stay until every warp has given them back.
    const auto give_back = [&](uint32_t i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty + i % ITEMS);
    };

    if (warp < 8) {
        // ------------------------------------------------ softmax
        const int t = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;            // row of the tile = TMEM lane
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem_base + lane_off + (uint32_t)(t * TQ);
        const uint32_t tO = tmem_base + lane_off + (uint32_t)(256 + t * 128);
        const int r_tok = r * a.inv_gc >> 16, r_head = r - r_tok * a.gc;
        if (warp == 0 && lane < 2) a.desc[2 * (2 * blockIdx.x + lane) + 1] = make_int4(0, 0, 0, 0);
        __syncwarp();
        // steps and items of this row tile, steps of tile B, single items with shares of both so far (barrier phases)
        uint32_t c = 0, items = 0, c_b = 0, shares = 0;
        bool good = true;
        for (uint32_t it = 0; good; give_back(it++)) {
            if (!(good = wait_on(item_full + it % ITEMS, (it / ITEMS) & 1))) break;
            const Item &w = ring[it % ITEMS];
            if (w.j0 >= w.j1) break;
            if (!w.active(t)) continue;
            const int n_tok = t && w.n_b ? w.n_b : w.n_a;
            const bool busy = quarter * 32 < n_tok * a.gc;   // this warp has rows of tokens
            float scale = a.scale_log2;
            if constexpr (F8) {
                // q to f16 in place: a row's largest |q| goes to [2^14, 2^15): exact but for elements 2^-29 of it and smaller
                if (!(good = wait_on(q_full + t, items & 1))) break;
                if (busy) {
                    const float ks = p.cache.k_scale[w.head];
                    uint8_t *row = sQ + t * S::TILE + r * 128;
                    const auto at = [&](int ch) {
                        return reinterpret_cast<uint4 *>(row + (ch >> 3) * S::ATOM + (((ch & 7) ^ (r & 7)) << 4));
                    };
                    float top = 0.f;
                    #pragma unroll 4
                    for (int ch = 0; ch < D / 8; ++ch) {
                        const uint4 x = *at(ch);
                        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
                        #pragma unroll
                        for (int i = 0; i < 4; ++i) top = fmax3(top, fabsf(bf16_lo(v[i])), fabsf(bf16_hi(v[i])));
                    }
                    const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
                    const float up = copysignf(__uint_as_float((uint32_t)(14 - e + 127) << 23), ks);
                    // (a scale of 0 still masks: -inf times a small number)
                    scale = fmaxf(a.scale_log2 * fabsf(ks) * __uint_as_float((uint32_t)(e - 14 + 127) << 23), 1e-37f);
                    #pragma unroll 4
                    for (int ch = 0; ch < D / 8; ++ch) {
                        uint4 x = *at(ch);
                        x.x = pack_f16x2(bf16_lo(x.x) * up, bf16_hi(x.x) * up);
                        x.y = pack_f16x2(bf16_lo(x.y) * up, bf16_hi(x.y) * up);
                        x.z = pack_f16x2(bf16_lo(x.z) * up, bf16_hi(x.z) * up);
                        x.w = pack_f16x2(bf16_lo(x.w) * up, bf16_hi(x.w) * up);
                        *at(ch) = x;
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready + t);
            }
            float m_use = -INFINITY, l = 0.f;
            const int first = w.first(t), stride = w.stride(), end = w.j1;
            for (int j = first; j < end; j += stride, ++c) {
                if (!(good = wait_on(s_full + t, c & 1))) break;
                const int valid = w.len - j * TK;    // keys of the tile
                if (busy) {
                    tc_fence_after();
                    constexpr int HELD = S::HELD;
                    uint32_t v[HELD];
                    float mx[8];
                    #pragma unroll
                    for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
                    const auto load = [&](int at) {
                        #pragma unroll
                        for (int q = 0; q < HELD; q += 32) tmem_ld32(tS + at + q, *reinterpret_cast<uint32_t (*)[32]>(&v[q]));
                        tmem_ld_wait();
                    };
                    // scores behind the segment: -inf, in place
                    #pragma unroll 1
                    for (int at = valid & ~31; __builtin_expect(at < TK, 0); at += 32) {
                        uint32_t x[32];
                        tmem_ld32(tS + at, x);
                        tmem_ld_wait();
                        #pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (at + i >= valid) x[i] = __float_as_uint(-INFINITY);
                        tmem_st32(tS + at, x);
                        tmem_st_wait();
                    }
                    #pragma unroll (HELD < TK ? 1 : 2)
                    for (int at = 0; at < TK; at += HELD) {
                        load(at);
                        #pragma unroll
                        for (int k = 0; k < HELD; k += 16)   // three-input maxima: chain u takes scores u, u + 8, ...
                            #pragma unroll
                            for (int u = 0; u < 8; ++u)
                                mx[u] = fmax3(mx[u], __uint_as_float(v[k + u]), __uint_as_float(v[k + u + 8]));
                    }
                    const float mt =
                        fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(fmax3(mx[3], mx[4], mx[5]), mx[6], mx[7])) * scale;
                    float alpha = 1.f;
                    bool raise = false;
                    if (j == first) {
                        m_use = mt;
                    } else if (mt > m_use + S::RAISE) {
                        alpha = ex2(m_use - mt);
                        m_use = mt;
                        raise = true;
                    }
                    // P = 2^(s * scale - m) (times UP), packed in pairs over the scores it comes from
                    const float off = m_use == -INFINITY ? 0.f : S::UP_LOG2 - m_use;   // (only -inf scores so far: weights 0)
                    const uint64_t scale2 = f32x2(scale, scale), off2 = f32x2(off, off);
                    uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
                    #pragma unroll (HELD < TK ? 1 : 2)
                    for (int at = 0; at < TK; at += HELD) {
                        if (HELD < TK) load(at);
                        #pragma unroll
                        for (int q = 0; q < HELD; q += 32) {
                            uint32_t pk[16];
                            #pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float x0, x1;
                                f32x2_split(ffma2(f32x2(__uint_as_float(v[q + 2 * i]), __uint_as_float(v[q + 2 * i + 1])), scale2,
                                                  off2), x0, x1);
                                const float p0 = ex2(x0), p1 = ex2(x1);
                                rs2[i & 3] = fadd2(rs2[i & 3], f32x2(p0, p1));
                                if constexpr (F8) pk[i] = pack_f16x2(p0, p1);
                                else pk[i] = S::SPLIT ? cut_bf16x2(p0, p1) : pack_bf16x2(p0, p1);
                                if (S::SPLIT) {
                                    v[q + 2 * i] = __float_as_uint(p0);
                                    v[q + 2 * i + 1] = __float_as_uint(p1);
                                }
                            }
                            tmem_st16(tS + at + q / 2, pk);
                            if constexpr (S::SPLIT) {
                                // what the cut left, larger by 2^-18 of the weight: above 0, as is then its product with an infinite value
                                constexpr float up = 1.f + 0x1p-18f;
                                #pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float p0 = __uint_as_float(v[q + 2 * i]), p1 = __uint_as_float(v[q + 2 * i + 1]);
                                    float x0, x1;
                                    f32x2_split(ffma2(f32x2(p0, p1), f32x2(up, up), f32x2(minus_cut(p0), minus_cut(p1))), x0, x1);
                                    pk[i] = pack_bf16x2(x0, x1);
                                }
                                tmem_st16(tS + at + HELD / 2 + q / 2, pk);
                            }
                        }
                    }
                    float rs = 0.f;
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float r0, r1;
                        f32x2_split(rs2[q], r0, r1);
                        rs += r0 + r1;
                    }
                    l = l * alpha + rs;
                    // O is rescaled after the previous product of this tile has completed
                    if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
                        if (!(good = wait_on(pv_done + t, (c - 1) & 1))) break;
                        tc_fence_after();
                        #pragma unroll 1
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t o[32];
                            tmem_ld32(tO + cc * 32, o);
                            tmem_ld_wait();
                            #pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st32(tO + cc * 32, o);
                        }
                    }
                    tmem_st_wait();
                }
                if (!F8 && __builtin_expect(valid < TK, 0) && (t == 0 || w.n_b == 0)) {
                    // values behind the segment may be anything (0 * NaN): cleared by the warps of the first tile that
                    // uses them, before their P is announced
                    const uint32_t at = w.pos + (j - w.j0);
                    if (!(good = wait_on(v_full + at % NSV, (at / NSV) & 1))) break;
                    uint8_t *tile = sV + at % NSV * S::TILE;
                    for (int i = valid * 8 + r; i < TK * 8; i += 128)
                        #pragma unroll
                        for (int cc = 0; cc < D / 64; ++cc)
                            *reinterpret_cast<uint4 *>(tile + cc * S::ATOM + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + t);
            }
            if (!good) break;
            ++items;
            const bool whole = w.parts == 0, single = w.n_b == 0, merge = single && w.active(1);
            float2 ml = make_float2(m_use, l);
            if (__builtin_expect(single && t == 1, 0)) {
                // tile A's warps merge the two shares of a single tile; the last such item's must have been read
                if (shares > 0) good = wait_on(o_free, (shares - 1) & 1);
                ++shares;
                ml_s[r] = ml;
                __syncwarp();
                if (lane == 0) mbar_arrive(l_full);
                continue;
            }
            // The next item's first product (which overwrites O) waits for this warp's next P, written after these reads.
            good = wait_on(pv_done + t, (c - 1) & 1);
            float f0 = 1.f, f1 = 0.f;
            if (t == 0 && w.active(1)) c_b += single ? (end - first) >> 1 : end - first;
            if (__builtin_expect(merge, 0)) {   // (tile B's softmax has seen its products before the last)
                good = good && wait_on(l_full, shares++ & 1) && wait_on(pv_done + 1, (c_b - 1) & 1);
                const float2 y = ml_s[r];
                const float top = fmaxf(ml.x, y.x), none = top == -INFINITY ? 0.f : top;
                f0 = ex2(ml.x - none);
                f1 = ex2(y.x - none);
                ml = make_float2(top, ml.y * f0 + y.y * f1);
            }
            if (!good) break;
            tc_fence_after();
            if (__builtin_expect(!whole, 0) && warp == 0 && lane == 0) {
                int4 *d = a.desc + 2 * (2 * blockIdx.x + (w.j0 == 0 ? 1 : 0));
                d[0] = make_int4(w.row0, w.n_a, w.n_b, w.head * a.chunks + w.chunk);
                d[1] = make_int4(w.parts, w.owner, 0, 0);
            }
            const bool live = busy && r_tok < n_tok && r_tok < a.tok && w.chunk * TQ + r_head < a.group;
            const long long row = w.row0 + t * a.tok + r_tok;
            const int qh = w.head * a.group + w.chunk * TQ + r_head;
            const long long slot = (long long)(2 * blockIdx.x + (w.j0 == 0 ? 1 : 0)) * 2 + t;   // of a part
            if (whole) {
                const float f = MODE == ROWS ? 1.f / ml.y : 1.f / S::UP;
                f0 *= f;
                f1 *= f;
            }
            uint8_t *buf = smem + S::OFF_OUT + warp * 2048;
            bf16 *base = MODE != ROWS ? nullptr
                                      : p.o + (long long)(w.row0 + t * a.tok) * p.ld_o +
                                            (long long)(w.head * a.group + w.chunk * TQ) * D + (lane & 3) * 8;
            const int heads = a.group - w.chunk * TQ, toks = min(n_tok, a.tok);
            #pragma unroll 1
            for (int col = busy ? 0 : D; col < D; col += 32) {
                // O (of the two halves) of 32 columns, scaled
                uint32_t x[32];
                tmem_ld32(tO + col, x);
                tmem_ld_wait();
                #pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f0);
                if (__builtin_expect(merge, 0)) {
                    uint32_t y[32];
                    tmem_ld32(tO + 128 + col, y);
                    tmem_ld_wait();
                    #pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(fmaf(__uint_as_float(y[i]), f1, __uint_as_float(x[i])));
                }
                if (__builtin_expect(!whole, 0)) {
                    float *dst = a.part + slot * (D * 128) + col * 128 + r;
                    if (live) {
                        #pragma unroll
                        for (int i = 0; i < 32; ++i) dst[i * 128] = __uint_as_float(x[i]);
                    }
                } else if constexpr (MODE == ROWS) {
                    // Through shared memory, so that four lanes write 64 bytes of one row (a lane's own row in pieces of
                    // 16 bytes touches 32 lines per store: three times as long).
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const auto pair = [&](int i) {
                            return pack_bf16x2(__uint_as_float(x[8 * q + i]), __uint_as_float(x[8 * q + i + 1]));
                        };
                        *reinterpret_cast<uint4 *>(buf + lane * 64 + ((q ^ (lane >> 1 & 3)) << 4)) =
                            make_uint4(pair(0), pair(2), pair(4), pair(6));
                    }
                    __syncwarp();
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = 8 * i + (lane >> 2);
                        const uint4 out = *reinterpret_cast<const uint4 *>(buf + rr * 64 + (((lane & 3) ^ (rr >> 1 & 3)) << 4));
                        const int tk = (quarter * 32 + rr) * a.inv_gc >> 16, hd = quarter * 32 + rr - tk * a.gc;
                        if (tk < toks && hd < heads) *reinterpret_cast<uint4 *>(base + tk * p.ld_o + hd * D + col) = out;
                    }
                    __syncwarp();
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.pre_o + (row * p.nq + qh) * D + col);
                    if (live) {
                        #pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dst[q] = make_float4(__uint_as_float(x[4 * q]), __uint_as_float(x[4 * q + 1]),
                                                 __uint_as_float(x[4 * q + 2]), __uint_as_float(x[4 * q + 3]));
                    }
                }
            }
            if (live && !whole) a.ml[slot * 128 + r] = ml;
            if (MODE != ROWS && live && whole) p.pre_ml[row * p.nq + qh] = make_float2(ml.x, ml.y / S::UP);
            if (merge) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free);
            }
        }
    } else if (warp == 8) {
        // ------------------------------------------------ producer
        const int tile_shift = 7 - a.box_shift, boxes = 1 << tile_shift, per = 32 >> tile_shift;   // boxes of a tile, tiles of a batch
        const int my_tile = lane >> tile_shift, my_box = lane & (boxes - 1);
        const int page_mask = MODE == ROWS ? 0 : (1 << p.cache.page_shift) - 1;
        bool ok = true;
        uint32_t gk = 0, gv = 0, nq_loaded[2] = {0, 0};
        const auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, wait_bar(bar, parity, abort));
            return ok;
        };
        for (uint32_t it = 0; ok; give_back(it++)) {
            if (!wait(item_full + it % ITEMS, (it / ITEMS) & 1)) break;
            const Item &w = ring[it % ITEMS];
            if (w.j0 >= w.j1) break;
            const int head = w.head;
            const auto look_up = [&](int j) {   // page of this lane's box in the batch of tiles from j on
                const int key = (j + my_tile) * TK + (my_box << a.box_shift);
                if (MODE == ROWS || j + my_tile >= w.j1 || key >= w.len) return 0;
                return p.table[(long long)w.key0 * p.ld_table + (key >> p.cache.page_shift)];
            };
            int page = look_up(w.j0), next_page = 0, batch = w.j0;
            // tile j of K or V into dst, on bar
            const auto load = [&](int j, const CUtensorMap *m, uint8_t *dst, uint64_t *bar) {
                if constexpr (MODE == ROWS) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, S::TILE);
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d(dst + c * S::ATOM, m, bar, c * 64, head, w.key0 + j * TK);
                    }
                } else {
                    const int n = min(boxes, (w.len - j * TK + (1 << a.box_shift) - 1) >> a.box_shift);
                    if (lane == 0) mbar_arrive_expect_tx(bar, (n << a.box_shift) * D * (F8 ? 1 : 2));
                    __syncwarp();
                    if (my_tile == j - batch && my_box < n) {
                        int pg = page;
                        if (pg < 0 || pg >= p.cache.num_pages) {
                            report(p.status, ST_BOUNDS);
                            pg = p.cache.num_pages;   // outside the map: the box is filled with zeros
                        }
                        const int place = (j * TK + (my_box << a.box_shift)) & page_mask;
                        if constexpr (F8) {
                            tma_load_4d(dst + (my_box << a.box_shift) * D, m, bar, 0, place, head, pg);
                        } else {
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_4d(dst + c * S::ATOM + (my_box << a.box_shift) * 128, m, bar, c * 64, place, head, pg);
                        }
                    }
                }
            };
            for (int j = w.j0; j < w.j1; ++j) {
                if (MODE != ROWS) {
                    if (j == batch + per) batch = j, page = next_page;
                    if (j == batch) next_page = look_up(j + per);
                }
                if (gk >= NSK && !wait(k_empty + gk % NSK, (gk / NSK - 1) & 1)) break;
                load(j, &tmK, F8 ? raw_k(gk % NSK) : sK + gk % NSK * S::TILE, k_raw + gk % NSK);
                ++gk;
                if (j == w.j0) {
                    for (int t = 0; t < (w.active(1) ? 2 : 1); ++t) {   // (a single tile's rows for both)
                        if (nq_loaded[t] > 0 && !wait(q_empty + t, (nq_loaded[t] - 1) & 1)) break;
                        ++nq_loaded[t];
                        if (lane == 0) {
                            mbar_arrive_expect_tx(q_full + t, a.tok * a.gc * D * 2);
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_4d(sQ + t * S::TILE + c * S::ATOM, &tmQ, q_full + t, c * 64, w.chunk * TQ, head,
                                            w.row0 + (w.n_b ? t * a.tok : 0));
                        }
                    }
                    // the next item's rows on their way to L2, if it is known (their tiles are free once this one's last scores are done)
                    const uint32_t ahead = it + 1;
                    if (ok && mbar_try_wait(smem_u32(item_full + ahead % ITEMS), (ahead / ITEMS) & 1) && lane == 0) {
                        const Item &x = ring[ahead % ITEMS];
                        if (x.j0 < x.j1)
                            for (int t = 0; t < (x.n_b > 0 ? 2 : 1); ++t)
                                for (int c = 0; c < D / 64; ++c)
                                    tma_prefetch_4d(&tmQ, c * 64, x.chunk * TQ, x.head, x.row0 + t * a.tok);
                    }
                    if (!ok) break;
                }
                if (gv >= NSV && !wait(v_empty + gv % NSV, (gv / NSV - 1) & 1)) break;
                load(j, &tmV, F8 ? raw_v(gv % NSV) : sV + gv % NSV * S::TILE, v_raw + gv % NSV);
                ++gv;
                __syncwarp();
            }
        }
        if (!ok) {
            // a wait ran out: leave once the copies in flight have landed (each of these waits is limited too)
            if (lane == 0) {
                report(p.status, ST_TIMEOUT);
                *abort = 1;
                const int never = 0;
                for (uint32_t f = gk > NSK ? gk - NSK : 0; f < gk; ++f) wait_bar(k_raw + f % NSK, (f / NSK) & 1, &never);
                for (uint32_t f = gv > NSV ? gv - NSV : 0; f < gv; ++f) wait_bar(v_raw + f % NSV, (f / NSV) & 1, &never);
                for (int t = 0; t < 2; ++t)
                    if (nq_loaded[t]) wait_bar(q_full + t, (nq_loaded[t] - 1) & 1, &never);
            }
            __syncwarp();
        }
    } else if (warp < 11) {
        // ------------------------------------------------ products: one thread for each row tile
        // A product of 128 x 128 x 16 takes 64 cycles, and its issue about as long; a wait or a commit costs the issuing
        // thread 50 to 90 more, so with one thread for both tiles the tensor cores stood still a third of the time (4096
        // tokens over 4096 keys, 64 heads over 8 of 128, as it was then: 440 us, with two threads 392).
        constexpr uint32_t kind = F8 ? 0u : (1u << 7) | (1u << 10);   // A and B f16, or bf16
        constexpr uint32_t base = (1u << 4) | kind | ((uint32_t)(TQ >> 4) << 24);
        constexpr uint32_t idesc_s = base | ((uint32_t)(TK >> 3) << 17);
        constexpr uint32_t idesc_o = base | ((uint32_t)(D >> 3) << 17) | (1u << 16);   // B (V) is MN-major
        if (lane == 0) {
            const int t = warp - 9;
            const uint32_t q_lo = (smem_u32(sQ + t * S::TILE) >> 4) | (1u << 16);   // (K-major: the leading offset is not used)
            const uint32_t k_lo = (smem_u32(sK) >> 4) | (1u << 16);
            const uint32_t v_lo = (smem_u32(sV) >> 4) | ((uint32_t)(S::ATOM >> 4) << 16);   // MN-major: 64 columns, ATOM bytes apart
            const uint32_t tS = tmem_base + t * TQ, tO = tmem_base + 256 + t * 128;
            bool ok = true;
            uint32_t gk = 0, gv = 0, np = 0, items = 0, turns = 0, merged = 0;   // ring positions; P tiles, items, turns, shares of single items of this row tile
            // K and V tiles are released by both threads; those of the other tile's steps at once
            const auto skip_k = [&]() {
                ok = wait_bar(k_full + gk % NSK, (gk / NSK) & 1, abort);
                if (ok) mbar_arrive(k_empty + gk++ % NSK);
                return ok;
            };
            const auto skip_v = [&]() {
                ok = wait_bar(v_full + gv % NSV, (gv / NSV) & 1, abort);
                if (ok) mbar_arrive(v_empty + gv++ % NSV);
                return ok;
            };
            for (uint32_t it = 0; ok; mbar_arrive(item_empty + it++ % ITEMS)) {
                ok = wait_bar(item_full + it % ITEMS, (it / ITEMS) & 1, abort);
                if (!ok) break;
                const Item &w = ring[it % ITEMS];
                if (w.j0 >= w.j1) break;
                const bool both = w.n_b > 0;
                if (__builtin_expect(!w.active(t), 0)) {
                    for (int j = w.j0; j < w.j1 && ok; ++j) ok = skip_k() && skip_v();
                    continue;
                }
                ok = wait_bar((F8 ? q_ready : q_full) + t, items & 1, abort);
                const int begin = w.j0, first = w.first(t), stride = w.stride(), end = w.j1;
                if (__builtin_expect(ok && first > begin, 0)) skip_k();
                // The first scores, then each step's value product with the next step's scores.  A pair's tiles take turns (else both
                // would do the same at the same time, and the tensor cores stand still during both softmaxes: 590 us
                // in the case above).  Of a single tile's steps every other one is this thread's; each K and V tile between
                // two of its own is released before it waits for a later one (they arrive in the order K, V, K, V, ...).
                #pragma unroll 1
                for (int j = first - stride; j < end && ok; j += stride) {
                    if (j >= first) {   // O_t (+)= P_t V, P_t in the columns of tile t's S
                        const uint32_t s = gv % NSV;
                        ok = wait_bar(v_full + s, (gv / NSV) & 1, abort) && wait_bar(p_full + t, np++ & 1, abort);
                        // the share of the single item before is still being read
                        if (ok && j == first && t == 1 && merged) ok = wait_bar(o_free, (merged - 1) & 1, abort);
                    }
                    if (!ok) break;
                    if (j >= first) {
                        if (both && (t == 1 || turns > 0)) ok = wait_bar(turn + t, (turns - (t == 0)) & 1, abort);
                        if (!ok) break;
                        const uint32_t s = gv++ % NSV, vb = v_lo + s * (S::TILE >> 4);
                        tc_fence_after();
                        #pragma unroll
                        for (int kk = 0; kk < TK / 16; ++kk)
                            mma_ts(tO, tS + S::p_at(kk), vb + kk * (2048 >> 4), idesc_o, j > first || kk > 0);
                        if (S::SPLIT) {   // the weights' second halves
                            #pragma unroll
                            for (int kk = 0; kk < TK / 16; ++kk)
                                mma_ts(tO, tS + S::p_at(kk) + S::HELD / 2, vb + kk * (2048 >> 4), idesc_o, true);
                        }
                        umma_commit(pv_done + t);
                        umma_commit(v_empty + s);
                    }
                    if (j + stride < end) {   // S_t = Q_t K^T
                        const uint32_t s = gk % NSK, kb = k_lo + s * (S::TILE >> 4);
                        ok = wait_bar(k_full + s, (gk / NSK) & 1, abort);
                        if (!ok) break;
                        ++gk;
                        tc_fence_after();
                        #pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * S::ATOM + (kk & 3) * 32) >> 4;
                            mma_ss(tS, q_lo + off, kb + off, idesc_s, kk > 0);
                        }
                        if (both && j >= first) mbar_arrive(turn + (t ^ 1));
                        umma_commit(s_full + t);
                        umma_commit(k_empty + s);
                        if (j + 2 * stride >= end) umma_commit(q_empty + t);   // the item's last scores of this tile
                        if (__builtin_expect(!both, 0)) {
                            if (j + 1 >= begin) skip_v();
                            if (ok && j + 3 < end) skip_k();
                        }
                    } else if (both) {
                        mbar_arrive(turn + (t ^ 1));
                    } else if (__builtin_expect(j + 1 < end, 0)) {
                        skip_v();   // the other thread's last
                    }
                    turns += both && j >= first;
                }
                if (t == 1 && !both) ++merged;
                ++items;
            }
            if (!ok) {
                report(p.status, ST_TIMEOUT);
                *abort = 1;
            }
            umma_commit(drain + t);
            const int never = 0;
            wait_bar(drain + t, 0, &never);
        }
        __syncwarp();
    } else if (warp == 11) {
        if (lane == 0) {
            // ------------------------------------------------ the items of the run, handed to the other warps
            Walk<MODE> w;
            const bool any = blockIdx.x < G;
            w.begin(any ? runs.first(blockIdx.x) : 0, any ? runs.first(blockIdx.x + 1) : 0, snap, g, p.n_segs, a.tok, a.chunks);
            bool ok = true, more = true;
            int pos = 0;
            for (uint32_t it = 0; ok && more; ++it) {
                if (it >= ITEMS) ok = wait_bar(item_empty + it % ITEMS, (it / ITEMS - 1) & 1, abort);
                if (!ok) break;
                more = w.next(g, a.tok, a.chunks, p.nkv);
                Item &x = ring[it % ITEMS];
                x.j0 = more ? w.j0 : 0;
                x.j1 = more ? w.j1 : 0;
                if (more) {
                    x.row0 = cq[w.s] + w.tok0;
                    x.n_a = w.n_a;
                    x.n_b = w.n_b;
                    x.head = w.head;
                    x.chunk = w.chunk;
                    x.len = w.len;
                    x.key0 = MODE == ROWS ? ck[w.s] : w.s;
                    x.parts = 0;
                    if (w.j0 > 0 || w.j1 < w.steps) {
                        x.owner = runs.owner(w.start);
                        x.parts = runs.owner(w.start + ((w.steps - 1) << w.shift)) - x.owner + 1;
                    }
                    x.pos = pos;
                    pos += w.j1 - w.j0;
                }
                mbar_arrive(item_full + it % ITEMS);
            }
            if (!ok) {
                report(p.status, ST_TIMEOUT);
                *abort = 1;
            }
        }
    } else if constexpr (F8) {
        // ------------------------------------------------ e4m3 -> f16
        uint32_t gt = 0;   // key tiles so far
        bool good = true;
        // A warp takes 32 rows, all of them into registers before it writes one (in place).
        const auto convert = [&](const uint8_t *src, uint8_t *out, uint64_t *raw, uint64_t *full, uint32_t phase, int keep) {
            if (!(good = wait_on(raw, phase & 1))) return;
            constexpr int N = D / 16;   // chunks of a lane, and of a row
            uint4 x[N];
            #pragma unroll
            for (int i = 0; i < N; ++i) x[i] = *reinterpret_cast<const uint4 *>(src + (warp - 12) * 32 * D + (i * 32 + lane) * 16);
            __syncwarp();
            #pragma unroll
            for (int i = 0; i < N; ++i) {
                const int row = (warp - 12) * 32 + (i * 32 + lane) / N, c = 2 * (lane % N);
                if (row >= keep) x[i] = make_uint4(0, 0, 0, 0);   // values behind the segment may be anything (0 * NaN)
                uint8_t *at = out + (c >> 3) * S::ATOM + row * 128;
                *reinterpret_cast<uint4 *>(at + (((c & 7) ^ (row & 7)) << 4)) = make_uint4(
                    e4m3x2_f16x2(x[i].x), e4m3x2_f16x2(x[i].x >> 16), e4m3x2_f16x2(x[i].y), e4m3x2_f16x2(x[i].y >> 16));
                *reinterpret_cast<uint4 *>(at + ((((c & 7) + 1) ^ (row & 7)) << 4)) = make_uint4(
                    e4m3x2_f16x2(x[i].z), e4m3x2_f16x2(x[i].z >> 16), e4m3x2_f16x2(x[i].w), e4m3x2_f16x2(x[i].w >> 16));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
        };
        for (uint32_t it = 0; good; give_back(it++)) {
            if (!(good = wait_on(item_full + it % ITEMS, (it / ITEMS) & 1))) break;
            const Item &w = ring[it % ITEMS];
            if (w.j0 >= w.j1) break;
            for (int j = w.j0; j < w.j1 && good; ++j, ++gt) {
                const uint32_t k = gt % NSK, v = gt % NSV;
                convert(raw_k(k), sK + k * S::TILE, k_raw + k, k_full + k, gt / NSK, TK);
                if (good) convert(raw_v(v), sV + v * S::TILE, v_raw + v, v_full + v, gt / NSV, w.len - j * TK);
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// Joins the parts of the items that several CTAs shared, in key order: part 0 is slot 1 of the first CTA, part i slot 0 of the
// i-th after it.  JOIN_Z blocks per part (blockIdx.x: CTA, blockIdx.y: slot), each with its share of the item's output: warps
// take 32 rows by four columns, a lane per row.  Bound by the chain item -> maxima -> parts, so a warp should have one or two shares.
constexpr int JOIN_Z = 8;
template <int D, int MODE>
__global__ void __launch_bounds__(256) attention_cross_join_kernel(const __grid_constant__ Args a) {
    pdl_trigger();
    pdl_wait();
    const AttentionCross &p = a.p;
    const int4 *desc = a.desc + 2 * (2 * blockIdx.x + blockIdx.y);
    const int4 it = __ldcg(desc), of = __ldcg(desc + 1);
    const int n = of.x, first = of.y, lane = threadIdx.x & 31;
    if (n == 0) return;
    const int head = it.w / a.chunks, chunk = it.w - head * a.chunks;
    const int quarters_a = (min(it.y, a.tok) * a.gc + 31) >> 5, quarters_b = (min(it.z, a.tok) * a.gc + 31) >> 5;
    const int units = (quarters_a + quarters_b) * (D / 4);
    for (int u = (((int)blockIdx.x - first) * JOIN_Z + (int)blockIdx.z) * 8 + (threadIdx.x >> 5); u < units; u += n * JOIN_Z * 8) {
        const int q = u / (D / 4), col = u % (D / 4) * 4, t = q >= quarters_a ? 1 : 0;
        const int r = (t ? q - quarters_a : q) * 32 + lane, r_tok = r * a.inv_gc >> 16, r_head = r - r_tok * a.gc;
        if (r_tok >= (t ? it.z : it.y) || r_tok >= a.tok || chunk * TQ + r_head >= a.group) continue;
        const auto slot = [&](int i) { return (long long)(2 * (first + i) + (i == 0 ? 1 : 0)) * 2 + t; };
        // eight parts at a time, all their loads in flight
        constexpr int BATCH = 8;
        float top = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        #pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += BATCH) {
            float2 ml[BATCH];
            float4 x[BATCH];
            #pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + k < n) {
                    const float *src = a.part + slot(i0 + k) * (D * 128) + (long long)col * 128 + r;
                    ml[k] = __ldcg(a.ml + slot(i0 + k) * 128 + r);
                    x[k] = make_float4(__ldcg(src), __ldcg(src + 128), __ldcg(src + 256), __ldcg(src + 384));
                }
            }
            const float before = top;
            #pragma unroll
            for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
            const float base = top == -INFINITY ? 0.f : top, c = ex2(before - base);
            acc = make_float4(acc.x * c, acc.y * c, acc.z * c, acc.w * c);
            l *= c;
            #pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const float f = ex2(ml[k].x - base);
                l = fmaf(ml[k].y, f, l);
                acc.x = fmaf(x[k].x, f, acc.x);
                acc.y = fmaf(x[k].y, f, acc.y);
                acc.z = fmaf(x[k].z, f, acc.z);
                acc.w = fmaf(x[k].w, f, acc.w);
            }
        }
        const long long row = it.x + t * a.tok + r_tok;
        const int h = head * a.group + chunk * TQ + r_head;
        if (MODE == ROWS) {
            const float f = 1.f / l;
            *reinterpret_cast<uint2 *>(p.o + row * p.ld_o + (long long)h * D + col) =
                make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
        } else {
            constexpr float f = 1.f / Shape<D, MODE>::UP;
            *reinterpret_cast<float4 *>(p.pre_o + (row * p.nq + h) * D + col) =
                make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
            if (col == 0) p.pre_ml[row * p.nq + h] = make_float2(top, l * f);
        }
    }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

template <int D, int MODE>
cudaError_t launch(const AttentionCross &p, Args &a, int sms, long long most, cudaStream_t st) {
    using S = Shape<D, MODE>;
    static_assert(S::BYTES <= 232448, "shared memory of one CTA");
    static std::atomic<bool> ready[kMaxDevices];   // the shared-memory opt-in, per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready[dev].load()) {
        cudaError_t e = cudaFuncSetAttribute(attention_cross_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
        if (e != cudaSuccess) return e;
        ready[dev].store(true);
    }
    char *ws = static_cast<char *>(p.workspace) + kArrivalBytes;
    a.desc = reinterpret_cast<int4 *>(ws);
    a.ml = reinterpret_cast<float2 *>(ws + up256((size_t)sms * 4 * sizeof(int4)));
    a.part = reinterpret_cast<float *>(a.ml + (size_t)sms * 4 * 128);
    CUtensorMap tq, tk, tv;
    bool ok = make_tmap_heads(&tq, p.q, D, a.group, p.nkv, p.Tq, p.ld_q, a.gc, a.tok);
    if (MODE == ROWS) {
        // (without any key nothing is loaded; a map still needs an address)
        const bool any = p.max_keys > 0;
        ok = ok && make_tmap_heads(&tk, any ? p.k : p.q, D, 1, any ? p.nkv : 1, any ? p.max_keys : 1, any ? p.ld_k : D, 0, TK) &&
             make_tmap_heads(&tv, any ? p.v : p.q, D, 1, any ? p.nkv : 1, any ? p.max_keys : 1, any ? p.ld_v : D, 0, TK);
    } else {
        ok = ok && make_tmap_pages(&tk, p.cache, p.cache.k, 1 << a.box_shift) &&
             make_tmap_pages(&tv, p.cache, p.cache.v, 1 << a.box_shift);
    }
    if (!ok) return cudaErrorInvalidValue;
    const int grid = (int)std::min<long long>(sms, std::max<long long>(most, 1));
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3(grid), dim3(S::THREADS), S::BYTES, st, at);
    cudaError_t e = cudaLaunchKernelEx(&cfg, attention_cross_kernel<D, MODE>, tq, tk, tv, a);
    if (e != cudaSuccess) return e;
    cfg = pdl_config(dim3(grid, 2, JOIN_Z), dim3(256), 0, st, at);
    return cudaLaunchKernelEx(&cfg, attention_cross_join_kernel<D, MODE>, a);
}

}  // namespace

size_t attention_cross_workspace_bytes(int num_sms, int d) {
    const size_t own = kArrivalBytes + up256((size_t)num_sms * 4 * sizeof(int4)) +
                       (size_t)num_sms * 4 * 128 * (sizeof(float2) + d * sizeof(float));
    return std::max(own, attention_packed_workspace_bytes(num_sms));
}

long long attention_cross_weight(int Tq, int max_keys, int n_segs, int nq, int nkv) {
    return weight_bound(Tq, max_keys, n_segs, nq, nkv);
}

cudaError_t launch_attention_cross(const AttentionCross &p, cudaStream_t st) {
    if (p.Tq <= 0 || p.n_segs <= 0) return cudaSuccess;
    const int sms = device_num_sms();
    if (sms <= 0) return cudaErrorNoDevice;
    Args a{};
    a.p = p;
    a.group = p.nq / p.nkv;
    a.gc = std::min(a.group, TQ);
    a.chunks = (a.group + TQ - 1) / TQ;
    a.tok = TQ / a.gc;
    a.inv_gc = (65536 + a.gc - 1) / a.gc;
    const bool pages = p.key_lens != nullptr;
    a.box_shift = pages ? std::min(7, p.cache.page_shift) : 7;
    const int d = p.d;
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d));
    const long long most = attention_cross_weight(p.Tq, p.max_keys, p.n_segs, p.nq, p.nkv);
    if (!pages) return d == 128 ? launch<128, ROWS>(p, a, sms, most, st) : launch<64, ROWS>(p, a, sms, most, st);
    if (p.cache.f8) return d == 128 ? launch<128, PAGES8>(p, a, sms, most, st) : launch<64, PAGES8>(p, a, sms, most, st);
    return d == 128 ? launch<128, PAGES>(p, a, sms, most, st) : launch<64, PAGES>(p, a, sms, most, st);
}

}  // namespace h3
