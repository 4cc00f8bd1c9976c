// Attention of one new token of each sequence over a paged key/value cache.
//
// For q head h of kv head g: s_i = q . k_i / sqrt(d), o = sum_i softmax(s)_i v_i over the len cached
// tokens, in one pass over the keys with the running maximum m and sum l of the softmax (scores in
// log2 units: p = 2^(s log2e - m)).
//
// What bounds it: every cached byte is read once, and the q heads of a kv head (nq/nkv of them) do
// 2 flops each per byte pair: 8 flops a byte with 8 heads over bf16, far below the tensor cores'
// rate, so the bound is the memory's.  Hence:
//  * The keys of all (sequence, kv head) segments are laid end to end in tiles of 64 (e4m3: 128) and cut into one
//    equal run of tiles per CTA, one CTA per SM, whatever the lengths are: a run may end inside a
//    segment, whose parts are then joined (below).  Lengths are read on the device.
//  * Two producer warps, one for K and one for V, keep up to STAGES tiles in flight through TMA (a box
//    per page, one lane per box, their page numbers looked up a batch ahead); eight warps compute.
//  * The products run on mma.sync m16n8k16 with the q heads as the 16 rows: there are at most 16 rows
//    of work per key, which a 128-row tcgen05 tile would leave mostly empty, and a warp that
//    holds scores, weights and output in its own registers needs no exchange with other warps per tile.
//    Each warp takes 16 (32) keys of a tile with its own m, l and output; groups of four warps take the
//    tiles of the run in turn, so that their chains of product, softmax and product overlap.
//  * With at most 8 heads the rows 8-15 of the weight matrix P would be padding: they carry
//    P's rounding remainder p - bf16(p) instead, so the value product loses nothing to the 8-bit mantissa
//    at no cost (more than 8 heads: a second product).  e4m3 values are exact in f16, so that path
//    runs in f16, with q scaled by a power of two per head into f16's range and p by 2^14: f16 ends at
//    2^-24, so the two halves then leave an error of at most 2^-39 of a warp's largest weight, far below the
//    fp32 sums; unscaled, every weight under 2^-25 of the largest would be lost to o but counted in l.
// Measured (64 q heads over 8 kv heads of 128, pages of 64): 64 sequences of 5000 to 8192 tokens in bf16, 1.7 GB,
// 248-251 us = 6.8 TB/s, the measured copy rate; in e4m3 139-140 us (6.0 TB/s: the conversions of every key and value
// to f16 then take most of the time between two tiles); one sequence of 1025 tokens 7.3 us, which is
// the chain length -> page number -> tile -> products -> join across CTAs.  Calls that fill the SMs take 8 to
// 12 us more than their bytes at the copy rate (16 of those sequences 70 us, 62.5 of them bytes): 2.5 until the first tile
// lands, the rest the joins at the end and the spread of the SMs' rates.
#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace h3 {

namespace {

constexpr int WK = 128;                 // keys per CTA of the weight sums; score rows are padded to it
constexpr int MAX_CTAS = 1024;          // arrival counters at the head of the workspace
constexpr int WROWS = 16;               // heads of a warp: the rows of a product
constexpr int MAX_ROWS = 32;            // heads of a segment, at most

// BLOCKS: blocks of 8 heads of a segment: 1, 2, or 4
template <int D, bool F8, int BLOCKS>
struct Shape {
    // Two groups of four compute warps.  Segments of up to 16 heads: they take the tiles of a run in turn.  Of up
    // to 32 (SPLIT): both take every tile, 16 heads each, so that a key is read once for 32 heads.
    static constexpr int GROUPS = 2;
    static constexpr bool SPLIT = BLOCKS == 4;
    static constexpr int ROWS = SPLIT ? 32 : 16;            // rows kept for a segment's heads
    static constexpr int TK = F8 ? 128 : 64;                // keys per tile
    static constexpr int KS = TK / 4, NT = KS / 8;          // keys of a warp, in column tiles of 8
    static constexpr int CWARPS = 4 * GROUPS, THREADS = (CWARPS + 2) * 32;
    static constexpr int ROW = D * (F8 ? 1 : 2);            // bytes of a key
    static constexpr int BOX = ROW < 128 ? 64 : 128;        // bytes of a box row (= swizzle width)
    static constexpr float UP = F8 ? 16384.f : 1.f;         // weights, and so l and o, are held times this
    static constexpr int TILE = TK * ROW;                   // K or V of one tile
    // a multiple of the groups: a stage then always serves the same group, or both, which see each of its phases
    static constexpr int STAGES = TILE >= 16384 ? 4 : 8;
    static constexpr int LDO = D + 8;                       // padded row of the output exchange
    static constexpr int OFF_O = STAGES * 2 * TILE;
    static constexpr int OFF_ML = OFF_O + CWARPS * 8 * LDO * 4;
    static constexpr int OFF_PRE = OFF_ML + 2 * CWARPS * WROWS * 4;
    static constexpr int OFF_LEN = OFF_PRE + (kMaxSeqs + 1) * 4;
    static constexpr int LDQ = 2 * D + 16;                  // padded row of q (bytes)
    static constexpr int OFF_Q = (OFF_LEN + kMaxSeqs * 4 + 15) & ~15;
    static constexpr int OFF_BAR = OFF_Q + 2 * ROWS * LDQ;
    static constexpr int BYTES = OFF_BAR + (2 * STAGES + 4) * 8 + 80 + 1024;   // + alignment of the base
};

struct Args {
    AttentionDecode p;
    int group;      // q heads per kv head
    int chunks;     // segments per kv head: ceil(group / 16), or / 32 above 16
    int box_shift;  // log2 of the places of a page one box covers
    float *part;    // [cta][2][ROWS][D] partial outputs, unnormalised
    float2 *ml;     // [cta][2][ROWS] their running maximum and sum
    uint32_t *count;
    float2 *stat;   // [n_seqs][nq] (m, 1/l), with weights
    float *scores;  // [n_seqs][nq][ld_scores] scores in log2 units, with weights
    long long ld_scores;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
// C (16 x 8) += A (16 x 16) B (16 x 8), fp32 accumulation; bf16, or f16 operands with F8.
template <bool F8>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F8)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two e4m3 bytes -> two f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) {
    float2 r;
    asm("{.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(v));
    return r;
}
// p rounded to the operand type, and what the rounding left, rounded too.
template <bool F8>
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    if constexpr (F8) {
        hi = pack_f16x2(a, b);
        const float2 r = unpack_f16x2(hi);
        lo = pack_f16x2(a - r.x, b - r.y);
    } else {
        hi = pack_bf16x2(a, b);
        lo = pack_bf16x2(a - bf16_lo(hi), b - bf16_hi(hi));
    }
}
// Two bf16 with their magnitudes held to the largest finite one (NaN too).  One instruction per two values of V:
// 3% where segments have 32 heads (32 sequences of 20,000 to 24,000 tokens 124 -> 128 us), nothing measurable elsewhere.
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
    uint32_t r;
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(0x7f7f7f7fu), "r"(v));
    return r;
}
template <int THREADS>
__device__ __forceinline__ void compute_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a tile of swizzled box rows.
template <int D, bool F8>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    constexpr int TK = Shape<D, F8, 1>::TK;
    if constexpr (Shape<D, F8, 1>::BOX == 128) return (c >> 3) * (TK * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    else return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Walks the tiles (of TK keys) of a run: segment (b, u) with u = kv head * chunks + chunk, tile j of it.
template <int TK>
struct Walk {
    int b, u, j, len, tiles;
    __device__ __forceinline__ void start(int t, const int *pre, const int *lens, int n_seqs) {
        int lo = 0, hi = n_seqs;   // the b with pre[b] <= t < pre[b + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= t) lo = mid;
            else hi = mid;
        }
        b = lo;
        load(lens);
        const int off = t - pre[b];
        u = off / tiles;
        j = off - u * tiles;
    }
    __device__ __forceinline__ void load(const int *lens) {
        len = lens[b];
        tiles = (len + TK - 1) / TK;
    }
    // next segment (its tile 0); the caller knows that one follows
    __device__ __forceinline__ void next(int units, const int *lens) {
        j = 0;
        if (++u < units) return;
        u = 0;
        do {
            ++b;
            load(lens);
        } while (tiles == 0);
    }
};

template <int D, bool F8, int BLOCKS>
__global__ void __launch_bounds__(Shape<D, F8, BLOCKS>::THREADS, 1)
    attention_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const Args a) {
    using S = Shape<D, F8, BLOCKS>;
    constexpr int STAGES = S::STAGES, CWARPS = S::CWARPS, TK = S::TK, NT = S::NT, ROWS = S::ROWS;
    constexpr bool WIDE = BLOCKS > 1, SPLIT = S::SPLIT;   // WIDE: a warp has more than 8 heads
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float *sm_o = reinterpret_cast<float *>(smem + S::OFF_O);
    float *sm_m = reinterpret_cast<float *>(smem + S::OFF_ML), *sm_l = sm_m + CWARPS * WROWS;
    int *pre = reinterpret_cast<int *>(smem + S::OFF_PRE), *lens = reinterpret_cast<int *>(smem + S::OFF_LEN);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::OFF_BAR), *empty = full + STAGES;
    uint64_t *q_full = empty + STAGES, *q_empty = q_full + 2;
    volatile int *abort = reinterpret_cast<volatile int *>(q_empty + 2);
    int *s_last = const_cast<int *>(abort) + 1;   // [2]
    int *s_warp = s_last + 2;   // [CWARPS + 2] scan of the warps' sums

    const AttentionDecode &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = p.cache.nkv * a.chunks;

    pdl_trigger();
    if (tid == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + i, 2);
            mbar_init(empty + i, SPLIT ? CWARPS : 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(q_empty + i, CWARPS);
        }
        *abort = 0;
        fence_barrier_init();
    }
    pdl_wait();

    // pre[b] = tiles of the sequences before b: four sequences per thread, scanned over the block
    {
        int n[4], sum = 0;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = 4 * tid + i;
            n[i] = 0;
            if (b < p.n_seqs) {
                const int len = p.seq_lens[b], c = min(max(len, 0), p.max_len);
                lens[b] = c;
                if (len != c && blockIdx.x == 0) report(p.status, ST_BOUNDS);
                n[i] = (c + TK - 1) / TK * units;
            }
            sum += n[i];
        }
        int inc = sum;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        int at = inc - sum;
        for (int w = 0; w < warp; ++w) at += s_warp[w];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = 4 * tid + i;
            if (b <= p.n_seqs) pre[b] = at;
            at += n[i];
        }
        __syncthreads();
    }
    // the run of CTA c: T / G tiles, one more for the first T % G
    const unsigned T = (unsigned)pre[p.n_seqs], G = min(T, gridDim.x);   // CTAs that have a run
    // sequences without tokens: zero rows
    for (int b = blockIdx.x; b < p.n_seqs; b += gridDim.x)
        if (pre[b + 1] == pre[b])
            for (int i = tid; i < p.nq * D / 8; i += S::THREADS)
                *reinterpret_cast<uint4 *>(p.o + b * p.ld_o + 8 * i) = make_uint4(0, 0, 0, 0);
    if (blockIdx.x >= G) return;
    const unsigned run = T / G, longer = T - run * G;
    const int t0 = (int)(blockIdx.x * run + min(blockIdx.x, longer)), t1 = t0 + (int)(run + (blockIdx.x < longer));
    const auto owner = [&](int t) {   // the CTA whose run holds tile t
        const unsigned split = longer * (run + 1);
        return (int)((unsigned)t < split ? (unsigned)t / (run + 1) : longer + ((unsigned)t - split) / run);
    };
    const auto kv_head = [&](int u) { return a.chunks == 1 ? u : u / a.chunks; };

    Walk<TK> w;
    w.start(t0, pre, lens, p.n_seqs);

    if (warp >= CWARPS) {
        // ------------------------------------------------ producers: q and K, V
        const bool is_v = warp > CWARPS;
        // A batch of 32 boxes, one per lane, is looked up while the batch before it is issued: a lane
        // finds its tile's segment and its box's page, and later issues that box itself.
        const int tile_shift = (TK == 128 ? 7 : 6) - a.box_shift;   // log2 of the boxes of a tile
        const int boxes = 1 << tile_shift, per = 32 >> tile_shift;  // boxes of a tile, tiles of a batch
        const int my_tile = lane >> tile_shift, my_box = lane & (boxes - 1);
        const int page_mask = (1 << p.cache.page_shift) - 1;
        struct Box {
            int page, place, head, n;   // n: boxes that the tile has
            int b, u;                   // the tile's segment if it is the run's first of it, else b = -1
        };
        const auto look_up = [&](int t) {
            Box x{0, 0, 0, 0, -1, 0};
            if (t >= t1) return x;
            Walk<TK> v;
            v.start(t, pre, lens, p.n_seqs);
            const int key = v.j * TK + (my_box << a.box_shift);
            x.n = min(boxes, (v.len - v.j * TK + (1 << a.box_shift) - 1) >> a.box_shift);
            x.head = kv_head(v.u);
            if (v.j == 0 || t == t0) x.b = v.b, x.u = v.u;
            x.place = key & page_mask;
            if (my_box < x.n) x.page = p.table[(long long)v.b * p.ld_table + (key >> p.cache.page_shift)];
            return x;
        };
        int stage = 0, round = 0, segs = 0;
        bool ok = true;
        Box cur = look_up(t0 + my_tile);
        for (int tb = t0; tb < t1 && ok; tb += per) {
            const Box next = look_up(tb + per + my_tile);
            for (int i = 0; i < per && tb + i < t1; ++i) {
                // a segment's q rows come first, into one of two buffers
                const int qb = __shfl_sync(0xffffffffu, cur.b, i * boxes), qu = __shfl_sync(0xffffffffu, cur.u, i * boxes);
                if (qb >= 0 && !is_v) {
                    const int buf = segs & 1;
                    if (segs > 1) ok = mbar_wait(q_empty + buf, ((segs >> 1) - 1) & 1, abort);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const int head = kv_head(qu), chunk = qu - head * a.chunks;
                    const int rows = min(ROWS, a.group - chunk * ROWS);
                    if (lane == 0) mbar_arrive_expect_tx(q_full + buf, rows * D * 2);
                    __syncwarp();
                    if (lane < rows)
                        bulk_load(smem + S::OFF_Q + (buf * ROWS + lane) * S::LDQ,
                                  p.q + qb * p.ld_q + (long long)(head * a.group + chunk * ROWS + lane) * D, D * 2,
                                  q_full + buf);
                    ++segs;
                }
                if (round > 0) ok = mbar_wait(empty + stage, (round - 1) & 1, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t *tile = smem + (stage * 2 + is_v) * S::TILE;
                if (lane == i * boxes) mbar_arrive_expect_tx(full + stage, (cur.n << a.box_shift) * S::ROW);
                __syncwarp();
                if (my_tile == i && my_box < cur.n) {
                    int page = cur.page;
                    if (page < 0 || page >= p.cache.num_pages) {
                        report(p.status, ST_BOUNDS);
                        page = p.cache.num_pages;   // outside the map: the box is filled with zeros
                    }
                    #pragma unroll
                    for (int x = 0; x < S::ROW / S::BOX; ++x)
                        tma_load_4d(tile + x * (TK * S::BOX) + (my_box << a.box_shift) * S::BOX, is_v ? &tmV : &tmK,
                                    full + stage, x * (S::BOX / (F8 ? 1 : 2)), cur.place, cur.head, page);
                }
                if (++stage == STAGES) stage = 0, ++round;
            }
            cur = next;
        }
        if (!ok) {
            // a wait ran out: leave once the copies in flight have landed (each of these waits is limited too)
            if (lane == 0) {
                report(p.status, ST_TIMEOUT);
                *abort = 1;
                const int never = 0;
                const int issued = round * STAGES + stage;
                for (int f = max(0, issued - STAGES); f < issued; ++f)
                    mbar_wait(full + f % STAGES, (f / STAGES) & 1, &never);
                for (int f = max(0, segs - 2); f < segs; ++f) mbar_wait(q_full + (f & 1), (f >> 1) & 1, &never);
            }
            __syncwarp();
        }
        return;
    }

    // ---------------------------------------------------- compute warps
    const int g = lane >> 2, tq = lane & 3;   // fragment row and column pair
    const float base_scale = 1.4426950408889634f / sqrtf((float)D);
    const int group = warp >> 2, slice = (warp & 3) * S::KS;
    const int wrow = SPLIT ? group * WROWS : 0;   // this warp's first row of the segment's
    // this lane's row and 16-byte chunk in the ldmatrix of 16 keys: K (keys 0-7 / 8-15 as the column
    // tiles) and V (transposed, as the two halves of the contraction); e4m3 rows pair them the other way
    const int row_v = (lane & 7) + ((lane >> 3) & 1) * 8, chunk_v = lane >> 4;
    const int row_k = F8 ? row_v : (lane & 7) + (lane >> 4) * 8, chunk_k = F8 ? chunk_v : (lane >> 3) & 1;
    int stage = 0, round = 0, turn = 0;   // turn: the group whose tile this is
    // parts of segments that other CTAs share, joined at the end: [0] the run's first segment if it
    // began before the run, [1] its last if it goes on behind it
    struct Part {
        int b, u, seg, seg_end;
    } shared[2];
    shared[0].b = shared[1].b = -1;
    const int trow = tid / (D / 4), tcol = tid % (D / 4) * 4;   // this thread's output in the sums of the joins
    const auto store = [&](int b, int h, float4 v, float m, float l, float vs) {
        const float inv = 1.f / l, f = inv * vs;
        *reinterpret_cast<uint2 *>(p.o + b * p.ld_o + (long long)h * D + tcol) =
            make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
        if (a.stat && tcol == 0) a.stat[(long long)b * p.nq + h] = make_float2(m, inv * S::UP);
    };
    const auto give_up = [&]() {   // on the data; the control flow (barriers, counters) goes on to the end
        if (lane == 0) {
            report(p.status, ST_TIMEOUT);
            *abort = 1;
        }
        __syncwarp();
    };
    int segs = 0;

    for (int t = t0; t < t1; ++segs) {
        const int seg = t - w.j, seg_end = seg + w.tiles;   // this segment's tiles in the whole row of tiles
        const int j1 = min(w.tiles, t1 - seg);              // this run's part of it: [w.j, j1)
        const int kvh = kv_head(w.u), chunk = w.u - kvh * a.chunks, h0 = kvh * a.group + chunk * ROWS;
        const int rows = min(ROWS, a.group - chunk * ROWS);   // heads of the segment

        // q as the A operand: rows = heads, the contraction over d in steps of 16
        uint32_t qa[D / 16][WIDE ? 4 : 2];
        float scale0 = base_scale, scale1 = base_scale;
        {
            const float ks = F8 ? p.cache.k_scale[kvh] : 1.f;   // (its load goes out before the wait)
            if (!mbar_wait(q_full + (segs & 1), (segs >> 1) & 1, abort)) give_up();
            const uint8_t *q0 = smem + S::OFF_Q + ((segs & 1) * ROWS + wrow + g) * S::LDQ, *q1 = q0 + 8 * S::LDQ;
            const bool in0 = wrow + g < rows, in1 = WIDE && wrow + g + 8 < rows;
            #pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                // bf16: columns 2t, 2t+1 and 2t+8, 2t+9 of the step; e4m3: 4t .. 4t+3 (the bytes a
                // lane holds of a key), the same order on both sides of the product
                const int c0 = 16 * k + (F8 ? 4 * tq : 2 * tq), c1 = c0 + (F8 ? 2 : 8);
                qa[k][0] = in0 ? *reinterpret_cast<const uint32_t *>(q0 + 2 * c0) : 0u;
                qa[k][1] = in0 ? *reinterpret_cast<const uint32_t *>(q0 + 2 * c1) : 0u;
                if constexpr (WIDE) {
                    qa[k][2] = in1 ? *reinterpret_cast<const uint32_t *>(q1 + 2 * c0) : 0u;
                    qa[k][3] = in1 ? *reinterpret_cast<const uint32_t *>(q1 + 2 * c1) : 0u;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_empty + (segs & 1));
            if constexpr (F8) {
                #pragma unroll
                for (int r = 0; r < (WIDE ? 2 : 1); ++r) {
                    float top = 0.f;
                    #pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        #pragma unroll
                        for (int i = 0; i < 2; ++i)
                            top = fmaxf(top, fmaxf(fabsf(bf16_lo(qa[k][2 * r + i])), fabsf(bf16_hi(qa[k][2 * r + i]))));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // the largest |q| goes to [2^14, 2^15): exact but for elements 2^-29 of it and smaller
                    const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
                    const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
                    const float down = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
                    #pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        #pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t &x = qa[k][2 * r + i];
                            x = pack_f16x2(bf16_lo(x) * up, bf16_hi(x) * up);
                        }
                    (r ? scale1 : scale0) = base_scale * ks * down;
                }
            }
        }

        float o[D / 8][4];
        #pragma unroll
        for (int i = 0; i < D / 8; ++i)
            #pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        for (; w.j < j1; ++w.j, ++t, turn = turn + 1 == S::GROUPS ? 0 : turn + 1) {
            if (SPLIT || turn == group) {
                if (!mbar_wait(full + stage, round & 1, abort)) give_up();
                const int key0 = w.j * TK + slice;
                if (key0 < w.len) {
                    const uint32_t kt = smem_u32(smem + stage * 2 * S::TILE), vt = kt + S::TILE;
                    float s[NT][4] = {};
                    if constexpr (F8) {
                        #pragma unroll
                        for (int k = 0; k < D / 16; k += 2)
                            #pragma unroll
                            for (int n = 0; n < NT; n += 2) {
                                uint32_t r[4];   // (keys 0-7, 8-15) x (step k, k + 1)
                                ldsm4(r, kt + chunk_at<D, F8>(slice + 8 * n + row_k, k + chunk_k));
                                #pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    mma<F8>(s[n + (i & 1)], qa[k + i / 2][0], WIDE ? qa[k + i / 2][WIDE ? 2 : 0] : 0u,
                                            qa[k + i / 2][1], WIDE ? qa[k + i / 2][WIDE ? 3 : 0] : 0u,
                                            e4m3x2_f16x2(r[i]), e4m3x2_f16x2(r[i] >> 16));
                            }
                    } else {
                        float s2[NT][4] = {};   // even and odd steps: two chains of products per key tile
                        #pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            #pragma unroll
                            for (int n = 0; n < NT; n += 2) {
                                uint32_t r[4];
                                ldsm4(r, kt + chunk_at<D, F8>(slice + 8 * n + row_k, 2 * k + chunk_k));
                                #pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    mma<F8>(k & 1 ? s2[n + i] : s[n + i], qa[k][0], WIDE ? qa[k][WIDE ? 2 : 0] : 0u, qa[k][1],
                                            WIDE ? qa[k][WIDE ? 3 : 0] : 0u, r[2 * i], r[2 * i + 1]);
                            }
                        #pragma unroll
                        for (int n = 0; n < NT; ++n)
                            #pragma unroll
                            for (int k = 0; k < 4; ++k) s[n][k] += s2[n][k];
                    }
                    const bool tail = key0 + S::KS > w.len;
                    float x0 = -INFINITY, x1 = -INFINITY;
                    #pragma unroll
                    for (int n = 0; n < NT; ++n)
                        #pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            s[n][k] *= scale0;
                            if (WIDE) s[n][2 + k] *= scale1;
                            if (tail && key0 + 8 * n + 2 * tq + k >= w.len) s[n][k] = s[n][2 + k] = -INFINITY;
                            x0 = fmaxf(x0, s[n][k]);
                            if (WIDE) x1 = fmaxf(x1, s[n][2 + k]);
                        }
                    if (a.scores) {
                        #pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float *dst = a.scores + ((long long)w.b * p.nq + h0 + wrow + g) * a.ld_scores + key0 + 8 * n + 2 * tq;
                            if (wrow + g < rows) *reinterpret_cast<float2 *>(dst) = make_float2(s[n][0], s[n][1]);
                            if (WIDE && wrow + g + 8 < rows)
                                *reinterpret_cast<float2 *>(dst + 8 * a.ld_scores) = make_float2(s[n][2], s[n][3]);
                        }
                    }
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                    if (WIDE) {
                        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
                    }
                    // a larger maximum: rescale what has been summed (the first slice scales zeros)
                    if (__any_sync(0xffffffffu, x0 > m0 || (WIDE && x1 > m1))) {
                        const float n0 = fmaxf(m0, x0), c0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0);
                        float c1 = c0;
                        m0 = n0;
                        l0 *= c0;
                        if (WIDE) {
                            const float n1 = fmaxf(m1, x1);
                            c1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
                            m1 = n1;
                            l1 *= c1;
                        }
                        #pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            o[i][0] *= c0;
                            o[i][1] *= c0;
                            o[i][2] *= c1;
                            o[i][3] *= c1;
                        }
                    }
                    const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
                    #pragma unroll
                    for (int n = 0; n < NT; ++n)
                        #pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            s[n][k] = ex2(s[n][k] - z0) * S::UP;
                            l0 += s[n][k];
                            if (WIDE) {
                                s[n][2 + k] = ex2(s[n][2 + k] - z1) * S::UP;
                                l1 += s[n][2 + k];
                            }
                        }
                    #pragma unroll
                    for (int y = 0; y < NT / 2; ++y) {   // 16 keys at a time
                        uint32_t hi[4], lo[4];   // the A operand's four registers
                        split2<F8>(s[2 * y][0], s[2 * y][1], hi[0], lo[0]);
                        split2<F8>(s[2 * y + 1][0], s[2 * y + 1][1], hi[2], lo[2]);
                        if (WIDE) {
                            split2<F8>(s[2 * y][2], s[2 * y][3], hi[1], lo[1]);
                            split2<F8>(s[2 * y + 1][2], s[2 * y + 1][3], hi[3], lo[3]);
                        } else {
                            hi[1] = lo[0];
                            hi[3] = lo[2];
                        }
                        // values behind the sequence may be anything (0 * NaN): cleared in the last slice
                        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                        if (tail) {
                            const int left = w.len - key0 - 16 * y - 2 * tq;
                            keep0 = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
                            keep1 = (left > 8 ? 0xffffu : 0u) | (left > 9 ? 0xffff0000u : 0u);
                        }
                        #pragma unroll
                        for (int c = 0; c < S::ROW / 16; c += 2) {
                            uint32_t r[4];   // (keys 0-7, 8-15) x (chunk c, c + 1)
                            ldsm4t(r, vt + chunk_at<D, F8>(slice + 16 * y + row_v, c + chunk_v));
                            if (tail) {
                                r[0] &= keep0;
                                r[1] &= keep1;
                                r[2] &= keep0;
                                r[3] &= keep1;
                            }
                            #pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                if constexpr (F8) {
                                    // a lane holds columns 2n, 2n + 1 of two keys: even and odd columns as two tiles
                                    #pragma unroll
                                    for (int odd = 0; odd < 2; ++odd) {
                                        const uint32_t sel = odd ? 0x31u : 0x20u;
                                        const uint32_t b0 = e4m3x2_f16x2(__byte_perm(r[2 * i], 0u, sel));
                                        const uint32_t b1 = e4m3x2_f16x2(__byte_perm(r[2 * i + 1], 0u, sel));
                                        mma<F8>(o[2 * (c + i) + odd], hi[0], hi[1], hi[2], hi[3], b0, b1);
                                        if (WIDE) mma<F8>(o[2 * (c + i) + odd], lo[0], lo[1], lo[2], lo[3], b0, b1);
                                    }
                                } else {
                                    mma<F8>(o[c + i], hi[0], hi[1], hi[2], hi[3], r[2 * i], r[2 * i + 1]);
                                    // an infinite value is in the sum already: times a remainder of 0 or less it would be NaN
                                    if (WIDE) mma<F8>(o[c + i], lo[0], lo[1], lo[2], lo[3], finite2(r[2 * i]), finite2(r[2 * i + 1]));
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + stage);
            }
            if (++stage == STAGES) stage = 0, ++round;
        }

        // ------------------------------------------------ join the warps' parts
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        if (WIDE) {
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        }
        if (tq == 0) {
            sm_m[warp * WROWS + g] = m0;
            sm_l[warp * WROWS + g] = l0;
            sm_m[warp * WROWS + g + 8] = m1;
            sm_l[warp * WROWS + g + 8] = l1;
        }
        compute_sync<CWARPS * 32>();
        const bool whole = seg >= t0 && seg_end <= t1;
        const float vs = F8 ? p.cache.v_scale[kvh] : 1.f;
        const int slot = 2 * blockIdx.x + (seg < t0 ? 0 : 1);
        if (!whole) shared[seg < t0 ? 0 : 1] = Part{w.b, w.u, seg, seg_end};
        #pragma unroll
        for (int r8 = 0; r8 < (WIDE ? 16 : 8); r8 += 8) {
            // the warps that share rows: all, or (SPLIT) those of a group
            constexpr int SHARE = SPLIT ? 4 : CWARPS;
            float top = -INFINITY;
            #pragma unroll
            for (int i = 0; i < SHARE; ++i) top = fmaxf(top, sm_m[((SPLIT ? 4 * group : 0) + i) * WROWS + r8 + g]);
            const float mine = r8 ? m1 : m0, f = mine == -INFINITY ? 0.f : ex2(mine - top);
            float *dst = sm_o + (warp * 8 + g) * S::LDO;
            const auto out = [&](int i, int k) {
                if constexpr (WIDE) return o[i][r8 / 4 + k] * f;
                // (an infinite sum stays: the remainders' is NaN there)
                return (fabsf(o[i][k]) == INFINITY ? o[i][k] : o[i][k] + o[i][k + 2]) * f;
            };
            #pragma unroll
            for (int i = 0; i < D / 8; i += 2) {
                if constexpr (F8) {   // even and odd columns of 16
                    *reinterpret_cast<float4 *>(dst + 8 * i + 4 * tq) =
                        make_float4(out(i, 0), out(i + 1, 0), out(i, 1), out(i + 1, 1));
                } else {
                    *reinterpret_cast<float2 *>(dst + 8 * i + 2 * tq) = make_float2(out(i, 0), out(i, 1));
                    *reinterpret_cast<float2 *>(dst + 8 * i + 8 + 2 * tq) = make_float2(out(i + 1, 0), out(i + 1, 1));
                }
            }
            compute_sync<CWARPS * 32>();
            #pragma unroll
            for (int q = 0; q < (SPLIT ? 2 : 1); ++q) {
                const int row = q * WROWS + r8 + trow;
                if (trow >= 8 || row >= rows) continue;
                float mm = -INFINITY, ll = 0.f;
                #pragma unroll
                for (int i = q * 4; i < q * 4 + SHARE; ++i) mm = fmaxf(mm, sm_m[i * WROWS + r8 + trow]);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                #pragma unroll
                for (int i = q * 4; i < q * 4 + SHARE; ++i) {
                    const float wm = sm_m[i * WROWS + r8 + trow];
                    ll += wm == -INFINITY ? 0.f : sm_l[i * WROWS + r8 + trow] * ex2(wm - mm);
                    const float4 x = *reinterpret_cast<const float4 *>(sm_o + (i * 8 + trow) * S::LDO + tcol);
                    acc.x += x.x;
                    acc.y += x.y;
                    acc.z += x.z;
                    acc.w += x.w;
                }
                if (whole) {
                    store(w.b, h0 + row, acc, mm, ll, vs);
                } else {
                    *reinterpret_cast<float4 *>(a.part + ((long long)slot * ROWS + row) * D + tcol) = acc;
                    if (tcol == 0) a.ml[slot * ROWS + row] = make_float2(mm, ll);
                }
            }
            compute_sync<CWARPS * 32>();
        }
        if (t < t1) w.next(units, lens);
    }

    // ---------------------------------------------------- join the parts of shared segments
    // The CTA whose part arrives last joins them, in the order of the keys.  More parts than one batch of
    // loads holds are joined in two steps: groups of GROUP first, each by the last of its CTAs into the
    // place of its first part, then the groups by the last of those (26,000 and 37,000 tokens, one kv head of 64:
    // 22.5 -> 14.1 us).  The result is the same whoever is last.  (The barrier at the end of the
    // loop above orders all threads' parts before the release.)
    if (shared[0].b < 0 && shared[1].b < 0) return;
    constexpr int LPR = D / 4, BATCH = LPR < 24 ? LPR : 24, GROUP = 16;   // LPR: lanes of a row
    const auto arrive = [&](uint32_t *count, int n) {   // whether this is the last of n; the counter is then 0 again
        uint32_t before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
        if (before != (uint32_t)(n - 1)) return 0;
        *count = 0u;
        return 1;
    };
    // part i of a segment whose first CTA is `first`: slot 1 of that one (the segment begins in its run), slot 0 of the others
    const auto slot_of = [&](int first, int i) { return 2 * (first + i) + (i == 0 ? 1 : 0); };
    const auto group_of = [&](int first, int n) { return n > BATCH ? ((int)blockIdx.x - first) / GROUP * GROUP : 0; };
    const auto size_of = [&](int n, int begin) { return n > BATCH ? min(GROUP, n - begin) : n; };
    if (tid < 2) {
        const Part &x = shared[tid];
        s_last[tid] = 0;
        if (x.b >= 0) {
            const int first = owner(x.seg), n = owner(x.seg_end - 1) - first + 1, begin = group_of(first, n);
            s_last[tid] = arrive(a.count + slot_of(first, begin), size_of(n, begin));
        }
    }
    compute_sync<CWARPS * 32>();
    #pragma unroll 1
    for (int x = 0; x < 2; ++x) {
        if (!s_last[x]) continue;
        const Part y = x ? shared[1] : shared[0];
        const int first = owner(y.seg), n = owner(y.seg_end - 1) - first + 1, begin = group_of(first, n);
        const int kvh = kv_head(y.u), chunk = y.u - kvh * a.chunks;
        const int rows = min(ROWS, a.group - chunk * ROWS);
        const float vs = F8 ? p.cache.v_scale[kvh] : 1.f;
        // The parts begin, begin + STEP, ... (count of them): up to BATCH at a time, all their loads in flight.  A lane
        // takes four columns of each, and of one part (lane li: part li of the batch) the row's maximum and sum.
        const auto join = [&](auto step, int begin, int count, bool final) {
            constexpr int STEP = decltype(step)::value;
            #pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += CWARPS * 32 / LPR) {
                const int li = lane % LPR, row = (r0 + trow) % ROWS;   // (rows past the segment's last: not stored)
                const long long head = (long long)slot_of(first, begin) * ROWS + row;   // the first, then the others
                const long long rest = (long long)(2 * (first + begin)) * ROWS + row;
                const auto at = [&](int k) { return k == 0 ? head : rest + k * (2 * STEP * ROWS); };
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                float mm = -INFINITY, ll = 0.f;
                for (int i0 = 0; i0 < count; i0 += BATCH) {
                    float2 ml = make_float2(-INFINITY, 0.f);
                    if (li < BATCH && i0 + li < count) ml = __ldcg(a.ml + at(i0 + li));
                    float4 v[BATCH];
                    #pragma unroll
                    for (int k = 0; k < BATCH; ++k)
                        v[k] = i0 + k < count ? __ldcg(reinterpret_cast<const float4 *>(a.part + at(i0 + k) * D + tcol))
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
                    float top = ml.x;
                    #pragma unroll
                    for (int off = LPR / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    top = fmaxf(top, mm);
                    const float c = mm == -INFINITY ? 0.f : ex2(mm - top), f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
                    mm = top;
                    ll = fmaf(ll, c, ml.y * f);
                    acc = make_float4(acc.x * c, acc.y * c, acc.z * c, acc.w * c);
                    #pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const float fk = __shfl_sync(0xffffffffu, f, k, LPR);   // 0 past the last part
                        acc.x = fmaf(v[k].x, fk, acc.x);
                        acc.y = fmaf(v[k].y, fk, acc.y);
                        acc.z = fmaf(v[k].z, fk, acc.z);
                        acc.w = fmaf(v[k].w, fk, acc.w);
                    }
                }
                #pragma unroll
                for (int off = LPR / 2; off > 0; off >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, off);
                if (r0 + trow < rows) {
                    if (final) {
                        store(y.b, kvh * a.group + chunk * ROWS + row, acc, mm, ll, vs);
                    } else {
                        *reinterpret_cast<float4 *>(a.part + head * D + tcol) = acc;
                        if (tcol == 0) a.ml[head] = make_float2(mm, ll);
                    }
                }
            }
        };
        join(std::integral_constant<int, 1>{}, begin, size_of(n, begin), n <= BATCH);
        if (n > BATCH) {
            compute_sync<CWARPS * 32>();
            const int groups = (n + GROUP - 1) / GROUP;
            if (tid == 0) s_last[x] = arrive(a.count + 2 * MAX_CTAS + first, groups);
            compute_sync<CWARPS * 32>();
            if (s_last[x]) join(std::integral_constant<int, GROUP>{}, 0, groups, true);
        }
    }
}

// weight_out[b][i] = weight_in[b][i] + sum over the q heads of their p_i, from the stored scores and
// each head's (m, 1/l).  A CTA takes 128 keys of a sequence, four per lane (512 contiguous bytes a warp
// load); warp w sums the heads w, w + 8, ... in order and the eight sums are added in order, so the
// result is the same on every run.  Reads 4 bytes per head and key, mostly from L2 where the
// attention left them.
__global__ void __launch_bounds__(256) attention_weight_kernel(const AttentionDecode p, const float *scores,
                                                               const float2 *stat, long long ld_scores) {
    __shared__ float4 part[8][WK / 4];
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.y, i0 = blockIdx.x * WK, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = min(max(p.seq_lens[b], 0), p.max_len);
    if (i0 >= len) return;
    const int i = i0 + threadIdx.x;
    const bool out = threadIdx.x < WK && i < len;
    const float start = out && p.weight_in ? p.weight_in[b * p.ld_weight + i] : 0.f;
    const float *s = scores + (long long)b * p.nq * ld_scores + i0 + 4 * lane;   // rows are padded to WK
    const float2 *st = stat + (long long)b * p.nq;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    #pragma unroll 8
    for (int h = warp; h < p.nq; h += 8) {
        const float4 x = *reinterpret_cast<const float4 *>(s + h * ld_scores);   // (behind the sequence: anything, unused)
        const float2 ml = st[h];
        acc.x = fmaf(ex2(x.x - ml.x), ml.y, acc.x);
        acc.y = fmaf(ex2(x.y - ml.x), ml.y, acc.y);
        acc.z = fmaf(ex2(x.z - ml.x), ml.y, acc.z);
        acc.w = fmaf(ex2(x.w - ml.x), ml.y, acc.w);
    }
    part[warp][lane] = acc;
    __syncthreads();
    if (out) {
        float sum = 0.f;
        #pragma unroll
        for (int w = 0; w < 8; ++w) sum += reinterpret_cast<const float *>(part[w])[threadIdx.x];
        p.weight_out[b * p.ld_weight + i] = start + sum;
    }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace: arrival counters, partial outputs, their (m, l), then with weights (m, 1/l) and scores.
struct Layout {
    size_t part, ml, stat, scores, bytes;
    long long ld_scores;
};
Layout layout(int ctas, int n_seqs, int nq, int max_len, bool weights) {
    Layout y;
    y.part = 3 * MAX_CTAS * sizeof(uint32_t);
    y.ml = y.part + (size_t)ctas * 2 * MAX_ROWS * 128 * sizeof(float);
    y.stat = y.ml + up256((size_t)ctas * 2 * MAX_ROWS * sizeof(float2));
    y.ld_scores = (max_len + WK - 1) / WK * WK;
    y.scores = y.stat + (weights ? up256((size_t)n_seqs * nq * sizeof(float2)) : 0);
    y.bytes = y.scores + (weights ? (size_t)n_seqs * nq * (size_t)y.ld_scores * sizeof(float) : 0);
    return y;
}

template <int D, bool F8, int BLOCKS>
cudaError_t launch_kernel(const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, int grid, cudaStream_t st) {
    static std::atomic<bool> ready[kMaxDevices];   // the shared-memory opt-in, per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    constexpr int bytes = Shape<D, F8, BLOCKS>::BYTES;
    static_assert(bytes <= 232448, "shared memory of one CTA");
    if (!ready[dev].load()) {
        cudaError_t e = cudaFuncSetAttribute(attention_decode_kernel<D, F8, BLOCKS>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ready[dev].store(true);
    }
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3(grid), dim3(Shape<D, F8, BLOCKS>::THREADS), bytes, st, at);
    return cudaLaunchKernelEx(&cfg, attention_decode_kernel<D, F8, BLOCKS>, tk, tv, a);
}

}  // namespace

size_t attention_decode_workspace_bytes(int num_sms, int n_seqs, int nq, int max_len, bool weights) {
    if (num_sms <= 0 || num_sms > MAX_CTAS || n_seqs < 0 || n_seqs > kMaxSeqs || nq < 1 || nq > 65536 || max_len < 0 ||
        max_len > kMaxCacheLen ||
        // tiles of 64 or 128 keys, counted in 32 bits; the producers look up to two batches of 32 boxes past a run's end
        (long long)n_seqs * nq * (((long long)max_len + 63) / 64) > INT_MAX - 64)
        return 0;
    return layout(num_sms, n_seqs, nq, max_len, weights).bytes;
}

cudaError_t launch_attention_decode(const AttentionDecode &p, cudaStream_t st) {
    if (p.n_seqs <= 0) return cudaSuccess;
    const int sms = device_num_sms();
    const Layout y = layout(sms, p.n_seqs, p.nq, p.max_len, p.weight_out != nullptr);
    char *ws = static_cast<char *>(p.workspace);
    Args a{};
    a.p = p;
    a.group = p.nq / p.cache.nkv;
    // More than 16 heads of a kv head: segments of 32 heads read a key once, segments of 16 once for every 16
    // heads but from L2 where the cache fits there, with twice the segments and half the rows to join.  40 q heads over 2 kv
    // heads of 128, 32 and 8 sequences of 20,000 to 24,000 tokens (787 and 197 MB by max_len): 128 and 46 us against
    // 211 and 54; 64 over 1, two sequences of 25,000 (25 MB): 35 us against 24; e4m3, 8 sequences (98 MB): 45 against 43.
    const double bytes = 2.0 * p.n_seqs * p.max_len * p.cache.nkv * p.cache.d * (p.cache.f8 ? 1 : 2);
    const bool split = a.group > WROWS && bytes > 1e8;
    const int rows = split ? 2 * WROWS : WROWS;   // heads of a segment
    a.chunks = (a.group + rows - 1) / rows;
    a.box_shift = std::min(6, p.cache.page_shift);
    a.count = reinterpret_cast<uint32_t *>(ws);
    a.part = reinterpret_cast<float *>(ws + y.part);
    a.ml = reinterpret_cast<float2 *>(ws + y.ml);
    if (p.weight_out) {
        a.stat = reinterpret_cast<float2 *>(ws + y.stat);
        a.scores = reinterpret_cast<float *>(ws + y.scores);
        a.ld_scores = y.ld_scores;
    }
    CUtensorMap tk, tv;
    if (!make_tmap_cache(&tk, p.cache, p.cache.k) || !make_tmap_cache(&tv, p.cache, p.cache.v))
        return cudaErrorInvalidValue;
    // one CTA per SM, fewer where the lengths cannot hold as many tiles
    const long long most = (long long)p.n_seqs * p.cache.nkv * a.chunks * ((p.max_len + (p.cache.f8 ? 127 : 63)) / (p.cache.f8 ? 128 : 64));
    const int grid = (int)std::min<long long>(sms, std::max<long long>(most, 1));
    const auto run = [&](auto d, auto f8) {
        constexpr int D = decltype(d)::value;
        constexpr bool F8 = decltype(f8)::value;
        return a.group <= 8 ? launch_kernel<D, F8, 1>(tk, tv, a, grid, st)
                            : (split ? launch_kernel<D, F8, 4>(tk, tv, a, grid, st)
                                     : launch_kernel<D, F8, 2>(tk, tv, a, grid, st));
    };
    const std::integral_constant<int, 128> d128;
    const std::integral_constant<int, 64> d64;
    const cudaError_t e = p.cache.d == 128 ? (p.cache.f8 ? run(d128, std::true_type{}) : run(d128, std::false_type{}))
                                           : (p.cache.f8 ? run(d64, std::true_type{}) : run(d64, std::false_type{}));
    if (e != cudaSuccess || !p.weight_out || p.max_len == 0) return e;
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = pdl_config(dim3((p.max_len + WK - 1) / WK, p.n_seqs), dim3(256), 0, st, at);
    return cudaLaunchKernelEx(&cfg, attention_weight_kernel, p, (const float *)a.scores, (const float2 *)a.stat, a.ld_scores);
}

}  // namespace h3
