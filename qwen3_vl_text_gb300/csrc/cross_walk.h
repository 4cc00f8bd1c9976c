// How attention_cross.cu lays its work end to end and cuts it into runs: the arithmetic alone, which the kernel and
// a host program (the tests) compile alike.
#pragma once

#include <algorithm>

#ifdef __CUDACC__
#define H3_WALK __device__ __forceinline__
#else
#define H3_WALK inline
#endif

namespace h3 {
namespace cross {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

constexpr int TQ = 128, TK = 128;           // rows of a tile, keys of a step
enum { ROWS = 0, PAGES = 1, PAGES8 = 2 };   // keys: packed rows, bf16 pages, e4m3 pages
constexpr int FIXED = 2;   // weight of an item's beginning and end (a pair's step: 2)

// Offsets come from the device and may be anything: each is held to [0, most] ...
H3_WALK int clamped(int x, int most) { return min(max(x, 0), most); }
// ... and those of queries then to none before it, so that no row of queries is in two segments: weight_bound holds for such.
H3_WALK void ascend(int *v, int n) {
    for (int i = 1; i < n; ++i) v[i] = max(v[i], v[i - 1]);
}

// The group [rows[g], rows[g + 1]) of n that sequence b is in, -1: none.  Of offsets that run back some group that holds b
// or none, the same for every caller.
H3_WALK int group_of(const int *rows, int n, int b) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (rows[mid] <= b) lo = mid;
        else hi = mid;
    }
    return n > 0 && rows[lo] <= b && b < rows[lo + 1] ? lo : -1;
}

// Weight of the items of one kv head's share of a segment: pairs of row tiles and a last single one.
H3_WALK int unit_weight(int tiles, int steps) { return (tiles >> 1) * (2 * steps + FIXED) + (tiles & 1) * (steps + FIXED); }

// The segments, in shared memory: tokens [cq[s], cq[s + 1]), keys [ck[s], ck[s + 1]) or (pages) the first ck[s] of s;
// pre[s]: weight of the segments before s.
struct Segments {
    const int *pre, *cq, *ck;
};
template <int MODE>
H3_WALK int seg_keys(const Segments &g, int s) {
    return MODE == ROWS ? max(g.ck[s + 1] - g.ck[s], 0) : g.ck[s];
}
H3_WALK int seg_tokens(const Segments &g, int s) { return max(g.cq[s + 1] - g.cq[s], 0); }

// Walks the items of a run [w0, end) of weights.
template <int MODE>
struct Walk {
    // the segment: index, keys, steps, tokens, tiles
    int s, len, steps, n, tiles;
    // the item: kv head and share of its group, block of two tiles, first token in the segment, tokens of its tiles
    // (n_b 0: single), steps of this run [j0, j1), first weight, weight of a step - 1
    int head, chunk, blk, tok0, n_a, n_b, j0, j1, start, shift;
    int w0, end;
    bool snap;   // the run takes the items that begin in it, whole (packed rows only)

    H3_WALK void load(const Segments &g, int tok) {
        len = seg_keys<MODE>(g, s);
        steps = (len + TK - 1) / TK;
        n = seg_tokens(g, s);
        tiles = (n + tok - 1) / tok;
    }
    H3_WALK void begin(int first, int behind, bool whole, const Segments &g, int n_segs, int tok, int chunks) {
        snap = MODE == ROWS && whole;
        w0 = first;
        end = behind;
        start = behind;
        j1 = -1;
        if (first >= behind) return;
        int lo = 0, hi = n_segs;   // the s with pre[s] <= w0 < pre[s + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (g.pre[mid] <= w0) lo = mid;
            else hi = mid;
        }
        s = lo;
        load(g, tok);
        int off = w0 - g.pre[s];
        const int pair = 2 * steps + FIXED, unit = unit_weight(tiles, steps), u = off / unit;
        off -= u * unit;
        head = u / chunks;
        chunk = u - head * chunks;
        blk = min(off / pair, tiles >> 1);
        start = w0 - (off - blk * pair);
        shift = 2 * blk + 1 < tiles ? 1 : 0;
        if (MODE == ROWS && snap && start < w0) j1 = 0;   // the run before has it: on to the next
    }
    H3_WALK int weight() const { return (steps << shift) + FIXED; }
    H3_WALK bool next(const Segments &g, int tok, int chunks, int nkv) {
        while (true) {
            if (j1 >= 0 && start < end) {   // on from the item before
                start += weight();
                if (start >= end) return false;
                if (2 * ++blk >= tiles) {
                    blk = 0;
                    if (++chunk == chunks) {
                        chunk = 0;
                        if (++head == nkv) {
                            head = 0;
                            do ++s;
                            while (g.pre[s + 1] == g.pre[s]);
                            load(g, tok);
                        }
                    }
                }
            }
            if (start >= end) return false;
            shift = 2 * blk + 1 < tiles ? 1 : 0;
            tok0 = blk * 2 * tok;
            n_a = min(tok, n - tok0);
            n_b = shift ? min(tok, n - tok0 - tok) : 0;
            // step j belongs to the run that holds weight start + (j << shift)
            j0 = MODE == ROWS && snap ? 0 : max((w0 - start + shift) >> shift, 0);
            j1 = MODE == ROWS && snap ? steps : min((end - start + shift) >> shift, steps);
            if (j0 < j1) return true;
        }
    }
};

// The runs: T / G weights each, one more for the first T % G.
struct Runs {
    unsigned run, longer;
    H3_WALK Runs(unsigned T, unsigned G) : run(G ? T / G : 0), longer(T - run * G) {}
    H3_WALK int first(unsigned c) const { return (int)(c * run + min(c, longer)); }
    H3_WALK int owner(unsigned w) const {
        const unsigned split = longer * (run + 1);
        return (int)(w < split ? w / (run + 1) : longer + (w - split) / run);
    }
};

// Bound on the weight of a call, for any lengths of segments that have no row of queries in common; -1 where it passes 2e9.
inline long long weight_bound(int Tq, int max_keys, int n_segs, int nq, int nkv) {
    const int group = nq / nkv, gc = std::min(group, TQ), chunks = (group + TQ - 1) / TQ, tok = TQ / gc;
    // (every segment's last tile of rows may be partial)
    const double tiles = (double)Tq / (2 * tok) + std::min(n_segs, Tq);
    const double steps = (double)max_keys / TK + 1;
    const double most = (double)nkv * chunks * tiles * (2 * steps + FIXED);
    return most > 2e9 ? -1 : (long long)most + 1;
}

// Few rows, by attention_decode.cu: tiles of 64 keys that a segment of `tokens` queries over `keys` keys takes, the rows of each
// kv head (its group of q heads of every query) `rows` at a time ...
H3_WALK int packed_tiles(int tokens, int keys, int group, int nkv, int rows) {
    return (keys + 63) / 64 * nkv * ((tokens * group + rows - 1) / rows);
}
// ... and a bound on all segments', 8 rows at a time; -1 where 32 bits do not hold it and the runs' look-ahead.
inline long long packed_bound(int Tq, int Tk, int n_segs, int nq, int nkv) {
    const long long chunks = ((long long)Tq * (nq / nkv) + 7) / 8 + n_segs, most = nkv * chunks * ((long long)Tk / 64 + 1);
    return most > 2147483647LL - 65 ? -1 : most;
}

}  // namespace cross
}  // namespace h3
