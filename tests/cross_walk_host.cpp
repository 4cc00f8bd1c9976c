// The walk of attention_cross.cu on the host: every step of every item by exactly one run, cut items in parts that follow
// one another, rows and keys inside the call.  Prints "ok <cases>", or what is wrong.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <unordered_map>
#include <vector>

#include "cross_walk.h"

using namespace h3::cross;

namespace {

std::mt19937 rng(5);
int below(int n) { return n > 0 ? (int)(rng() % (unsigned)n) : 0; }

[[noreturn]] void wrong(const char *f, ...) {
    va_list a;
    va_start(a, f);
    vprintf(f, a);
    va_end(a);
    printf("\n");
    exit(1);
}

struct Case {
    int Tq, Tk, nq, nkv;
    std::vector<int> cq, ck;   // offsets as the kernel has them
};

// Offsets as the kernel takes them: of queries in order, of keys each by itself.
std::vector<int> taken(std::vector<int> v, int most, bool in_order = true) {
    for (int &x : v) x = clamped(x, most);
    if (in_order) ascend(v.data(), (int)v.size());
    return v;
}

// What the kernel does with a call's segments: weights laid end to end, cut into a run per CTA, walked.
template <int MODE>
void check(const Case &c, int sms, bool whole, bool every_step) {
    const int S = (int)c.cq.size() - 1, group = c.nq / c.nkv, gc = std::min(group, TQ), chunks = (group + TQ - 1) / TQ, tok = TQ / gc;
    const long long bound = weight_bound(c.Tq, c.Tk, S, c.nq, c.nkv);
    if (bound < 0) return;
    std::vector<int> pre(S + 1);
    const Segments g{pre.data(), c.cq.data(), c.ck.data()};
    long long T = 0;
    for (int s = 0; s < S; ++s) {
        pre[s] = (int)T;
        const long long tiles = (seg_tokens(g, s) + tok - 1) / tok, steps = (seg_keys<MODE>(g, s) + TK - 1) / TK;
        if (steps) T += (long long)c.nkv * chunks * ((tiles >> 1) * (2 * steps + FIXED) + (tiles & 1) * (steps + FIXED));
        if (T > bound) wrong("weight %lld of the first %d segments, bound %lld", T, s + 1, bound);
    }
    pre[S] = (int)T;
    const unsigned G = std::min((unsigned)T / 2, (unsigned)sms);
    if (!G) return;
    const Runs runs((unsigned)T, G);
    struct Seen {
        long long steps = 0;
        int parts = 0, owner = 0, of = 0;
    };
    std::unordered_map<uint64_t, Seen> seen;   // by segment, head, chunk, block
    int last_end = 0;
    for (unsigned r = 0; r < G; ++r) {
        Walk<MODE> w;
        memset(&w, 0x5a, sizeof w);
        if (runs.first(r) != last_end) wrong("run %u begins at %d, not %d", r, runs.first(r), last_end);
        last_end = runs.first(r + 1);
        if (last_end - runs.first(r) < 2) wrong("run %u is shorter than a step", r);
        w.begin(runs.first(r), last_end, whole, g, S, tok, chunks);
        while (w.next(g, tok, chunks, c.nkv)) {
            if (w.s < 0 || w.s >= S || w.head < 0 || w.head >= c.nkv || w.chunk < 0 || w.chunk >= chunks || w.blk < 0 ||
                2 * w.blk >= w.tiles || w.j0 < 0 || w.j1 > w.steps || w.n_a < 1 || w.n_b < 0)
                wrong("an item outside: segment %d head %d chunk %d block %d", w.s, w.head, w.chunk, w.blk);
            const long long row0 = (long long)c.cq[w.s] + w.tok0, row1 = row0 + w.n_a + w.n_b;
            if (row0 < 0 || row1 > c.Tq || row1 > c.cq[w.s + 1]) wrong("rows %lld to %lld of %d", row0, row1, c.Tq);
            const long long key0 = MODE == ROWS ? c.ck[w.s] : 0;
            if (key0 < 0 || key0 + w.len > c.Tk) wrong("keys %lld and %d on of %d", key0, w.len, c.Tk);
            if (whole && MODE == ROWS && (w.j0 || w.j1 != w.steps)) wrong("a whole item is cut");
            Seen &x = seen[(((uint64_t)w.s * c.nkv + w.head) * chunks + w.chunk) * 16777216 + w.blk];
            const int owner = runs.owner(w.start), parts = runs.owner(w.start + ((w.steps - 1) << w.shift)) - owner + 1;
            if (x.steps != w.j0) wrong("step %d follows step %lld", w.j0, x.steps);
            x.steps += w.j1 - w.j0;
            if (w.j0 > 0 || w.j1 < w.steps) {
                if (x.parts == 0) x.owner = owner, x.of = parts;
                if (owner != x.owner || parts != x.of || (int)r != owner + x.parts) wrong("part %d of %d in run %u, the first in %d", x.parts, parts, r, owner);
                ++x.parts;
            }
            if (x.steps == w.steps && x.parts != x.of) wrong("%d parts of %d", x.parts, x.of);
        }
    }
    if (!every_step) return;
    uint64_t want = 0;
    for (int s = 0; s < S; ++s)
        if (seg_keys<MODE>(g, s) > 0) {
            const int tiles = (seg_tokens(g, s) + tok - 1) / tok, steps = (seg_keys<MODE>(g, s) + TK - 1) / TK;
            for (int h = 0; h < c.nkv; ++h)
                for (int y = 0; y < chunks; ++y)
                    for (int b = 0; 2 * b < tiles; ++b, ++want) {
                        const auto i = seen.find((((uint64_t)s * c.nkv + h) * chunks + y) * 16777216 + b);
                        if (i == seen.end() || i->second.steps != steps) wrong("segment %d head %d block %d: steps missing", s, h, b);
                    }
        }
    if (want != seen.size()) wrong("%zu items of %llu", seen.size(), (unsigned long long)want);
}

void check_all(const Case &c, int sms, bool every_step) {
    check<ROWS>(c, sms, false, every_step);
    check<ROWS>(c, sms, true, every_step);
    Case p = c;   // pages: the first ck[s] keys of row s of a table
    for (size_t s = 0; s + 1 < c.ck.size(); ++s) p.ck[s] = std::max(c.ck[s + 1] - c.ck[s], 0);
    check<PAGES>(p, sms, false, every_step);

    for (int b = -1; b < (int)c.cq.size() + 3; ++b) {   // (as offsets of sequences)
        const int S = (int)c.cq.size() - 1, at = group_of(c.cq.data(), S, b);
        int want = -1;
        for (int i = 0; i < S; ++i)
            if (c.cq[i] <= b && b < c.cq[i + 1]) want = i;
        if (at != want) wrong("sequence %d in group %d, not %d", b, at, want);
    }

    const long long bound = packed_bound(c.Tq, c.Tk, (int)c.cq.size() - 1, c.nq, c.nkv);
    long long tiles = 0;
    for (size_t s = 0; s + 1 < c.cq.size() && bound >= 0 && (long long)c.Tq * (c.nq / c.nkv) <= 32768; ++s) {
        tiles += packed_tiles(c.cq[s + 1] - c.cq[s], p.ck[s], c.nq / c.nkv, c.nkv, 8);
        if (tiles > bound) wrong("%lld tiles of the first %zu segments, bound %lld", tiles, s + 1, bound);
    }
}

// Segments that follow one another, empty ones among them.
int ascending(int cases) {
    for (int it = 0; it < cases; ++it) {
        Case c;
        const int S = 1 + below(it % 3 ? 4 : 70), same = below(2), kk = below(1500), qq = below(600);
        c.nkv = 1 + below(10);
        c.nq = c.nkv * (1 + below(it % 4 ? 16 : 300));
        c.cq.assign(S + 1, 0);
        c.ck.assign(S + 1, 0);
        for (int s = 0; s < S; ++s) {
            c.cq[s + 1] = c.cq[s] + (same ? qq : below(below(4) ? 300 : 1));
            c.ck[s + 1] = c.ck[s] + (same ? kk : below(below(5) ? 900 : 1));
        }
        c.Tq = c.cq[S] + below(3);
        c.Tk = c.ck[S] + below(3);
        check_all(c, it % 5 ? 1 + below(152) : 152, true);
    }
    return cases;
}

// Offsets of any values, as a device array may hold them: clamped and put in order like the kernel's.
int any_offsets(int cases) {
    for (int it = 0; it < cases; ++it) {
        Case c;
        const int S = 1 + below(it % 2 ? 8 : 1024), kind = it % 4;
        c.nkv = 1 << below(4);
        c.nq = c.nkv * (1 + below(16));
        c.Tq = 1 + below(it % 3 ? 2000 : 40000);
        c.Tk = 1 + below(it % 3 ? 5000 : 300000);
        std::vector<int> q(S + 1), k(S + 1);
        for (int s = 0; s <= S; ++s) {
            const auto value = [&](int most) {
                if (kind == 0) return s % 2 ? most : 0;                       // back to the beginning every second time
                if (kind == 1) return (int)(rng() - (1u << 31));              // anything
                if (kind == 2) return s % 3 == 1 ? most - below(5) : below(most + 1);
                return (int)((long long)most * s / S) - (below(20) ? 0 : below(most + 1));   // in order, but for some
            };
            q[s] = value(c.Tq);
            k[s] = value(c.Tk);
        }
        const std::vector<int> back = taken(q, c.Tq, false);
        for (int b = 0; b < 50; ++b) {
            const int at = group_of(back.data(), S, b);
            if (at >= S || (at >= 0 && (back[at] > b || back[at + 1] <= b))) wrong("sequence %d in group %d", b, at);
        }
        c.cq = taken(q, c.Tq);
        c.ck = taken(k, c.Tk, false);
        check_all(c, it % 5 ? 1 + below(152) : 152, true);
    }
    return cases;
}

}  // namespace

int main(int argc, char **argv) { printf("ok %d\n", argc > 1 ? any_offsets(400) : ascending(1500)); }
