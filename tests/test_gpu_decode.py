"""Decoding from a paged key/value cache: the three operators against the float64 oracle, their
edges (empty and ragged sequences, pages that end inside a tile, stale NaN behind a sequence, bad
pages, slots and lengths, ties), graphs and streams, and a run of them together.

Tolerances.  A bf16 output is rounded once: half a step, 2^-8 of the value, plus the fp32 noise
of its terms.  Norm and rotation: the factors' relative error is below 2^-20, so the noise is at
most 2^-20 (|a| + |b|) for a rotated pair.  Attention: with S1 = max_i sum_e |q_e k_ie| / sqrt(d),
the fp32 score of d products is off by at most DELTA = 16 * 2^-24 * S1 (16 accumulation steps of
16 products, and the same again for the base-2 exponent); a weight p is off by a factor of at
most 1 + 2 DELTA + 2^-16 (2^-16: p carried to the value product as two halves of 8 bits each), hence
o by that times A = sum_i p_i |v_i|, and an accumulated weight by that times sum_h p_h plus fp32
roundings (2^-22).  An e4m3 value is off by half a step: 2^-4 of the value, 2^-10 at least.
"""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import qwen3_vl_text_gb300 as Q  # noqa: E402

BF16, E4M3 = "bf16", "e4m3"


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, device="cuda", generator=g)).to(torch.bfloat16)


def _pool(g, pages, nkv, page, d, dtype, apart=0):
    """K and V pools of NaN (nothing may read a place that holds no token), in one allocation with
    `apart` unused elements behind each page's K and V; and their scales."""
    one = nkv * page * d
    both = torch.full((pages, 2, one + apart), float("nan"), device="cuda", dtype=torch.bfloat16)
    scales = (None, None)
    if dtype == E4M3:
        both = both.to(torch.float8_e4m3fn)
        scales = tuple(0.01 + 0.02 * torch.rand(nkv, device="cuda", generator=g) for _ in range(2))
    k, v = (both[:, i, :one].unflatten(1, (nkv, page, d)) for i in range(2))
    return Q.KVCache(k, v, *scales)


def _raw(pool):
    return pool.view(torch.uint8) if pool.element_size() == 1 else pool.view(torch.int16)


def _fill(cache, table, lens, k, v):
    """Stores k, v [n][L, nkv, d] (float) through torch; returns the values the cache stands for."""
    kp, vp, ks, vs = cache.tensors
    page, out = cache.page_size, []
    for b, n in enumerate(lens):
        got = []
        for pool, x, sc in ((kp, k[b], ks), (vp, v[b], vs)):
            x = x[:n].float()
            x = x.to(torch.bfloat16) if sc is None else (x / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            i = torch.arange(n, device="cuda")
            _raw(pool)[table[b, i // page].long(), :, i % page] = _raw(x)
            got.append(_f64(x) * (1.0 if sc is None else _f64(sc)[:, None]))
        out.append(got)
    return out


def _table(g, n, cols, pages, spare=0):
    """Distinct random pages; -1 in the spare columns."""
    ids = torch.randperm(pages, device="cuda", generator=g)[:n * cols].to(torch.int32).view(n, cols)
    return torch.cat([ids, ids.new_full((n, spare), -1)], 1).contiguous()


# ---------------------------------------------------------------- norm, rotation, filling the cache

def _tables(T, d, g, grouped):
    ang = torch.rand(T, d // 2, device="cuda", generator=g) * 6.3
    cos, sin = ang.cos(), ang.sin()
    if not grouped:
        return cos, sin, cos, sin, 0
    S = (T + 31) // 32 * 32
    packed = [torch.nn.functional.pad(t, (0, 0, 0, S - T)).view(S, d // 8, 4).transpose(0, 1).contiguous()
              for t in (cos, sin)]
    return cos, sin, packed[0], packed[1], S


def _check_bf16(got, want, noise):
    bad = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + noise
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, worst {np.abs(got - want)[bad].max()}"


@pytest.mark.parametrize("T,nq,nkv,d,dtype,page,grouped,norm,rope", [
    (1, 64, 8, 128, BF16, 64, False, True, True), (1, 4, 2, 64, E4M3, 16, True, True, True),
    (37, 64, 8, 128, E4M3, 32, True, True, True), (130, 5, 5, 64, BF16, 256, False, True, True),
    (700, 24, 8, 128, BF16, 128, True, True, True), (3, 7, 1, 128, BF16, 16, False, True, False),
    (33, 3, 3, 64, E4M3, 64, False, False, True), (65, 2, 1, 128, BF16, 16, False, False, False),
    (2000, 1, 1, 64, BF16, 32, False, True, True), (311, 16, 16, 128, E4M3, 16, True, True, True)])
def test_qk_norm_rope_and_cache(T, nq, nkv, d, dtype, page, grouped, norm, rope):
    g = _gen(T * 7 + nq)
    W = (nq + 2 * nkv) * d
    buf = _randn(g, T, W + 24, scale=3.0)
    if T > 2:
        buf[2] = 0                                           # a row of zeros: the norm's eps
    qkv = buf[:, 8:8 + W]
    wq, wk = ((1 + 0.2 * torch.randn(2, d, device="cuda", generator=g)).to(torch.bfloat16)).unbind(0)
    cos, sin, pc, ps, stride = _tables(T, d, g, grouped)
    pages = (T + page - 1) // page + 2
    cache = _pool(g, pages, nkv, page, d, dtype, apart=32)
    before = [_raw(t).clone() for t in cache.tensors[:2]]
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:T].to(torch.int32)
    if T > 4:
        slots[1::5] = -1 - slots[1::5]                       # padding rows
    q_out = torch.full((T + 1, nq * d + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    k_out = torch.full((T + 1, nkv * d), 7.0, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (T, nq, nkv, d, wq if norm else None, wk if norm else None, 1e-6, pc if rope else None,
            ps if rope else None, stride if rope else 0)
    Q.h3enc_op_qk_norm_rope(qkv, *args, q_out, k_out, cache=cache, slots=slots, status=status)
    assert int(status.item()) == 0
    x = _f64(qkv).reshape(T, nq + 2 * nkv, d)
    c64, s64 = (_f64(cos), _f64(sin)) if rope else (None, None)
    want_q = O.decode.head_norm_rope(x[:, :nq], _f64(wq) if norm else None, 1e-6, c64, s64)
    want_k = O.decode.head_norm_rope(x[:, nq:nq + nkv], _f64(wk) if norm else None, 1e-6, c64, s64)

    def noise(y):      # 2^-20 of both elements of the pair, through the rotation |a| + |b| <= sqrt(2) |(a, b)|
        r = np.sqrt(y ** 2 + np.roll(y, d // 2, axis=-1) ** 2)
        return 2.0 ** -19 * r

    _check_bf16(_f64(q_out[:T, :nq * d]).reshape(want_q.shape), want_q, noise(want_q))
    _check_bf16(_f64(k_out[:T]).reshape(want_k.shape), want_k, noise(want_k))
    assert (q_out[T:] == 7).all() and (q_out[:, nq * d:] == 7).all() and (k_out[T:] == 7).all()

    # the cache: exactly the rows with a slot, everything else as it was
    live = slots >= 0
    pg, at = slots[live].long() // page, slots[live].long() % page
    rows = live.cpu().numpy()
    for pool, old, want, sc in ((cache.tensors[0], before[0], want_k, cache.tensors[2]),
                                (cache.tensors[1], before[1], x[:, nq + nkv:], cache.tensors[3])):
        got = _raw(pool)[pg, :, at].view(pool.dtype)
        if sc is None:
            _check_bf16(_f64(got), want[rows], noise(want[rows]))
        else:
            y = np.clip(want[rows] / _f64(sc)[:, None], -448, 448)
            assert (np.abs(_f64(got) - y) <= 2.0 ** -4 * np.abs(y) * (1 + 2.0 ** -15) + 2.0 ** -10).all()
        rest = _raw(pool).clone()
        rest[pg, :, at] = old[pg, :, at]
        assert torch.equal(rest, old)
    if dtype == E4M3:      # V has no arithmetic but the division: the bytes are the oracle's
        y = (_f64(qkv).reshape(T, -1, d)[rows][:, nq + nkv:].astype(np.float32)
             / cache.tensors[3].cpu().numpy()[:, None])
        assert np.array_equal(_f64(_raw(cache.tensors[1])[pg, :, at].view(torch.float8_e4m3fn)), O.fp8.e4m3_round(y))

    # in place, on another stream and without a cache: the same bits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Q.h3enc_op_qk_norm_rope(qkv, *args, qkv[:, :nq * d], qkv[:, nq * d:(nq + nkv) * d])
    side.synchronize()
    assert torch.equal(qkv[:, :nq * d], q_out[:T, :nq * d]) and torch.equal(qkv[:, nq * d:(nq + nkv) * d], k_out[:T])
    assert torch.equal(qkv[:, (nq + nkv) * d:].float(), torch.from_numpy(x[:, nq + nkv:].reshape(T, -1)).cuda().float())


def test_qk_norm_rope_slot_past_the_cache_is_reported_and_not_stored():
    g = _gen(5)
    cache = _pool(g, 3, 2, 16, 64, BF16)
    qkv = _randn(g, 4, 8 * 64)
    slots = torch.tensor([47, 48, 2 ** 31 - 1, 0], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Q.h3enc_op_qk_norm_rope(qkv, 4, 4, 2, 64, None, None, 0.0, None, None, cache=cache, slots=slots, status=status)
    assert int(status.item()) == 2
    k = cache.tensors[0]
    assert torch.equal(k[2, :, 15], qkv[0, 256:384].view(2, 64)) and torch.equal(k[0, :, 0], qkv[3, 256:384].view(2, 64))
    assert int(torch.isnan(k).sum()) == k.numel() - 2 * 128


def test_qk_norm_rope_matches_the_fused_projection():
    """A plain projection followed by the operator gives what the projection's own epilogue gives:
    both norm and rotate in fp32 and round once, the operator from the bf16 projection (2^-8 of
    every element of the vector before the norm, so 2^-8 of the output vector's norm, and each
    side's own rounding)."""
    g = _gen(6)
    M, K, nq, nkv, d = 70, 256, 4, 2, 128
    A, Wt = _randn(g, M, K), _randn(g, (nq + 2 * nkv) * d, K, scale=0.1)
    w = (1 + 0.1 * torch.randn(2, d, device="cuda", generator=g)).to(torch.bfloat16)
    cos, sin, _, _, _ = _tables(M, d, g, False)
    fused, plain = (torch.empty(M, (nq + 2 * nkv) * d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    Q.h3enc_op_gemm_qkv_rope(A, Wt, fused, M, K, nq, nkv, d, w[0], w[1], 1e-6, cos, sin)
    Q.h3enc_op_gemm(A, Wt, plain, M, (nq + 2 * nkv) * d, K, Q.EPI_STORE)
    Q.h3enc_op_qk_norm_rope(plain, M, nq, nkv, d, w[0], w[1], 1e-6, cos, sin, 0, plain[:, :nq * d],
                            plain[:, nq * d:(nq + nkv) * d])
    a, b = (_f64(t).reshape(M, -1, d) for t in (plain, fused))
    assert (np.linalg.norm(a - b, axis=-1) <= 3 * 2.0 ** -8 * np.linalg.norm(b, axis=-1)).all()
    assert np.array_equal(a[:, nq + nkv:], b[:, nq + nkv:])


# ---------------------------------------------------------------- attention of one token

def _attend_case(g, lens, nq, nkv, d, dtype, page, gain=1.0, apart=0, spare=1):
    n, cols = len(lens), max(1, -(-max(lens) // page))
    pages = n * cols + 3
    cache = _pool(g, pages, nkv, page, d, dtype, apart)
    table = _table(g, n, cols, pages, spare)
    for b, L in enumerate(lens):                              # columns behind the last page are no pages
        table[b, -(-L // page):] = -1
    k = [_randn(g, L, nkv, d, scale=gain) for L in lens]
    v = [_randn(g, L, nkv, d) for L in lens]
    kv = _fill(cache, table, lens, k, v)
    q = _randn(g, n, nq * d + 16, scale=gain)[:, 8:8 + nq * d]
    return cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), q, kv


def _workspace(n, nq, max_len, weights=False):
    return torch.zeros(Q.h3enc_op_attention_decode_workspace_bytes(n, nq, max_len, weights), dtype=torch.uint8,
                       device="cuda")


def _check_attention(o, q, kv, lens, nq, d, w_in=None, w_out=None):
    for b, L in enumerate(lens):
        qb, (k, v) = _f64(q[b]).reshape(nq, d), kv[b]
        want, p = O.decode.attend_one(qb, k, v)
        got = _f64(o[b]).reshape(nq, d)
        if L == 0:
            assert not got.any()
            continue
        rep = nq // k.shape[1]
        s1 = np.stack([np.abs(k[:, h // rep]) @ np.abs(qb[h]) for h in range(nq)]).max(1) / d ** 0.5
        rel = 2 * 2.0 ** -20 * s1 + 2.0 ** -16
        A = np.stack([p[h] @ np.abs(v[:, h // rep]) for h in range(nq)])
        bad = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + rel[:, None] * A
        assert not bad.any(), f"sequence {b} (length {L}): {int(bad.sum())} off by up to {np.abs(got - want)[bad].max()}"
        if w_out is not None:
            base = 0.0 if w_in is None else _f64(w_in[b, :L])
            assert (np.abs(w_out[b, :L].double().cpu().numpy() - base - p.sum(0))
                    <= (rel + 2.0 ** -20) @ p + 2.0 ** -22 * (base + p.sum(0))).all(), f"weights of sequence {b}"


CASES = [
    ([1], 64, 8, 128, BF16, 64), ([1], 4, 2, 64, E4M3, 16), ([0], 8, 8, 64, BF16, 16),
    ([1025], 64, 8, 128, BF16, 64), ([63, 64, 65, 0, 127, 129, 1], 16, 2, 128, BF16, 32),
    ([15, 16, 17, 33, 250, 0, 0], 4, 2, 64, BF16, 16), ([700, 3, 511], 16, 16, 64, E4M3, 128),
    ([300, 999, 64], 64, 8, 128, E4M3, 16), ([513, 77], 32, 1, 64, BF16, 256), ([200, 1000], 48, 2, 128, BF16, 64),
    ([345, 12], 40, 1, 128, E4M3, 32), ([20000], 8, 1, 128, BF16, 128), ([9001], 12, 4, 64, E4M3, 64),
    ([9000, 30000], 12, 1, 64, BF16, 32), ([40000], 16, 1, 128, BF16, 64), ([30000, 5], 24, 2, 128, E4M3, 16),
    ([110000], 40, 2, 128, BF16, 64), ([205000, 33], 76, 4, 64, E4M3, 256),       # segments of 32 heads (over 100 MB)
    ([700, 65], 64, 1, 128, BF16, 16), ([30000], 40, 2, 128, E4M3, 64), ([129, 20000], 20, 1, 64, E4M3, 32),
    ([5000, 1, 0, 3333], 28, 4, 128, BF16, 256), ([31] * 200, 2, 1, 64, BF16, 16), ([130] * 70 + [0] * 9, 8, 4, 128, BF16, 64),
]


@pytest.mark.parametrize("lens,nq,nkv,d,dtype,page", CASES)
@pytest.mark.parametrize("weights", [False, True])
def test_attention_decode(lens, nq, nkv, d, dtype, page, weights):
    g = _gen(sum(lens) + nq)
    cache, table, seq, q, kv = _attend_case(g, lens, nq, nkv, d, dtype, page, gain=1.5, apart=16)
    n, bound = len(lens), max(lens) + 5 if max(lens) % page else max(lens)
    bound = min(bound, table.shape[1] * page)
    o = torch.full((n + 1, nq * d + 8), 5.0, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = _workspace(n, nq, bound, weights)
    w_in = w_out = None
    if weights:
        w_in = torch.rand(n, bound + 3, device="cuda", generator=g)
        w_out = torch.full_like(w_in, -3.0)
    Q.h3enc_op_attention_decode(q, o[:n], cache, table, seq, nq, bound, ws, w_in, w_out, status=status)
    assert int(status.item()) == 0
    assert (o[n:] == 5).all() and (o[:, nq * d:] == 5).all()
    _check_attention(o[:n, :nq * d], q, kv, lens, nq, d, w_in, w_out)
    if weights:
        for b, L in enumerate(lens):
            assert (w_out[b, L:] == -3).all()
        again = w_in.clone()                                  # accumulated in place: the same bits
        Q.h3enc_op_attention_decode(q, o[:n], cache, table, seq, nq, bound, ws, again, again)
        for b, L in enumerate(lens):
            assert torch.equal(again[b, :L], w_out[b, :L]) and torch.equal(again[b, L:], w_in[b, L:])
    first = o.clone()
    for _ in range(3):                                        # the same workspace, the same bits
        o.fill_(5.0)
        Q.h3enc_op_attention_decode(q, o[:n], cache, table, seq, nq, bound, ws, w_in, w_out)
        assert torch.equal(o, first)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_attention_decode_of_large_and_small_scores(dtype):
    """Scores of up to several thousand (one key takes all) and queries of 1e-20 and 1e30."""
    lens, nq, nkv, d = [700, 150], 16, 2, 128
    g = _gen(9)
    cache, table, seq, q, kv = _attend_case(g, lens, nq, nkv, d, dtype, 64)
    for gain in (300.0, 1e-20, 2.0 ** 100):
        x = (q.float() * gain).to(torch.bfloat16)
        if gain > 1e6:
            x[:, d:] = 0                                      # one huge head; its ties are decided far from rounding
        o = torch.empty(2, nq * d, device="cuda", dtype=torch.bfloat16)
        Q.h3enc_op_attention_decode(x, o, cache, table, seq, nq, 700, _workspace(2, nq, 700))
        assert torch.isfinite(o).all()
        if gain > 1e6:
            for b in range(2):
                s = kv[b][0][:, 0] @ _f64(x[b])[:d]
                top = np.argsort(s)[-1]
                assert np.sort(s)[-1] - np.sort(s)[-2] > 1e6
                _check_bf16(_f64(o[b])[:d], kv[b][1][top, 0], 0.0)
        else:
            _check_attention(o, x, kv, lens, nq, d)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("n,L,nq,nkv,d,bound", [
    (32, 1000, 64, 8, 128, 1000), (20, 8192, 16, 2, 128, 8192), (30, 1500, 4, 2, 64, 1500), (20, 3000, 24, 2, 64, 3000),
    (60, 1111, 40, 2, 128, 16384)])                            # the last: segments of 32 heads (by the bound)
def test_attention_decode_of_a_sink_and_a_long_light_tail(n, L, nq, nkv, d, bound, dtype):
    """One key of score 16 to 22 above all others and of value zero: the output is the sum of the many
    light keys, every one of them far below 2^-20 of the largest weight.  Many segments, so that a
    warp holds the sink together with a long part of the tail."""
    g, page = _gen(n + L), 64
    lens = [L - i for i in range(n)]
    cache, table, seq, q, _ = _attend_case(g, lens, nq, nkv, d, dtype, page, spare=1 + (bound - L) // page)
    q = q.clone()
    q.view(n, nq, d)[..., 0] = 64.0
    k = [_randn(g, x, nkv, d) for x in lens]
    v = [1 + _randn(g, x, nkv, d) for x in lens]               # a mean, so that a lost share shows
    for b in range(n):
        at = (37 * b) % lens[b]
        k[b][..., 0] = 0
        k[b][at] = 0
        k[b][at, :, 0] = (16 + b % 7) * d ** 0.5 / 64.0
        v[b][at] = 0
    kv = _fill(cache, table, lens, k, v)
    o = torch.empty(n, nq * d, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(n, bound, device="cuda")
    Q.h3enc_op_attention_decode(q, o, cache, table, seq, nq, bound, _workspace(n, nq, bound, True), None, w)
    _check_attention(o, q, kv, lens, nq, d, None, w)


@pytest.mark.parametrize("nq,nkv,d,lens,bound", [
    (8, 2, 128, [300, 1, 64], 300), (6, 3, 64, [77, 2000], 2000), (24, 2, 128, [300, 1, 64], 300), (16, 1, 64, [77, 2000], 2000),
    (40, 1, 128, [300, 1, 200], 400000), (24, 1, 64, [5000, 17], 400000)])       # the last two: segments of 32 heads
def test_attention_decode_of_infinite_values(nq, nkv, d, lens, bound):
    """Infinite values of positive weight give an infinite output, of both signs or NaN among them NaN, and leave the
    other elements alone; a key of score minus infinity counts for nothing."""
    g, n, page = _gen(nq + d), len(lens), 64
    cache, table, seq, q, _ = _attend_case(g, lens, nq, nkv, d, BF16, page, spare=bound // page + 1)
    q = q.clone()
    q.view(n, nq, d)[..., 0] = q.view(n, nq, d)[..., 0].abs() + 0.5
    k, v = [_randn(g, L, nkv, d) for L in lens], [_randn(g, L, nkv, d) for L in lens]
    inf = float("inf")
    for b, L in enumerate(lens):
        v[b][0, :, 1] = inf
        v[b][L - 1, :, 2] = -inf
        v[b][L // 2, :, 3] = float("nan")
        if L > 1:
            v[b][L // 3, :, 4] = v[b][L - 1, :, 4] = inf
            v[b][0, :, 5], v[b][L - 1, :, 5] = inf, -inf
            k[b][L // 2 + 1 if L > 20 else 0, :, 0] = -inf
            if L <= 20:
                v[b][0, :, 1] = v[b][0, :, 5] = 0.5            # (0 * inf)
    kv = _fill(cache, table, lens, k, v)
    o = torch.empty(n, nq * d, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(n, bound, device="cuda")
    Q.h3enc_op_attention_decode(q, o, cache, table, seq, nq, bound, _workspace(n, nq, bound, True), None, w)
    for b, L in enumerate(lens):
        got, qb = _f64(o[b]).reshape(nq, d), _f64(q[b]).reshape(nq, d)
        at = np.isfinite(kv[b][0]).all(axis=(1, 2))            # without the key of no weight: the same sums
        kb, vb = kv[b][0][at], kv[b][1][at]
        with np.errstate(invalid="ignore"):
            want = O.decode.attend_one(qb, kb, vb)[0]
        assert not np.isfinite(want[:, [1, 2, 3]]).all(axis=1).any()
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
        assert (np.sign(got) == np.sign(want))[np.isinf(want)].all()
        at0 = w[b, :L].cpu().numpy()[~at]
        assert (at0 == 0).all() and np.isfinite(w[b, :L].cpu().numpy()).all()
        cols = np.isfinite(vb).all(axis=(0, 1))                # (elements that are finite in every key)
        kz, vz, gz = kb, np.where(cols, vb, 0.0), torch.from_numpy(np.where(cols, got, 0.0).reshape(-1))
        _check_attention(gz[None], q[b:b + 1], [(kz, vz)], [len(kb)], nq, d)


def test_attention_decode_bad_pages_and_lengths_are_reported():
    lens, nq, nkv, d, page = [100, 64], 8, 2, 64, 16
    g = _gen(10)
    cache, table, seq, q, kv = _attend_case(g, lens, nq, nkv, d, BF16, page)
    ws, status = _workspace(2, nq, 112), torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.empty(2, nq * d, device="cuda", dtype=torch.bfloat16)
    for bad in (-1, cache.num_pages, 2 ** 31 - 1, -2 ** 31):  # a page of zeros
        t = table.clone()
        t[0, 2] = bad
        status.zero_()
        Q.h3enc_op_attention_decode(q, o, cache, t, seq, nq, 112, ws, status=status)
        assert int(status.item()) == 2
        zk, zv = (x.copy() for x in kv[0])
        zk[32:48] = 0
        zv[32:48] = 0
        _check_attention(o, q, [(zk, zv), kv[1]], lens, nq, d)
    status.zero_()                                            # lengths outside [0, max_len] are clamped
    Q.h3enc_op_attention_decode(q, o, cache, table, torch.tensor([101, -5], dtype=torch.int32, device="cuda"), nq, 100, ws,
                                status=status)
    assert int(status.item()) == 2
    _check_attention(o, q, [kv[0], (kv[1][0][:0], kv[1][1][:0])], [100, 0], nq, d)


def test_attention_decode_shares_pages_between_sequences():
    """Two sequences with a common prefix (the same pages), and one page twice in one sequence."""
    nq, nkv, d, page = 8, 2, 128, 32
    g = _gen(11)
    cache, table, _, q, kv = _attend_case(g, [128, 128, 128], nq, nkv, d, BF16, page)
    table[1, :2] = table[0, :2]
    table[2, 3] = table[2, 0]
    k, v = ([kv[b][i].copy() for b in range(3)] for i in range(2))
    for x in (k, v):
        x[1][:64] = x[0][:64]
        x[2][96:] = x[2][:32]
    lens = [128, 100, 120]
    o = torch.empty(3, nq * d, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(3, 128, device="cuda")
    Q.h3enc_op_attention_decode(q, o, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), nq, 128,
                                _workspace(3, nq, 128, True), None, w)
    _check_attention(o, q, [(k[b][:L], v[b][:L]) for b, L in enumerate(lens)], lens, nq, d, None, w)


def test_attention_decode_cache_beyond_32_bit_offsets():
    """Pages more than 2^31 elements into the pool (4.3 GB of K)."""
    nq, nkv, d, page = 8, 1, 128, 16
    g = _gen(12)
    pages = 2 ** 31 // (page * d) + 40
    k, v = (torch.zeros(pages, nkv, page, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cache = Q.KVCache(k, v)
    table = torch.tensor([[pages - 1, 3, pages - 30, pages - 7]], dtype=torch.int32, device="cuda")
    kv = _fill(cache, table, [60], [_randn(g, 60, nkv, d)], [_randn(g, 60, nkv, d)])
    q = _randn(g, 1, nq * d)
    o, seq = torch.empty_like(q), torch.tensor([60], dtype=torch.int32, device="cuda")
    Q.h3enc_op_attention_decode(q, o, cache, table, seq, nq, 64, _workspace(1, nq, 64))
    _check_attention(o, q, kv, [60], nq, d)
    qkv = _randn(g, 1, (nq + 2) * d)
    slot = torch.tensor([(pages - 2) * page + 5], dtype=torch.int32, device="cuda")
    Q.h3enc_op_qk_norm_rope(qkv, 1, nq, 1, d, None, None, 0.0, None, None, cache=cache, slots=slot)
    assert torch.equal(k[pages - 2, 0, 5], qkv[0, nq * d:(nq + 1) * d])
    w = torch.rand(1, 64, device="cuda", generator=g)
    kept, new = torch.empty(1, 20, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    out = torch.tensor([[pages - 20, pages - 21]], dtype=torch.int32, device="cuda")
    Q.h3enc_op_cache_evict(cache, table, seq, 64, 20, w, torch.empty_like(w), kept, new, page_table_out=out)
    i = kept[0].long()
    assert torch.equal(k[out[0, torch.arange(20, device="cuda") // page].long(), 0, torch.arange(20, device="cuda") % page],
                       k[table[0, i // page].long(), 0, i % page])


def test_attention_decode_in_a_graph_reads_lengths_and_pages_anew():
    """One captured call (weights accumulated in place) replayed while the lengths, pages, queries
    and cache change underneath, against eager calls on a second workspace."""
    nq, nkv, d, page, n = 16, 2, 64, 16, 5
    g = _gen(13)
    cases = [_attend_case(_gen(100 + i), lens, nq, nkv, d, BF16, page) for i, lens in
             enumerate(([400, 0, 17, 64, 399], [5, 400, 1, 0, 300], [0, 0, 0, 0, 1], [400] * 5))]
    cache, table, seq, q, _ = _attend_case(g, [400] * n, nq, nkv, d, BF16, page)
    q = q.contiguous()
    o, w = torch.empty_like(q), torch.zeros(n, 400, device="cuda")
    ws = _workspace(n, nq, 400, True)

    def call(wspace, cache, table, seq, q, o, w):
        Q.h3enc_op_attention_decode(q, o, cache, table, seq, nq, 400, wspace, w, w)

    call(ws, cache, table, seq, q, o, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws, cache, table, seq, q, o, w)
    ws2 = _workspace(n, nq, 400, True)
    for c2, t2, s2, q2, kv2 in cases + cases[:2]:
        t2 = torch.nn.functional.pad(t2, (0, table.shape[1] - t2.shape[1]), value=-1)
        start = torch.rand(n, 400, device="cuda", generator=g)
        want_o, want_w = torch.empty_like(o), start.clone()
        call(ws2, c2, t2, s2, q2, want_o, want_w)
        for dst, src in zip(cache.tensors[:2], c2.tensors[:2]):
            dst.zero_()
            dst[:src.shape[0]] = src[:dst.shape[0]]
        table.copy_(t2)
        seq.copy_(s2)
        q.copy_(q2)
        w.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o) and torch.equal(w, want_w)


def test_attention_decode_calls_of_other_sizes_share_a_workspace():
    g = _gen(14)
    a = _attend_case(g, [700, 1, 300], 32, 4, 128, BF16, 64)
    b = _attend_case(g, [90] * 40, 4, 2, 64, E4M3, 16)
    ws = _workspace(40, 32, 700, True)
    for _ in range(3):
        for (cache, table, seq, q, kv), nq, bound, weights in ((a, 32, 700, True), (b, 4, 96, False), (b, 4, 96, True),
                                                               (a, 32, 700, False)):
            n, d = len(kv), cache.head_dim
            o = torch.empty(n, nq * d, device="cuda", dtype=torch.bfloat16)
            w = torch.zeros(n, bound, device="cuda") if weights else None
            Q.h3enc_op_attention_decode(q, o, cache, table, seq, nq, bound, ws, None, w)
            _check_attention(o, q, kv, seq.tolist(), nq, d, None, w)


def test_attention_decode_on_two_streams_at_once():
    """Calls on two streams, each with its own workspace and outputs, against the same calls alone."""
    cases = [_attend_case(_gen(40 + i), [3000, 17, 900], 16, 2, 128, BF16, 64) for i in range(2)]
    spaces = [_workspace(3, 16, 3000, True) for _ in cases]
    outs = [(torch.empty(3, 16 * 128, device="cuda", dtype=torch.bfloat16), torch.zeros(3, 3000, device="cuda")) for _ in cases]

    def call(i, o, w):
        cache, table, seq, q, _ = cases[i]
        Q.h3enc_op_attention_decode(q, o, cache, table, seq, 16, 3000, spaces[i], None, w)

    alone = []
    for i in range(2):
        call(i, *outs[i])
        alone.append([t.clone() for t in outs[i]])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                for t in outs[i]:
                    t.zero_()
                call(i, *outs[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], alone[i]))


def test_attention_decode_refuses_a_small_or_misaligned_workspace():
    cache, table, seq, q, _ = _attend_case(_gen(15), [50], 8, 2, 64, BF16, 16)
    o = torch.empty(1, 8 * 64, device="cuda", dtype=torch.bfloat16)
    ws = _workspace(1, 8, 50)
    for bad in (None, ws[:-1], torch.zeros(ws.numel() + 256, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(Q.H3encError) as e:
            Q.h3enc_op_attention_decode(q, o, cache, table, seq, 8, 50, bad)
        assert e.value.code == 2


def test_attention_decode_workspace_of_sizes_that_the_call_refuses():
    size = Q.h3enc_op_attention_decode_workspace_bytes
    assert 0 < size(1, 8, 2 ** 30) < 2 ** 30 and size(1, 1, 2 ** 30, True) >= 4 * 2 ** 30
    for weights in (False, True):
        for max_len in (2 ** 30 + 1, 2 ** 31 - 127, 2 ** 31 - 1):
            assert size(1, 1, max_len, weights) == -1


def test_attention_decode_counts_its_tiles_in_32_bits():
    """2^31 - 2 = 154 * 13,944,699 tiles of 64 keys: the look-ahead behind the last of them would overflow."""
    size = Q.h3enc_op_attention_decode_workspace_bytes
    assert size(1, 154, 13944699 * 64) == -1 and size(154, 1, 13944699 * 64 - 63) == -1
    assert size(1, 154, 13944698 * 64) > 0                    # 2^31 - 156
    cache, table, seq, q, _ = _attend_case(_gen(16), [50], 154, 154, 64, BF16, 16)
    wide = torch.full((1, 13944699 * 4), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    o = torch.empty(1, 154 * 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(Q.H3encError) as e:
        Q.h3enc_op_attention_decode(q, o, cache, wide, seq, 154, 13944699 * 64, _workspace(1, 154, 64))
    assert e.value.code == 6


# ---------------------------------------------------------------- eviction

def _weights(g, n, cols, kind):
    w = torch.empty(n, cols, device="cuda").exponential_(generator=g)
    if kind == "ties":
        w = torch.randint(0, 3, (n, cols), device="cuda", generator=g).float() * torch.where(
            torch.rand(n, cols, device="cuda", generator=g) < 0.5, 1.0, -1.0)      # -0 and 0 among them
    elif kind == "equal":
        w.fill_(0.25)
    elif kind == "odd":
        r = torch.rand(n, cols, device="cuda", generator=g)
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), -1.0, 1e-45, -float("nan"))):
            w[(r >= 0.1 * i) & (r < 0.1 * (i + 1))] = x
    return w


@pytest.mark.parametrize("lens,nkv,d,dtype,page,budget,sink,recent,kind", [
    ([40, 16, 17, 0, 1, 33], 2, 64, BF16, 16, 16, 2, 4, "spread"),
    ([300, 299, 64, 128, 257], 1, 128, E4M3, 32, 128, 0, 0, "ties"),
    ([1000, 5, 700], 8, 128, BF16, 64, 600, 4, 100, "spread"),
    ([500, 400], 2, 64, E4M3, 128, 64, 32, 32, "spread"),          # nothing left for the weights to decide
    ([2100, 2049, 2048], 1, 64, BF16, 256, 2048, 0, 1, "equal"),
    ([777], 3, 128, BF16, 16, 1, 0, 0, "odd"), ([1500, 1024], 2, 64, BF16, 64, 1023, 7, 0, "odd"),
    ([9000], 1, 128, BF16, 128, 4500, 16, 512, "ties"), ([33000], 1, 64, E4M3, 256, 8000, 4, 64, "spread"),
    ([70000, 100], 1, 64, E4M3, 256, 100, 1, 1, "odd"), ([400000, 270001], 1, 64, E4M3, 256, 150000, 9, 5000, "ties")])
@pytest.mark.parametrize("in_place", [True, False])
def test_cache_evict(lens, nkv, d, dtype, page, budget, sink, recent, kind, in_place):
    g = _gen(sum(lens) + budget)
    n, top = len(lens), max(lens) + 3
    cols, out_cols = -(-top // page), -(-budget // page)
    pages = n * (cols + out_cols) + 2
    cache = _pool(g, pages, nkv, page, d, dtype, apart=48)
    for t in cache.tensors[:2]:
        _raw(t).copy_(torch.randint(-100, 100, _raw(t).shape, device="cuda", generator=g).to(_raw(t).dtype))
    before = [_raw(t).clone() for t in cache.tensors[:2]]
    ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table, out = ids[:n * cols].view(n, cols), ids[n * cols:n * (cols + out_cols)].view(n, out_cols)
    w = _weights(g, n, top + 5, kind)
    w_out = torch.full((n, top + 2), -7.0, device="cuda")
    kept = torch.full((n, budget + 2), -9, dtype=torch.int32, device="cuda")
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new, status = seq.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    Q.h3enc_op_cache_evict(cache, table, new, top, budget, w, w_out, kept, new,      # lengths updated in place
                           page_table_out=None if in_place else out, sink=sink, recent=recent, status=status)
    assert int(status.item()) == 0
    want = [b.clone() for b in before]
    wc = w.cpu().numpy()
    to = table if in_place else out
    for b, L in enumerate(lens):
        keep = O.decode.keep_heaviest(wc[b], L, budget, sink, recent)
        m = len(keep)
        assert int(new[b]) == m == min(L, budget)
        assert kept[b].tolist() == keep + [-1] * (budget - m) + [-9] * 2
        i = torch.tensor(keep, dtype=torch.long, device="cuda")
        assert torch.equal(w_out[b, :m].view(torch.int32), w[b, i].view(torch.int32))
        assert not w_out[b, m:top].any() and (w_out[b, top:] == -7).all()
        j = torch.arange(m, device="cuda")
        for pool, old in zip(want, before):
            pool[to[b, j // page].long(), :, j % page] = old[table[b, i // page].long(), :, i % page]
    for pool, x in zip(cache.tensors[:2], want):
        assert torch.equal(_raw(pool), x)


@pytest.mark.parametrize("n,nkv,d,dtype,budget", [
    (20, 8, 128, BF16, 900), (12, 8, 128, BF16, 1500), (12, 4, 128, BF16, 2900), (3, 1, 128, BF16, 5300),   # 128 to 1024 rows a chunk
    (20, 8, 128, E4M3, 1500), (12, 8, 128, E4M3, 2900), (2, 2, 128, E4M3, 5300), (40, 4, 64, E4M3, 2900), (40, 4, 64, BF16, 1500)])
def test_cache_evict_in_place_in_many_chunks(n, nkv, d, dtype, budget):
    """At least five chunks of rows per CTA, at every width of a slice, while another stream copies memory: the
    whole pool, from the same start, the same every time."""
    g, page = _gen(n * d + budget), 64
    top = budget + budget // 3
    lens = [top - 11 * i for i in range(n)]
    cols = -(-top // page)
    cache = _pool(g, n * cols, nkv, page, d, dtype)
    start = [torch.randint(-100, 100, _raw(t).shape, device="cuda", generator=g).to(_raw(t).dtype) for t in cache.tensors[:2]]
    table = _table(g, n, cols, n * cols)
    w = _weights(g, n, top, "spread")
    want, wc = [t.clone() for t in start], w.cpu().numpy()
    for b, L in enumerate(lens):
        keep = O.decode.keep_heaviest(wc[b], L, budget, 4, 64)
        i, j = torch.tensor(keep, device="cuda"), torch.arange(len(keep), device="cuda")
        for to, old in zip(want, start):
            to[table[b, j // page].long(), :, j % page] = old[table[b, i // page].long(), :, i % page]
    seq, new = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    kept, w_out = torch.empty(n, budget, dtype=torch.int32, device="cuda"), torch.empty_like(w)
    a, side = torch.empty(1 << 28, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(100):
        with torch.cuda.stream(side):
            a[1 << 27:] = a[:1 << 27]
        for t, old in zip(cache.tensors[:2], start):
            _raw(t).copy_(old)
        Q.h3enc_op_cache_evict(cache, table, seq, top, budget, w, w_out, kept, new, sink=4, recent=64)
        for t, x in zip(cache.tensors[:2], want):
            assert torch.equal(_raw(t), x)
    torch.cuda.synchronize()


def test_cache_evict_bad_pages_and_lengths_are_reported():
    g = _gen(20)
    nkv, d, page = 2, 64, 16
    cache = _pool(g, 20, nkv, page, d, BF16)
    for t in cache.tensors[:2]:
        t.copy_(_randn(g, *t.shape))
    before = [t.clone() for t in cache.tensors[:2]]
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    out = torch.arange(8, 12, dtype=torch.int32, device="cuda").view(2, 2)
    table[0, 1], out[1, 1] = 20, -1
    w = torch.arange(128, device="cuda", dtype=torch.float32).view(2, 64)
    kept, new = torch.empty(2, 32, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = torch.tensor([48, 70], dtype=torch.int32, device="cuda")
    Q.h3enc_op_cache_evict(cache, table, seq, 64, 32, w, torch.empty_like(w), kept, new, page_table_out=out,
                           status=status)
    assert int(status.item()) == 2
    assert kept.tolist() == [list(range(16, 48)), list(range(32, 64))] and new.tolist() == [32, 32]
    for t, old in zip(cache.tensors[:2], before):
        want = old.clone()
        want[9] = old[2]                 # sequence 0: its second page is bad, the third moves
        want[10] = old[6]                # sequence 1: its second target is bad
        assert torch.equal(t, want)
    status.zero_()
    seq = torch.tensor([-3, 5], dtype=torch.int32, device="cuda")
    Q.h3enc_op_cache_evict(cache, table, seq, 64, 32, w, torch.empty_like(w), kept, new, page_table_out=out,
                           status=status)
    assert int(status.item()) == 2 and new.tolist() == [0, 5]


@pytest.mark.parametrize("top", [60, 5000])
def test_cache_evict_of_the_largest_budget(top):
    """A budget of 2^31 - 1: everything is kept, and -1 fills the row of 8.6 GB to its end and not further."""
    g, budget = _gen(22), 2 ** 31 - 1
    cache = _pool(g, -(-top // 16), 1, 16, 64, BF16)
    for t in cache.tensors[:2]:
        t.copy_(_randn(g, *t.shape))
    before = [t.clone() for t in cache.tensors[:2]]
    table = torch.arange(cache.num_pages, dtype=torch.int32, device="cuda")[None]
    w, w_out = torch.rand(1, top, device="cuda", generator=g), torch.empty(1, top, device="cuda")
    guard = 1 << 15
    buf = torch.full((guard + budget + guard,), -9, dtype=torch.int32, device="cuda")
    kept, new = buf[guard:guard + budget][None], torch.zeros(1, dtype=torch.int32, device="cuda")
    Q.h3enc_op_cache_evict(cache, table, torch.tensor([top - 7], dtype=torch.int32, device="cuda"), top, budget, w, w_out, kept, new)
    assert int(new) == top - 7 and kept[0, :top - 7].tolist() == list(range(top - 7))
    rest = kept[0, top - 7:]
    assert int(rest.min()) == -1 and int(rest.max()) == -1
    assert (buf[:guard] == -9).all() and (buf[guard + budget:] == -9).all()
    assert torch.equal(w_out[0, :top - 7], w[0, :top - 7]) and not w_out[0, top - 7:].any()
    assert all(torch.equal(t, x) for t, x in zip(cache.tensors[:2], before))


def test_decoding_of_sequences_without_any_token():
    """max_len = 0: no page table at all, zero rows from the attention, nothing kept by the eviction."""
    g = _gen(21)
    cache = _pool(g, 2, 2, 16, 64, BF16)
    seq, table = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    q, o = _randn(g, 3, 8 * 64), torch.full((3, 8 * 64), 9.0, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(3, 4, device="cuda")
    Q.h3enc_op_attention_decode(q, o, cache, table, seq, 8, 0, _workspace(3, 8, 0, True), None, w)
    assert not o.any()
    kept, new = torch.zeros(3, 5, dtype=torch.int32, device="cuda"), torch.full((3,), 7, dtype=torch.int32, device="cuda")
    Q.h3enc_op_cache_evict(cache, table, seq, 0, 5, w, torch.ones_like(w), kept, new)
    assert (kept == -1).all() and not new.any()


def test_cache_evict_of_rows_without_any_place():
    """max_len = 0 with weights and page tables of no columns (which have no address)."""
    cache, none = _pool(_gen(23), 2, 2, 16, 64, BF16), torch.zeros(2, 0, device="cuda")
    seq, kept = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    new, table = torch.full((2,), 7, dtype=torch.int32, device="cuda"), none.to(torch.int32)
    for out in (None, table):
        Q.h3enc_op_cache_evict(cache, table, seq, 0, 5, none, none.clone(), kept.zero_(), new.fill_(7), page_table_out=out)
        assert (kept == -1).all() and not new.any()


# ---------------------------------------------------------------- together

def test_decode_step_captured_in_a_graph():
    """One decode step (norm, rotation and store; attention with weights; eviction into other pages)
    captured once and replayed on other projections, slots, lengths and weights, against the eager calls."""
    g = _gen(31)
    n, nq, nkv, d, page, top, budget = 3, 16, 4, 64, 16, 200, 96
    cols, out_cols = -(-top // page), -(-budget // page)
    pages = n * (cols + out_cols)
    wq, wk = ((1 + 0.1 * torch.randn(2, d, device="cuda", generator=g)).to(torch.bfloat16)).unbind(0)
    ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table, out = ids[:n * cols].view(n, cols), ids[n * cols:].view(n, out_cols)
    ws = _workspace(n, nq, top, True)

    def fresh(seed):
        h = _gen(seed)
        lens = torch.randint(1, top, (n,), device="cuda", generator=h, dtype=torch.int32)
        at = (lens - 1).long()
        return dict(kv=_randn(h, 2, pages, nkv, page, d), qkv=_randn(h, n, (nq + 2 * nkv) * d), lens=lens,
                    slots=(table[torch.arange(n, device="cuda"), at // page] * page + at % page).to(torch.int32),
                    cos=torch.randn(n, d // 2, device="cuda", generator=h).cos(), sin=torch.zeros(n, d // 2, device="cuda"),
                    w=torch.rand(n, top, device="cuda", generator=h), w2=torch.zeros(n, top, device="cuda"),
                    o=torch.zeros(n, nq * d, device="cuda", dtype=torch.bfloat16), q=torch.zeros(n, nq * d, device="cuda",
                                                                                                dtype=torch.bfloat16),
                    kept=torch.zeros(n, budget, device="cuda", dtype=torch.int32),
                    new=torch.zeros(n, device="cuda", dtype=torch.int32))

    def step(s):
        cache = Q.KVCache(s["kv"][0], s["kv"][1])
        Q.h3enc_op_qk_norm_rope(s["qkv"], n, nq, nkv, d, wq, wk, 1e-6, s["cos"], s["sin"], 0, s["q"], cache=cache,
                                slots=s["slots"])
        Q.h3enc_op_attention_decode(s["q"], s["o"], cache, table, s["lens"], nq, top, ws, s["w"], s["w"])
        Q.h3enc_op_cache_evict(cache, table, s["lens"], top, budget, s["w"], s["w2"], s["kept"], s["new"],
                               page_table_out=out, sink=2, recent=20)

    static = fresh(0)
    step(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(static)
    for seed in (1, 2, 3):
        want, start = fresh(seed), fresh(seed)
        step(want)
        for name, t in start.items():
            static[name].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for name, t in want.items():
            assert torch.equal(static[name], t), name


@pytest.mark.parametrize("dtype,heads", [(BF16, (8, 2, 64)), (E4M3, (16, 2, 128))])
def test_prompt_then_decode_with_eviction(dtype, heads):
    """Two prompts fill the cache from a plain projection, then tokens are added one at a time,
    each step projecting, norming, storing, attending and accumulating weights; when a sequence
    passes the limit the caches are cut to the budget.  Every step is compared with the oracle on
    the values the cache stands for, and the attention of the prompt's last row with the prefill's."""
    nq, nkv, d = heads
    page, budget, limit, hidden = 16, 40, 56, 256
    g = _gen(30)
    Wt = _randn(g, (nq + 2 * nkv) * d, hidden, scale=0.08)
    wq, wk = ((1 + 0.1 * torch.randn(2, d, device="cuda", generator=g)).to(torch.bfloat16)).unbind(0)
    N = Wt.shape[0]
    cols = limit // page + 1
    cache = _pool(g, 2 * cols, nkv, page, d, dtype)
    table = _table(g, 2, cols, 2 * cols)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    max_len = cols * page
    weight, spare = torch.zeros(2, max_len, device="cuda"), torch.zeros(2, max_len, device="cuda")
    ws = _workspace(2, nq, max_len, True)
    mirror = [[np.zeros((0, nkv, d)), np.zeros((0, nkv, d))] for _ in range(2)]

    def project(x, pos, slots, in_place=False):
        T = x.shape[0]
        qkv = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
        Q.h3enc_op_gemm(x, Wt, qkv, T, N, hidden, Q.EPI_STORE)
        cos, sin = (torch.empty(T, d // 2, device="cuda") for _ in range(2))
        p3 = pos.to(torch.int32).expand(3, T).contiguous()
        Q.h3enc_op_rope_table(p3, T, d, 5e6, (24, 20, 20), cos, sin)
        raw = _f64(qkv).reshape(T, -1, d)
        Q.h3enc_op_qk_norm_rope(qkv, T, nq, nkv, d, wq, wk, 1e-6, cos, sin, 0, qkv[:, :nq * d],
                                qkv[:, nq * d:(nq + nkv) * d], cache=cache, slots=slots, status=status)
        c, s = _f64(cos), _f64(sin)
        k = O.decode.head_norm_rope(raw[:, nq:nq + nkv], _f64(wk), 1e-6, c, s)
        return qkv, k, raw[:, nq + nkv:]

    def stands_for(b, length):
        i = torch.arange(length, device="cuda")
        out = []
        for pool, sc in ((cache.tensors[0], cache.tensors[2]), (cache.tensors[1], cache.tensors[3])):
            x = _f64(_raw(pool)[table[b, i // page].long(), :, i % page].view(pool.dtype))
            out.append(x if sc is None else x * _f64(sc)[:, None])
        return out

    lens = [23, 50]
    for b in range(2):                     # prompts
        T = lens[b]
        i = torch.arange(T, device="cuda")
        qkv, k, v = project(_randn(g, T, hidden), i, (table[b, i // page] * page + i % page).to(torch.int32))
        mirror[b] = [k, v]
        o = torch.empty(T, nq * d, device="cuda", dtype=torch.bfloat16)
        Q.h3enc_op_attention(qkv, o, T, nq, nkv, d)
        if dtype == BF16:                  # the prefill's last row = one token over the cache
            one = torch.empty(1, nq * d, device="cuda", dtype=torch.bfloat16)
            Q.h3enc_op_attention_decode(qkv[T - 1:, :nq * d], one, cache, table[b:b + 1],
                                        torch.tensor([T], dtype=torch.int32, device="cuda"), nq, max_len, ws)
            a, r = _f64(one).reshape(nq, d), _f64(o[T - 1]).reshape(nq, d)
            assert (np.linalg.norm(a - r, axis=1) <= 1.5e-2 * np.linalg.norm(r, axis=1)).all()   # the prefill's own bound
    position = list(lens)
    for step in range(25):
        pos = torch.tensor(position, device="cuda")
        at = torch.tensor(lens, device="cuda")
        rows = torch.arange(2, device="cuda")
        qkv, k, v = project(_randn(g, 2, hidden), pos, (table[rows, at // page] * page + at % page).to(torch.int32))
        lens = [x + 1 for x in lens]
        position = [x + 1 for x in position]
        seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        o, before = torch.empty(2, nq * d, device="cuda", dtype=torch.bfloat16), weight.clone()
        Q.h3enc_op_attention_decode(qkv[:, :nq * d], o, cache, table, seq, nq, max_len, ws, weight, weight, status=status)
        now = [stands_for(b, lens[b]) for b in range(2)]
        _check_attention(o, qkv[:, :nq * d], now, lens, nq, d, before, weight)
        for b in range(2):                 # what the cache stands for follows the exact tokens
            for m, x, y in zip((0, 1), (k, v), now[b]):
                mirror[b][m] = np.concatenate([mirror[b][m], x[b:b + 1]])
                tol = 2.0 ** -4 if dtype == E4M3 else 2.0 ** -8
                assert (np.abs(y - mirror[b][m]) <= tol * np.abs(mirror[b][m]) * (1 + 2.0 ** -10) + 1e-4).all()
        if max(lens) == limit:
            kept, new = torch.empty(2, budget, dtype=torch.int32, device="cuda"), torch.empty_like(seq)
            Q.h3enc_op_cache_evict(cache, table, seq, max_len, budget, weight, spare, kept, new, sink=2, recent=8,
                                   status=status)
            for b in range(2):
                keep = O.decode.keep_heaviest(weight[b].cpu().numpy(), lens[b], budget, 2, 8)
                assert kept[b].tolist() == keep + [-1] * (budget - len(keep))
                mirror[b] = [x[keep] for x in mirror[b]]
            weight, spare = spare, weight
            lens = new.tolist()
    assert int(status.item()) == 0
