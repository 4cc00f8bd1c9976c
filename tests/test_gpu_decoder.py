"""A decoder that reads an encoder's states: rows rotated and appended to a paged cache, attention of one new token
behind shared prefixes, and cross attention, against the float64 oracle; their edges (empty and ragged
sequences, pages that end inside a tile, stale NaN behind a sequence, bad pages and lengths), graphs and streams, and
a run of them together.

Tolerances.  A bf16 output is rounded once: half a step, 2^-8 of the value, plus the fp32 noise of its terms.
Rotation: the angle is a 64-bit fraction of a turn, so cos and sin are off by less than 2^-21 of the magnitude (fp32
rounding of the fraction and of sincospi), and the norm's factor by 2^-21: at most 2^-19 of a pair's length.
An e4m3 value is off by half a step: 2^-4 of the value, 2^-10 at least.
Attention: with S1 = max_i sum_e |q_e k_ie| / sqrt(d), the fp32 score of d products is off by at most DELTA = 16 * 2^-24 * S1
(16 accumulation steps of 16 products, and the same again for the base-2 exponent), so a weight by a factor of at most
1 + 2 DELTA; it enters the value product in bf16, 2^-8 of it (f16 behind an e4m3 cache: 2^-11, and at least 2^-37
absolutely; a sequence's own tokens, few queries, near prefixes and those in bf16: two halves, 2^-16).  With A = sum_i p_i |v_i| the output is off by A times that, 2^-18 A for
fp32 sums and the joins, and half a step of bf16.  An accumulated weight is off by 2 DELTA + 2^-18 of sum_h p_h.
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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


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


def _table(g, n, cols, pages, spare=0):
    """Distinct random pages; -1 in the spare columns."""
    ids = torch.randperm(pages, device="cuda", generator=g)[:n * cols].to(torch.int32).view(n, cols)
    return torch.cat([ids, ids.new_full((n, spare), -1)], 1).contiguous()


def _check_bf16(got, want, noise):
    bad = ~(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + noise)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, worst {np.nanmax(np.abs(got - want)[bad])}"


# ---------------------------------------------------------------- rotated rows, appended

def _pair_length(y, rot, interleaved):
    """Per element the length of the pair that it rotates in (of the element alone behind rot)."""
    other = np.zeros_like(y)
    if interleaved:
        other[..., 0:rot:2], other[..., 1:rot:2] = y[..., 1:rot:2], y[..., 0:rot:2]
    else:
        other[..., :rot // 2], other[..., rot // 2:rot] = y[..., rot // 2:rot], y[..., :rot // 2]
    return np.hypot(y, other)


def _angles(places, positions, rope_args):
    section = rope_args.get("section")
    w, magnitude = O.decoder.frequencies(**{k: v for k, v in rope_args.items() if k not in ("section", "interleaved")})
    if positions is None:
        return np.asarray(places, np.float64)[:, None] * w, magnitude
    pos = positions.cpu().numpy().astype(np.float64)
    axes = [O.decoder.axis_of(j, section) if section else 0 for j in range(len(w))]
    return np.stack([pos[a] * wj for a, wj in zip(axes, w)], 1), magnitude


ROPES = {
    "whole": lambda d: dict(rot=d, theta=5e6), "pairs": lambda d: dict(rot=d, theta=1e4, interleaved=True),
    "half": lambda d: dict(rot=d // 2, theta=1e6), "few": lambda d: dict(rot=16, theta=100.0, interleaved=True),
    "three quarters": lambda d: dict(rot=3 * d // 4, theta=1e4),
    "linear": lambda d: dict(rot=d, theta=1e4, scaling="linear", factor=8.0),
    "wavelength": lambda d: dict(rot=d, theta=5e5, scaling="wavelength", factor=8.0, original_len=8192),
    "yarn": lambda d: dict(rot=d, theta=1e6, scaling="yarn", factor=4.0, original_len=32768),
    "yarn pairs": lambda d: dict(rot=d // 2, theta=1e4, scaling="yarn", factor=40.0, original_len=4096, low_turns=2.0,
                                 high_turns=20.0, magnitude=1.5, interleaved=True),
    "axes": lambda d: dict(rot=d, theta=5e6, section=(24, 20, 20) if d == 128 else (12, 10, 10))}


def _rope(name, d):
    a = ROPES[name](d)
    kw = {k: v for k, v in a.items() if k != "rot"}
    return a, Q.Rope(a["rot"], **kw)


@pytest.mark.parametrize("name,counts,held,nq,nkv,d,dtype,page,norm,pad", [
    ("whole", [1], [0], 64, 8, 128, BF16, 64, True, 0), ("yarn", [1], [1 << 20], 4, 2, 64, E4M3, 256, True, 0),
    ("pairs", [1] * 37, None, 64, 8, 128, E4M3, 32, True, 3), ("half", [5, 0, 1, 130], None, 5, 5, 64, BF16, 256, True, 2),
    ("few", [3, 17, 64], None, 40, 2, 128, BF16, 16, False, 0), ("axes", [77, 1, 311], None, 16, 4, 128, BF16, 128, True, 1),
    ("axes", [40], [9], 4, 2, 64, E4M3, 16, True, 5), ("linear", [700], [3], 28, 4, 128, BF16, 64, False, 0),
    ("wavelength", [200] * 3, [100000, 0, 70000], 12, 1, 64, BF16, 16, True, 0), ("yarn pairs", [9, 33], None, 7, 1, 128, BF16, 64, False, 4),
    ("three quarters", [65, 2], None, 3, 3, 64, E4M3, 64, True, 0), (None, [65], [15], 2, 1, 128, BF16, 16, True, 1),
    ("whole", [2000], [0], 1, 1, 64, BF16, 32, True, 0), ("yarn", [1, 0] * 300 + [4, 400], None, 4, 2, 64, BF16, 16, True, 1)])
def test_rope_append(name, counts, held, nq, nkv, d, dtype, page, norm, pad):
    g = _gen(sum(counts) * 7 + nq)
    n, live = len(counts), sum(counts)
    T, W = live + pad, (nq + 2 * nkv) * d
    if held is None:
        held = [(i * 37) % 101 for i in range(n)]
    lens = [h + c for h, c in zip(held, counts)]
    buf = _randn(g, T, W + 24, scale=3.0)
    if T > 2:
        buf[2] = 0                                           # a row of zeros: the norm's eps
    qkv = buf[:, 8:8 + W]
    wq, wk = ((1 + 0.2 * torch.randn(2, d, device="cuda", generator=g)).to(torch.bfloat16)).unbind(0)
    max_len = max(max(lens), 1)
    cols = -(-max_len // page)
    touched = [sorted({p // page for p in range(h, h + c)}) for h, c in zip(held, counts)]
    pages = sum(map(len, touched)) + 3
    table = torch.full((n, cols + 1), -1, dtype=torch.int32, device="cuda")
    ids = iter(torch.randperm(pages, device="cuda", generator=g).tolist())
    for b, cs in enumerate(touched):
        if cs:
            table[b, torch.tensor(cs, device="cuda")] = _i32([next(ids) for _ in cs])
    cache = _pool(g, pages, nkv, page, d, dtype, apart=32)
    before = [_raw(t).clone() for t in cache.tensors[:2]]
    args, rope = (dict(rot=16, theta=1.0), None) if name is None else _rope(name, d)
    positions = None
    if name == "axes":
        positions = torch.randint(-50, 100000, (3, T + 7), device="cuda", generator=g).to(torch.int32)[:, :T]
    single = all(c == 1 for c in counts)
    cu = None if single else _i32(np.concatenate([[0], np.cumsum(counts)]))
    q_out = torch.full((T + 1, nq * d + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    k_out = torch.full((T + 1, nkv * d), 7.0, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = dict(T=T, n_heads=nq, n_kv_heads=nkv, head_dim=d, w_q=wq if norm else None, w_k=wk if norm else None, eps=1e-6,
                rope=rope, positions=positions, seq_lens=_i32(lens), cu_rows=cu)
    Q.h3enc_op_rope_append(qkv, **call, q_out=q_out, k_out=k_out, cache=cache, page_table=table, max_len=max_len,
                           status=status)
    assert int(status.item()) == 0
    at = O.decoder.append_places(T, lens, None if single else np.concatenate([[0], np.cumsum(counts)]).tolist())
    assert at[live:] == [None] * pad and None not in at[:live]
    seq, place = (torch.tensor(v, device="cuda", dtype=torch.long) for v in zip(*at[:live]))
    angle, magnitude = _angles([p for _, p in at[:live]], positions[:, :live] if positions is not None else None, args)
    if name is None:
        angle = angle * 0
    x = _f64(qkv).reshape(T, nq + 2 * nkv, d)[:live]
    inter = args.get("interleaved", False)

    def want(heads, w):
        return O.decoder.rotate(O.decode.head_norm_rope(heads, _f64(w) if norm else None, 1e-6, None, None), angle, magnitude,
                                inter)

    want_q, want_k = want(x[:, :nq], wq), want(x[:, nq:nq + nkv], wk)

    def noise(y):
        return 2.0 ** -19 * _pair_length(y, args["rot"], inter)

    _check_bf16(_f64(q_out[:live, :nq * d]).reshape(want_q.shape), want_q, noise(want_q))
    _check_bf16(_f64(k_out[:live]).reshape(want_k.shape), want_k, noise(want_k))
    assert (q_out[live:] == 7).all() and (q_out[:, nq * d:] == 7).all() and (k_out[live:] == 7).all()

    # the cache: exactly the new tokens, everything else as it was
    pg, slot = table[seq, place // page].long(), place % page
    for pool, old, y, sc in ((cache.tensors[0], before[0], want_k, cache.tensors[2]),
                             (cache.tensors[1], before[1], x[:, nq + nkv:], cache.tensors[3])):
        got = _raw(pool)[pg, :, slot].view(pool.dtype)
        if sc is None:
            _check_bf16(_f64(got), y, noise(y))
        else:
            z = np.clip(y / _f64(sc)[:, None], -448, 448)
            assert (np.abs(_f64(got) - z) <= 2.0 ** -4 * np.abs(z) * (1 + 2.0 ** -15) + 2.0 ** -10).all()
        rest = _raw(pool).clone()
        rest[pg, :, slot] = old[pg, :, slot]
        assert torch.equal(rest, old)

    # in place, on another stream and without a cache: the same bits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Q.h3enc_op_rope_append(qkv, **call, q_out=qkv[:, :nq * d], k_out=qkv[:, nq * d:(nq + nkv) * d])
    side.synchronize()
    assert torch.equal(qkv[:live, :nq * d], q_out[:live, :nq * d])
    assert torch.equal(qkv[:live, nq * d:(nq + nkv) * d], k_out[:live])


def test_rope_append_reports_tokens_outside_the_cache():
    """Lengths and pages that do not fit: nothing of those tokens is stored, the others are."""
    g = _gen(5)
    cache = _pool(g, 3, 2, 16, 64, BF16)
    qkv = _randn(g, 6, 8 * 64)
    q_out = torch.zeros(6, 256, device="cuda", dtype=torch.bfloat16)
    table = _i32([[0, 1], [2, 3], [-1, 2], [2, 2 ** 31 - 1], [2, 0], [1, 0]])
    lens = _i32([3, 17, 1, 33, 0, -(2 ** 31)])        # stored; page 3; page -1; place 32; place -1; far below
    for cu in (None, _i32([0, 1, 2, 3, 4, 5, 6])):
        cache.tensors[0].fill_(float("nan"))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Q.h3enc_op_rope_append(qkv, 6, 4, 2, 64, None, None, 0.0, None, None, q_out, cache=cache, page_table=table,
                               seq_lens=lens, max_len=32, cu_rows=cu, status=status)
        assert int(status.item()) == 2
        k = cache.tensors[0]
        assert torch.equal(k[0, :, 2], qkv[0, 256:384].view(2, 64)) and int(torch.isnan(k).sum()) == k.numel() - 128
        assert torch.equal(q_out, qkv[:, :256])


def test_rope_append_rows_without_sequences():
    """Row offsets that begin late, stand still, run back or end early: only rows inside a sequence are written."""
    g = _gen(6)
    qkv = _randn(g, 10, 3 * 64)
    for cu, written in (([2, 2, 5, 5], {2, 3, 4}), ([0, 0, 0, 0], set()), ([0, 20, 20, 20], set(range(10))),
                        ([-3, 1, 1, 2], {0, 1})):
        q_out = torch.full((10, 64), 7.0, device="cuda", dtype=torch.bfloat16)
        Q.h3enc_op_rope_append(qkv, 10, 1, 1, 64, None, None, 0.0, None, None, q_out, seq_lens=_i32([9, 9, 9]), cu_rows=_i32(cu))
        for t in range(10):
            assert torch.equal(q_out[t], qkv[t, :64]) if t in written else bool((q_out[t] == 7).all()), (cu, t)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_positions_alone_and_far(inter):
    """Without sequences; positions up to the ends of int32, where an fp32 angle would be off by whole turns.  The
    frequencies' own rounding to 53 bits is 2^-53 * 2^31 radians there, far below the tolerance."""
    pos = [0, 1, -1, 4097, 10 ** 6, 2 ** 31 - 1, -(2 ** 31)]
    g = _gen(7)
    qkv = _randn(g, len(pos), 4 * 128)
    q_out = torch.empty(len(pos), 256, device="cuda", dtype=torch.bfloat16)
    Q.h3enc_op_rope_append(qkv, len(pos), 2, 1, 128, None, None, 0.0, Q.Rope(128, 5e6, interleaved=inter), _i32(pos), q_out)
    from decimal import Decimal, getcontext
    getcontext().prec = 50
    tau = Decimal("6.28318530717958647692528676655900576839433879875021")
    w, _ = O.decoder.frequencies(128, 5e6)
    angle = np.array([[float((Decimal(p) * Decimal(float(f))) % tau) for f in w] for p in pos])
    want = O.decoder.rotate(_f64(qkv).reshape(-1, 4, 128)[:, :2], angle, 1.0, inter)
    _check_bf16(_f64(q_out).reshape(want.shape), want, 2.0 ** -19 * _pair_length(want, 128, inter))


def test_rope_append_matches_the_tables_of_the_prefill():
    """The same rows through h3enc_op_rope_table and h3enc_op_qk_norm_rope: its tables hold fp32 angles, off by up to
    2^-24 * 2 of an angle of at most 500 plus the frequency's own 2^-24 of it: 2^-13, times a pair's length; both round once."""
    g = _gen(8)
    T, nq, nkv, d = 50, 4, 2, 128
    section = (24, 20, 20)
    pos = torch.randint(0, 500, (3, T), device="cuda", generator=g).to(torch.int32)
    cos, sin = (torch.empty(T, d // 2, device="cuda") for _ in range(2))
    Q.h3enc_op_rope_table(pos, T, d, 5e6, section, cos, sin)
    qkv = _randn(g, T, (nq + 2 * nkv) * d)
    w = (1 + 0.1 * torch.randn(2, d, device="cuda", generator=g)).to(torch.bfloat16)
    a, b = (torch.empty(T, nq * d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    Q.h3enc_op_qk_norm_rope(qkv, T, nq, nkv, d, w[0], w[1], 1e-6, cos, sin, 0, a)
    Q.h3enc_op_rope_append(qkv, T, nq, nkv, d, w[0], w[1], 1e-6, Q.Rope(d, 5e6, section=section), pos, b)
    a, b = (_f64(t).reshape(T, nq, d) for t in (a, b))
    assert (np.abs(a - b) <= 2.0 ** -7 * np.abs(b) * (1 + 2.0 ** -8) + 2.0 ** -12 * _pair_length(b, d, False)).all()


def test_rope_append_captured_and_replayed_with_other_lengths():
    g = _gen(9)
    n, nq, nkv, d, page = 5, 4, 2, 64, 16
    cache = _pool(g, n * 3, nkv, page, d, BF16)
    table = _table(g, n, 3, n * 3)
    lens = _i32([1, 5, 16, 17, 40])
    qkv, q_out = _randn(g, n, 8 * d), torch.zeros(n, nq * d, device="cuda", dtype=torch.bfloat16)
    rope = Q.Rope(d, 1e4)
    call = dict(T=n, n_heads=nq, n_kv_heads=nkv, head_dim=d, w_q=None, w_k=None, eps=0.0, rope=rope, seq_lens=lens,
                page_table=table, cache=cache, max_len=48)
    Q.h3enc_op_rope_append(qkv, **call, q_out=q_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.h3enc_op_rope_append(qkv, **call, q_out=q_out)
        lens.add_(1)
    want = []
    lens.copy_(_i32([1, 5, 16, 17, 40]))
    for step in range(3):
        qkv.copy_(_randn(g, n, 8 * d))
        want.append((qkv.clone(), lens.clone()))
        graph.replay()
    for q, length in want:
        at = length.long() - 1
        b = torch.arange(n, device="cuda")
        assert torch.equal(cache.tensors[1][table[b, at // page].long(), :, at % page], q[:, 6 * d:].view(n, nkv, d))
    angle = (want[-1][1].cpu().numpy() - 1.0)[:, None] * O.decoder.frequencies(d, 1e4)[0]
    y = O.decoder.rotate(_f64(want[-1][0]).reshape(n, 8, d)[:, :nq], angle, 1.0, False)
    _check_bf16(_f64(q_out).reshape(y.shape), y, 2.0 ** -19 * _pair_length(y, d, False))


# ---------------------------------------------------------------- cross attention

def _score_bound(q, k):
    """S1 of one sequence: q [M, nq, d], k [L, nkv, d]."""
    nq, nkv = q.shape[1], k.shape[1]
    return max(float((np.abs(q[:, h]) @ np.abs(k[:, h * nkv // nq]).T).max()) for h in range(nq)) / q.shape[2] ** 0.5


def _check_cross(got, q, k, v, p_err=2.0 ** -8):
    want = O.decoder.cross(q, k, v)
    if not len(k):
        assert not got.any()
        return
    delta = 16 * 2.0 ** -24 * _score_bound(q, k)
    A = O.decoder.cross(q, k, np.abs(v))
    _check_bf16(got, want, A * (2 * delta + p_err + 2.0 ** -18) * (1 + 2.0 ** -7))


def _cross_ws(d):
    return torch.zeros(Q.h3enc_op_attention_cross_workspace_bytes(d), dtype=torch.uint8, device="cuda")


CROSS = [
    ([1], [1], 1, 1, 64), ([1], [1], 64, 8, 128), ([1], [1024], 64, 8, 128), ([1], [5000], 12, 1, 64),
    ([1] * 7, [0, 1, 127, 128, 129, 300, 256], 40, 2, 128), ([3, 0, 130, 1, 33], [128, 50, 0, 700, 5], 8, 8, 64),
    ([300], [513], 4, 2, 64), ([257, 129], [640, 77], 28, 4, 128), ([40], [333], 10, 10, 128), ([700], [129], 2, 1, 128),
    ([5, 9], [260, 1], 130, 1, 64), ([70], [200], 256, 2, 64), ([2] * 150, [3 + i % 200 for i in range(150)], 4, 1, 128),
    ([1000], [64], 18, 18, 64), ([3, 2, 0, 4], [90, 700, 64, 0], 8, 1, 128), ([2, 3], [5, 1500], 12, 1, 64), ([1, 0, 900], [3, 77, 200], 4, 2, 64),
    ([32] * 3, [65, 1, 640], 6, 6, 128), ([1] * 1000 + [40], [1 + i % 9 for i in range(1000)] + [500], 2, 1, 64), ([31], [9000], 5, 1, 128), ([513, 1], [1, 4097], 20, 4, 64)]


@pytest.mark.parametrize("qlens,klens,nq,nkv,d", CROSS)
def test_attention_cross(qlens, klens, nq, nkv, d):
    g = _gen(sum(qlens) + sum(klens) + nq)
    before, behind = 3, 5                                     # rows of no sequence; NaN on the key side
    Tq, Tk = sum(qlens) + before + behind, sum(klens) + before + behind
    q = _randn(g, Tq, nq * d + 16, scale=2.0)[:, 8:8 + nq * d]
    kv = _randn(g, Tk, 2 * nkv * d + 24)
    kv[:before] = float("nan")
    kv[Tk - behind:] = float("nan")
    k, v = kv[:, :nkv * d], kv[:, nkv * d + 8:2 * nkv * d + 8]
    o = torch.full((Tq, nq * d + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    cu_q, cu_k = (_i32(before + np.concatenate([[0], np.cumsum(x)])) for x in (qlens, klens))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = _cross_ws(d)
    Q.h3enc_op_attention_cross(q, k, v, o[:, :nq * d], nq, nkv, d, ws, cu_q, cu_k, status)
    assert int(status.item()) == 0
    assert (o[:before] == 7).all() and (o[Tq - behind:] == 7).all() and (o[:, nq * d:] == 7).all()
    qf, kf, vf = _f64(q).reshape(Tq, nq, d), _f64(k).reshape(Tk, nkv, d), _f64(v).reshape(Tk, nkv, d)
    got = _f64(o[:, :nq * d]).reshape(Tq, nq, d)
    a = b = before
    for m, n in zip(qlens, klens):
        if m:
            _check_cross(got[a:a + m], qf[a:a + m], kf[b:b + n], vf[b:b + n])
        a, b = a + m, b + n
    # again, on another stream, in a workspace that holds the last call's: the same bits
    again = torch.zeros(Tq, nq * d, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Q.h3enc_op_attention_cross(q, k, v, again, nq, nkv, d, ws, cu_q, cu_k)
    side.synchronize()
    live = slice(before, Tq - behind)
    assert torch.equal(again[live], o[live, :nq * d])


@pytest.mark.parametrize("Tq,Tk,nq,nkv,d", [(4096, 300, 8, 1, 128), (2000, 1100, 10, 10, 64), (1000, 2500, 16, 4, 128)])
def test_attention_cross_of_many_items_with_boundaries_inside(Tq, Tk, nq, nkv, d):
    """More items than SMs: every boundary between two runs cuts one, whose two parts meet.  The same bits every time,
    whichever part is last, also over a workspace that other sizes have used."""
    g = _gen(Tq)
    q, kv = _randn(g, Tq, nq * d), _randn(g, Tk, 2 * nkv * d)
    k, v = kv[:, :nkv * d], kv[:, nkv * d:]
    ws, outs = _cross_ws(d), []
    for i in range(6):
        o = torch.zeros(Tq, nq * d, device="cuda", dtype=torch.bfloat16)
        Q.h3enc_op_attention_cross(q, k, v, o, nq, nkv, d, ws)
        outs.append(o)
        other = torch.zeros(1 + 700 * (i % 2), nq * d, device="cuda", dtype=torch.bfloat16)
        Q.h3enc_op_attention_cross(q[:len(other)], k[i:], v[i:], other, nq, nkv, d, ws)
    assert all(torch.equal(o, outs[0]) for o in outs)
    rows = torch.cat([torch.arange(0, Tq, 97), torch.arange(Tq - 3, Tq)]).cuda()
    _check_cross(_f64(outs[0][rows]).reshape(-1, nq, d), _f64(q[rows]).reshape(-1, nq, d), _f64(k).reshape(Tk, nkv, d),
                 _f64(v).reshape(Tk, nkv, d))


@pytest.mark.parametrize("n,m,keys,nq,nkv,d", [(64, 40, 333, 10, 10, 128), (64, 40, 600, 10, 10, 64), (64, 90, 900, 4, 2, 128),
                                                 (1, 40, 333, 10, 10, 128), (31, 40, 600, 10, 10, 64), (2, 300, 1024, 32, 4, 128)])
def test_attention_cross_of_many_whole_items(n, m, keys, nq, nkv, d):
    """Most items lie whole in a run, single tiles (two halves merged) and pairs, after others of the same CTA, with
    values behind the last segment that must not matter.  The same bits every time."""
    g = _gen(n * m + d)
    before, behind = 3, 5
    q, kv = _randn(g, n * m + before + behind, nq * d), _randn(g, n * keys + before + behind, 2 * nkv * d)
    kv[:before] = float("nan")
    kv[-behind:] = float("nan")
    k, v = kv[:, :nkv * d], kv[:, nkv * d:]
    cu_q, cu_k = _i32(before + m * np.arange(n + 1)), _i32(before + keys * np.arange(n + 1))
    ws, outs = _cross_ws(d), []
    for i in range(8):
        o = torch.zeros(len(q), nq * d, device="cuda", dtype=torch.bfloat16)
        Q.h3enc_op_attention_cross(q, k, v, o, nq, nkv, d, ws, cu_q, cu_k)
        outs.append(o)
    assert all(torch.equal(o, outs[0]) for o in outs)
    assert not outs[0][:before].any() and not outs[0][-behind:].any()
    for s in {0, min(1, n - 1), n // 2, n - 1}:
        a, b = slice(before + m * s, before + m * (s + 1)), slice(before + keys * s, before + keys * (s + 1))
        _check_cross(_f64(outs[0][a]).reshape(m, nq, d), _f64(q[a]).reshape(m, nq, d), _f64(k[b]).reshape(keys, nkv, d),
                     _f64(v[b]).reshape(keys, nkv, d))


def test_attention_cross_of_one_sequence_needs_no_offsets():
    g = _gen(1)
    q, kv = _randn(g, 50, 256), _randn(g, 200, 256)
    a, b = (torch.zeros(50, 256, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    Q.h3enc_op_attention_cross(q, kv[:, :128], kv[:, 128:], a, 4, 2, 64, _cross_ws(64))
    Q.h3enc_op_attention_cross(q, kv[:, :128], kv[:, 128:], b, 4, 2, 64, _cross_ws(64), _i32([0, 50]), None)
    assert torch.equal(a, b)
    _check_cross(_f64(a).reshape(50, 4, 64), _f64(q).reshape(50, 4, 64), _f64(kv[:, :128]).reshape(200, 2, 64),
                 _f64(kv[:, 128:]).reshape(200, 2, 64))
    Q.h3enc_op_attention_cross(q, kv[:0, :128], kv[:0, 128:], a, 4, 2, 64, _cross_ws(64))       # no states at all
    assert not a.any()
    Q.h3enc_op_attention_cross(q[:1], kv[:0, :128], kv[:0, 128:], b[:1], 4, 2, 64, _cross_ws(64))   # (few rows: another path)
    assert not b[0].any() and b[1:].any()
    Q.h3enc_op_attention_cross(q[:0], kv[:, :128], kv[:, 128:], a[:0], 4, 2, 64, _cross_ws(64))


def test_attention_cross_infinite_and_masked_values():
    """An infinite value where every weight is above 0 is an infinite output of that column and head; a score of -inf
    is a weight of 0; NaN and infinities of another sequence reach nothing."""
    g = _gen(2)
    L, d = 300, 64
    q, k, v = _randn(g, 8, d), _randn(g, L + 200, d), _randn(g, L + 200, d)
    k[L:], v[L:] = float("nan"), float("inf")
    v[17, 5] = float("inf")
    v[200, 6] = float("-inf")
    o = torch.zeros(8, d, device="cuda", dtype=torch.bfloat16)
    Q.h3enc_op_attention_cross(q, k, v, o, 1, 1, d, _cross_ws(d), _i32([0, 8, 8]), _i32([0, L, L + 200]))
    assert (o[:, 5] == float("inf")).all() and (o[:, 6] == float("-inf")).all()
    rest = [i for i in range(d) if i not in (5, 6)]
    clean = v[:L].clone()
    clean[:, 5:7] = 0
    want = O.decoder.cross(_f64(q)[:, None], _f64(k[:L])[:, None], _f64(clean)[:, None])[:, 0]
    assert np.abs(_f64(o)[:, rest] - want[:, rest]).max() < 2.0 ** -6
    # keys that every query scores -inf: the first tile, and a part of the last
    q2, k2 = q.abs() + 0.5, k[:L].clone()
    k2[:140, 0], k2[290:, 0] = float("-inf"), float("-inf")
    Q.h3enc_op_attention_cross(q2, k2, clean, o, 1, 1, d, _cross_ws(d))
    _check_cross(_f64(o)[:, None], _f64(q2)[:, None], _f64(k2[140:290])[:, None], _f64(clean[140:290])[:, None])


def test_attention_cross_far_apart_scores():
    """One key far above the others, in the first, a middle and the last tile: the raised maximum and the joined parts."""
    g = _gen(3)
    L, d = 2000, 128
    q, v = _randn(g, 16, d), _randn(g, L, d)
    for at in (0, 1000, L - 1):
        k = _randn(g, L, d)
        k[at] = (q[3].float() * 20).to(torch.bfloat16)
        o = torch.zeros(16, d, device="cuda", dtype=torch.bfloat16)
        Q.h3enc_op_attention_cross(q, k, v, o, 1, 1, d, _cross_ws(d))
        _check_cross(_f64(o)[:, None], _f64(q)[:, None], _f64(k)[:, None], _f64(v)[:, None])


@pytest.mark.parametrize("cu_q,cu_k", [([0, 5, 3, 8], [0, 10, 20, 30]), ([0, 3, 5, 8], [0, 20, 10, 30]), ([0, 3, 5, 9], [0, 10, 20, 30]),
                                       ([-1, 3, 5, 8], [0, 10, 20, 30]), ([0, 3, 5, 8], [0, 10, 20, 2 ** 31 - 1]),
                                       ([2 ** 31 - 1, -5, 8, 8], [9, 9, -9, 30])])
def test_attention_cross_reports_bad_offsets(cu_q, cu_k):
    g = _gen(4)
    q, k = _randn(g, 8, 128), _randn(g, 30, 128)
    o = torch.full((10, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Q.h3enc_op_attention_cross(q, k, k, o[:8], 2, 2, 64, _cross_ws(64), _i32(cu_q), _i32(cu_k), status)
    assert int(status.item()) == 2 and (o[8:] == 7).all()
    # the sequences whose offsets are sound are right
    if cu_q == [0, 3, 5, 8]:
        assert np.isfinite(_f64(o[:8])).all()
        _check_cross(_f64(o[:3]).reshape(3, 2, 64), _f64(q[:3]).reshape(3, 2, 64), *(_f64(k[:cu_k[1]]).reshape(-1, 2, 64),) * 2)


# The next ones are the three tests around them at sizes that the tcgen05 kernel takes (over 32 rows per kv head and sequence): cut into parts
# of single steps (one head), and whole items of many heads, pairs of row tiles (200 rows) and single ones (100), whose halves meet.
MANY_ROWS = [(200, 1), (200, 160), (100, 1), (100, 160)]


@pytest.mark.parametrize("rows,heads", MANY_ROWS)
def test_attention_cross_of_many_rows_infinite_and_masked_values(rows, heads):
    g = _gen(23 + rows + heads)
    L, d = 300, 64
    q, k, v = _randn(g, rows, heads * d), _randn(g, L + 200, heads * d), _randn(g, L + 200, heads * d)
    k[L:], v[L:] = float("nan"), float("inf")
    vh = v.view(L + 200, heads, d)
    vh[17, :, 5], vh[200, :, 6] = float("inf"), float("-inf")
    o = torch.zeros(rows, heads * d, device="cuda", dtype=torch.bfloat16)
    Q.h3enc_op_attention_cross(q, k, v, o, heads, heads, d, _cross_ws(d), _i32([0, rows, rows]), _i32([0, L, L + 200]))
    got = _f64(o).reshape(rows, heads, d)
    assert (got[..., 5] == np.inf).all() and (got[..., 6] == -np.inf).all()
    clean = v[:L].clone()
    clean.view(L, heads, d)[..., 5:7] = 0
    got[..., 5:7] = 0
    qf, kf, vf = (_f64(t).reshape(-1, heads, d) for t in (q, k[:L], clean))
    _check_cross(got, qf, kf, vf)
    # keys that every query scores -inf: two whole tiles (one of each half of a single tile's steps), and a part of the last
    for first, last in ((140, 290), (256, 290)):
        q2, k2 = q.abs() + 0.5, k[:L].clone()
        k2.view(L, heads, d)[:first, :, 0], k2.view(L, heads, d)[last:, :, 0] = float("-inf"), float("-inf")
        Q.h3enc_op_attention_cross(q2, k2, clean, o, heads, heads, d, _cross_ws(d))
        _check_cross(_f64(o).reshape(rows, heads, d), _f64(q2).reshape(rows, heads, d), kf[first:last], vf[first:last])


@pytest.mark.parametrize("rows,heads", MANY_ROWS)
@pytest.mark.parametrize("d,L", [(128, 2000), (64, 700)])
def test_attention_cross_of_many_rows_far_apart_scores(rows, heads, d, L):
    """Keys far above the others for some rows, in the first, a middle and the last tile, growing: the sums before each are rescaled."""
    g = _gen(24 + rows + heads + d)
    q, v = _randn(g, rows, heads * d), _randn(g, L, heads * d)
    for places in ((0,), (L // 2,), (L - 1,), (5, 200, L // 2, L - 40)):
        k = _randn(g, L, heads * d)
        for i, at in enumerate(places):
            k[at] = (q[(3, 17, 64, rows - 1)[i]].float() * (20 if len(places) == 1 else 4 + 6 * i)).to(torch.bfloat16)
            k[(at + 31) % L] = (q[3].float() * (4 + 3 * i)).to(torch.bfloat16)
        o = torch.zeros(rows, heads * d, device="cuda", dtype=torch.bfloat16)
        Q.h3enc_op_attention_cross(q, k, v, o, heads, heads, d, _cross_ws(d))
        some = sorted({0, 1, heads // 2, heads - 1} & set(range(heads)))   # heads that are compared
        qf, kf, vf, got = (_f64(t.view(-1, heads, d)[:, some]) for t in (q, k, v, o))
        for h in range(len(some)):       # (each head's own bound on scores)
            _check_cross(got[:, h:h + 1], qf[:, h:h + 1], kf[:, h:h + 1], vf[:, h:h + 1])


@pytest.mark.parametrize("qlens,klens,nq,nkv,d", [([1] * 5, [900, 3, 65, 700, 1000], 16, 2, 128), ([8], [900], 4, 1, 64), ([31], [900], 5, 5, 128),
                                                  ([2, 2], [900, 901], 32, 2, 64)])
def test_attention_cross_of_few_rows_keeps_the_bits_of_weights(qlens, klens, nq, nkv, d):
    g = _gen(25 + nq)
    q, kv = _randn(g, sum(qlens), nq * d), _randn(g, sum(klens), 2 * nkv * d)
    o = torch.zeros(sum(qlens), nq * d, device="cuda", dtype=torch.bfloat16)
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]) for x in (qlens, klens))
    Q.h3enc_op_attention_cross(q, kv[:, :nkv * d], kv[:, nkv * d:], o, nq, nkv, d, _cross_ws(d), _i32(cu_q), _i32(cu_k))
    caught = 0
    for s in range(len(qlens)):
        kf, vf = _f64(kv[cu_k[s]:cu_k[s + 1]]).reshape(-1, 2, nkv, d).transpose(1, 0, 2, 3)
        for t in range(cu_q[s], cu_q[s + 1]):
            qf, got = (_f64(x[t]).reshape(1, nq, d) for x in (q, o))
            _check_cross(got, qf, kf, vf, 2.0 ** -16)
            want, A = O.decoder.cross(qf, kf, vf)[0], O.decoder.cross(qf, kf, np.abs(vf))[0]
            noise = A * (2 * 16 * 2.0 ** -24 * _score_bound(qf, kf) + 2.0 ** -16 + 2.0 ** -18) * (1 + 2.0 ** -7)
            caught += (np.abs(_rounded_weights(qf[0], kf, vf, torch.bfloat16) - want) > 2.0 ** -8 * np.abs(want) + noise).sum()
    assert caught > 0       # (one rounding to bf16 would be seen)


@pytest.mark.parametrize("cu_q,cu_k,sound", [([0, 300, 100, 400], [0, 200, 300, 500], []), ([0, 150, 250, 400], [0, 300, 200, 500], [0]),
                                             ([0, 150, 250, 401], [0, 200, 300, 500], [0, 1]), ([-7, 150, 250, 400], [0, 200, 300, 500], [1, 2]),
                                             ([0, 150, 250, 400], [0, 200, 300, 2 ** 31 - 1], [0, 1]),
                                             ([2 ** 31 - 1, -5, 400, 400], [9, 9, -9, 500], [])])
def test_attention_cross_of_many_rows_reports_bad_offsets(cu_q, cu_k, sound):
    """As the test above with over 32 rows per kv head and sequence, which another kernel takes."""
    g = _gen(16)
    q, k = _randn(g, 400, 256), _randn(g, 500, 128)
    o = torch.full((410, 256), 7.0, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Q.h3enc_op_attention_cross(q, k, k, o[:400], 4, 2, 64, _cross_ws(64), _i32(cu_q), _i32(cu_k), status)
    assert int(status.item()) == 2 and (o[400:] == 7).all() and np.isfinite(_f64(o)).all()
    for s in sound:
        a, b = slice(cu_q[s], cu_q[s + 1]), slice(cu_k[s], cu_k[s + 1])
        _check_cross(_f64(o[a]).reshape(-1, 4, 64), _f64(q[a]).reshape(-1, 4, 64), *(_f64(k[b]).reshape(-1, 2, 64),) * 2)


def test_attention_cross_of_offsets_between_the_ends():
    """Every second offset back at 0: no row is in more than one sequence, so the weights stay within the call's bound (each
    sequence by itself, they would pass 32 bits; tests/cross_walk_host.cpp walks such calls on the host)."""
    g = _gen(17)
    n, Tq, Tk, d = 1024, 16384, 100000, 64
    q, kv = _randn(g, Tq, 64 * d), _randn(g, Tk, 16 * d)
    o = torch.full((Tq + 8, 64 * d), 7.0, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu_q, cu_k = (_i32([x * (i % 2) for i in range(n + 1)]) for x in (Tq, Tk))
    Q.h3enc_op_attention_cross(q, kv[:, :8 * d], kv[:, 8 * d:], o[:Tq], 64, 8, d, _cross_ws(d), cu_q, cu_k, status)
    assert int(status.item()) == 2 and (o[Tq:] == 7).all() and bool(torch.isfinite(o).all())


def test_attention_cross_of_few_rows_and_offsets_between_the_ends():
    """The same with so few rows that the decoding kernel takes them: 4096 queries of one head by each of 512 sequences would
    be 3.3e10 tiles.  The workspace still serves a sound call."""
    g = _gen(18)
    n, Tq, Tk, d = 1024, 4096, 500000, 64
    q, kv = _randn(g, Tq, 8 * d), _randn(g, Tk, 16 * d)
    o = torch.full((Tq + 8, 8 * d), 7.0, device="cuda", dtype=torch.bfloat16)
    status, ws = torch.zeros(1, dtype=torch.int32, device="cuda"), _cross_ws(d)
    cu_q, cu_k = (_i32([x * (i % 2) for i in range(n + 1)]) for x in (Tq, Tk))
    Q.h3enc_op_attention_cross(q, kv[:, :8 * d], kv[:, 8 * d:], o[:Tq], 8, 8, d, ws, cu_q, cu_k, status)
    assert int(status.item()) == 2 and (o[Tq:] == 7).all() and bool(torch.isfinite(o).all())
    Q.h3enc_op_attention_cross(q[:8], kv[:900, :8 * d], kv[:900, 8 * d:], o[:8], 8, 8, d, ws, _i32([0, 3, 8]), _i32([0, 200, 900]))
    for a, b in ((slice(0, 3), slice(0, 200)), (slice(3, 8), slice(200, 900))):
        _check_cross(_f64(o[a]).reshape(-1, 8, d), _f64(q[a]).reshape(-1, 8, d), *(_f64(t).reshape(-1, 8, d) for t in (kv[b, :8 * d], kv[b, 8 * d:])))


def test_attention_cross_captured_and_replayed_with_other_lengths():
    g = _gen(5)
    nq, nkv, d = 8, 2, 128
    q, kv = _randn(g, 100, nq * d), _randn(g, 1500, 2 * nkv * d)
    k, v = kv[:, :nkv * d], kv[:, nkv * d:]
    o = torch.zeros(100, nq * d, device="cuda", dtype=torch.bfloat16)
    cu_q, cu_k, ws = _i32([0, 100, 100]), _i32([0, 1500, 1500]), _cross_ws(d)
    Q.h3enc_op_attention_cross(q, k, v, o, nq, nkv, d, ws, cu_q, cu_k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.h3enc_op_attention_cross(q, k, v, o, nq, nkv, d, ws, cu_q, cu_k)
    for a, b in (([0, 100, 100], [0, 1500, 1500]), ([0, 1, 100], [0, 1, 1500]), ([0, 60, 61], [0, 700, 700])):
        cu_q.copy_(_i32(a))
        cu_k.copy_(_i32(b))
        o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            s, e = slice(a[i], a[i + 1]), slice(b[i], b[i + 1])
            if a[i] < a[i + 1]:
                _check_cross(_f64(o[s]).reshape(-1, nq, d), _f64(q[s]).reshape(-1, nq, d), _f64(k[e]).reshape(-1, nkv, d),
                             _f64(v[e]).reshape(-1, nkv, d))
        assert (o[a[2]:] == 3).all()


# ---------------------------------------------------------------- attention behind shared prefixes

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


SHARED = [
    # sequences of each group, lengths of the prefixes, own lengths
    ([1], [1], [0], 1, 1, 64, BF16, 16), ([1], [1000], [1], 64, 8, 128, BF16, 64), ([4], [129], [20, 0, 60, 1], 64, 8, 128, BF16, 128),
    ([1, 0, 3, 2], [700, 50, 0, 127], [5, 100, 3, 0, 40, 260], 4, 2, 64, BF16, 16), ([40], [640], [i * 7 for i in range(40)], 8, 1, 128, BF16, 32),
    ([2], [5000], [3, 9], 130, 1, 64, BF16, 256), ([17], [300], [1] * 17, 40, 2, 128, BF16, 64), ([70], [256], [2] * 70, 7, 7, 64, BF16, 16),
    ([1], [1], [0], 2, 1, 64, E4M3, 16), ([1], [1000], [1], 64, 8, 128, E4M3, 64), ([5], [257], [20, 0, 60, 1, 300], 28, 4, 128, E4M3, 128),
    ([1, 0, 3, 2], [700, 50, 0, 127], [5, 100, 3, 0, 40, 260], 4, 2, 64, E4M3, 32), ([40], [900], [i * 3 for i in range(40)], 20, 4, 64, E4M3, 256),
    ([33], [4000], [10] * 33, 12, 1, 128, E4M3, 16)]


def _far_bound(n, nkv, d, dtype):
    """A bound on the prefixes' lengths with which the call passes over them once for all (it goes by the bound)."""
    return int(2e8 / (2 * n * nkv * d * (2 if dtype == BF16 else 1))) + 1


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("groups,plens,lens,nq,nkv,d,dtype,page", SHARED)
def test_attention_decode_shared(groups, plens, lens, nq, nkv, d, dtype, page, far):
    g = _gen(sum(plens) + sum(lens) + nq)
    n, rows = len(lens), np.concatenate([[0], np.cumsum(groups)])
    assert rows[-1] == n
    max_prefix, max_len = max(plens), max(max(lens), 1)
    pcols, cols = -(-max_prefix // page), -(-max_len // page)
    pages = len(plens) * pcols + n * cols + 2
    cache = _pool(g, pages, nkv, page, d, dtype, apart=16)
    ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    if far:
        max_prefix = max(max_prefix, _far_bound(n, nkv, d, dtype))
    ptable = torch.cat([ids[:len(plens) * pcols].view(len(plens), pcols), ids.new_full((len(plens), 2 - (-max_prefix // page) - pcols), -1)], 1).contiguous()
    table = ids[len(plens) * pcols:][:n * cols].view(n, cols).contiguous()

    def tokens(ls):
        return [torch.randn(x, nkv, d, device="cuda", generator=g) for x in ls], [torch.randn(x, nkv, d, device="cuda", generator=g) for x in ls]

    pre, mine = _fill(cache, ptable, plens, *tokens(plens)), _fill(cache, table, lens, *tokens(lens))
    q = _randn(g, n, nq * d + 8, scale=2.0)[:, :nq * d]
    o = torch.full((n + 1, nq * d + 8), 7.0, device="cuda", dtype=torch.bfloat16)
    w_in = torch.rand(n, max_len + 3, device="cuda", generator=g)
    w_out = torch.full_like(w_in, -5.0)
    ws = torch.zeros(Q.h3enc_op_attention_decode_shared_workspace_bytes(n, nq, max_len, True), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    prefix_rows = _i32(rows) if len(groups) > 1 else None
    args = (cache, ptable, _i32(plens), max_prefix, table, _i32(lens), nq, max_len, ws)
    Q.h3enc_op_attention_decode_shared(q, o[:n, :nq * d], *args, prefix_rows=prefix_rows, weight_in=w_in, weight_out=w_out,
                                       status=status)
    assert int(status.item()) == 0
    assert (o[n:] == 7).all() and (o[:, nq * d:] == 7).all()
    qf, got = _f64(q).reshape(n, nq, d), _f64(o[:n, :nq * d]).reshape(n, nq, d)
    p_err = 2.0 ** -8 if dtype == BF16 else 2.0 ** -11
    m = nq // nkv
    for b in range(n):
        (pk, pv), (k, v) = pre[int(np.searchsorted(rows, b, side="right")) - 1], mine[b]
        want, p = O.decoder.attend_prefix(qf[b], pk, pv, k, v)
        if not len(pk) + len(k):
            assert not got[b].any()
            continue
        delta = 16 * 2.0 ** -24 * _score_bound(qf[b][None], np.concatenate([pk, k]))
        A = O.decoder.attend_prefix(qf[b], pk, np.abs(pv), k, np.abs(v))[0]
        light = 2.0 ** -37 * np.abs(pv).sum(0).repeat(m, 0) if dtype == E4M3 and len(pk) else 0.0
        _check_bf16(got[b], want, (A * (2 * delta + p_err + 2.0 ** -16 + 2.0 ** -18) + light) * (1 + 2.0 ** -7))
        w = _f64(w_out[b])
        assert (w[lens[b]:] == -5).all()
        p = p.sum(0)
        assert (np.abs(w[:lens[b]] - _f64(w_in[b])[:lens[b]] - p) <= (2 * delta + 2.0 ** -18) * p + 2.0 ** -22 * (1 + p)).all()
    # without weights, again, on another stream: the same bits
    again = torch.zeros(n, nq * d, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Q.h3enc_op_attention_decode_shared(q, again, *args, prefix_rows=prefix_rows)
    side.synchronize()
    assert torch.equal(again, o[:n, :nq * d])


def test_attention_decode_shared_without_prefixes_is_attention_decode():
    g = _gen(11)
    n, nq, nkv, d, page = 5, 8, 2, 128, 16
    cache = _pool(g, 40, nkv, page, d, BF16)
    table, lens = _table(g, n, 8, 40), [100, 0, 1, 128, 33]
    _fill(cache, table, lens, *([torch.randn(x, nkv, d, device="cuda", generator=g) for x in lens] for _ in range(2)))
    q = _randn(g, n, nq * d)
    a, b, c = (torch.zeros(n, nq * d, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    ws = torch.zeros(Q.h3enc_op_attention_decode_shared_workspace_bytes(n, nq, 128), dtype=torch.uint8, device="cuda")
    Q.h3enc_op_attention_decode(q, a, cache, table, _i32(lens), nq, 128, ws)
    Q.h3enc_op_attention_decode_shared(q, b, cache, table[:0], _i32([]), 0, table, _i32(lens), nq, 128, ws)
    assert torch.equal(a, b)
    # sequences of no group, and a group whose prefix is empty, have none either
    for bound in (64, _far_bound(n, nkv, d, BF16)):
        wide = table.new_zeros(2, -(-bound // page))
        Q.h3enc_op_attention_decode_shared(q, c, cache, wide, _i32([0, 0]), bound, table, _i32(lens), nq, 128, ws,
                                           prefix_rows=_i32([1, 2, 4]))
        assert torch.equal(a, c)
    Q.h3enc_op_attention_decode(q, c, cache, table, _i32(lens), nq, 128, ws)      # the workspace serves both
    assert torch.equal(a, c)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_attention_decode_shared_reports_bad_pages_and_lengths(dtype, far):
    """A page outside the cache reads as zero keys and values; a length outside its bound is clamped into it."""
    g = _gen(12)
    n, nq, nkv, d, page = 3, 4, 2, 64, 16
    cache = _pool(g, 30, nkv, page, d, dtype)
    ids = torch.randperm(30, device="cuda", generator=g).to(torch.int32)
    spare = _far_bound(n, nkv, d, dtype) // page + 1 if far else 0
    ptable, table = torch.cat([ids[:8], ids.new_full((spare,), -1)]).view(1, -1), ids[8:14].view(3, 2).contiguous()
    pk, pv = ([torch.randn(120, nkv, d, device="cuda", generator=g)] for _ in range(2))
    k, v = ([torch.randn(20, nkv, d, device="cuda", generator=g) for _ in range(n)] for _ in range(2))
    (pk, pv), = _fill(cache, ptable, [120], pk, pv)
    own = _fill(cache, table, [20] * n, k, v)
    q, o = _randn(g, n, nq * d), torch.zeros(n, nq * d, device="cuda", dtype=torch.bfloat16)
    ws = torch.zeros(Q.h3enc_op_attention_decode_shared_workspace_bytes(n, nq, 32), dtype=torch.uint8, device="cuda")

    def check(bad_page, prefix_len, max_prefix):
        t = ptable.clone()
        if bad_page is not None:
            t[0, 2] = bad_page
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Q.h3enc_op_attention_decode_shared(q, o, cache, t, _i32([prefix_len]), max_prefix, table, _i32([20] * n), nq, 32, ws,
                                           status=status)
        assert int(status.item()) == 2
        length = min(max(prefix_len, 0), max_prefix)
        kk, vv = pk[:length].copy(), pv[:length].copy()
        if bad_page is not None:
            kk[32:48], vv[32:48] = 0, 0
        for b in range(n):
            want, _ = O.decoder.attend_prefix(_f64(q[b]).reshape(nq, d), kk, vv, *own[b])
            assert np.abs(_f64(o[b]).reshape(nq, d) - want).max() <= 2.0 ** -6

    bound = page * spare if far else 120
    for page_no in (-1, 30, 2 ** 31 - 1, -(2 ** 31)):
        check(page_no, 120, bound)
    check(None, -3, bound)
    if not far:       # (the table holds no page for what a clamped length of that bound would read)
        check(None, 121, 120)
        check(None, 2 ** 31 - 1, 33)


def _rounded_weights(q, k, v, dtype):
    """One token's output if the weights, relative to the largest, were rounded to one number of 16 bits (a planted mistake)."""
    (nq, d), nkv = q.shape, k.shape[1]
    o = np.zeros(q.shape)
    for h in range(nq):
        s = k[:, h * nkv // nq] @ q[h] / d ** 0.5
        e = np.exp(s - s.max())
        p = torch.from_numpy(e * 2.0 ** 13).to(dtype).double().numpy() * 2.0 ** -13
        o[h] = p @ v[:, h * nkv // nq] / e.sum()
    return o


# Off by 2^-16 of a weight in two halves of bf16 (and 2^-18 where the first is cut), 2^-22 in two of f16, 2^-11 in one.
@pytest.mark.parametrize("dtype,far,p_err", [(BF16, False, 2.0 ** -16), (BF16, True, 2.0 ** -16 + 2.0 ** -18), (E4M3, False, 2.0 ** -22),
                                             (E4M3, True, 2.0 ** -11)])
@pytest.mark.parametrize("nq,nkv,d", [(8, 2, 128), (40, 2, 64)])
def test_attention_decode_shared_keeps_the_bits_of_weights(dtype, far, p_err, nq, nkv, d):
    g = _gen(20 + nq)
    n, page, P = 12, 64, 900
    cols = -(-P // page)
    bound = max(P, _far_bound(n, nkv, d, dtype)) if far else P
    cache = _pool(g, cols + n, nkv, page, d, dtype)
    ids = torch.randperm(cols + n, device="cuda", generator=g).to(torch.int32)
    ptable, table = torch.cat([ids[:cols], ids.new_full((-(-bound // page) - cols,), -1)]).view(1, -1), ids[cols:].view(n, 1).contiguous()
    lens = [(7 * b) % 60 for b in range(n)]
    rnd = lambda ls: [torch.randn(x, nkv, d, device="cuda", generator=g) for x in ls]   # noqa: E731
    (pk, pv), = _fill(cache, ptable, [P], rnd([P]), rnd([P]))
    own = _fill(cache, table, lens, rnd(lens), rnd(lens))
    q, o = _randn(g, n, nq * d), torch.zeros(n, nq * d, device="cuda", dtype=torch.bfloat16)
    ws = torch.zeros(Q.h3enc_op_attention_decode_shared_workspace_bytes(n, nq, page), dtype=torch.uint8, device="cuda")
    Q.h3enc_op_attention_decode_shared(q, o, cache, ptable, _i32([P]), bound, table, _i32(lens), nq, page, ws)
    caught = 0
    for b in range(n):
        k, v, qf = np.concatenate([pk, own[b][0]]), np.concatenate([pv, own[b][1]]), _f64(q[b]).reshape(nq, d)
        want, A = O.decode.attend_one(qf, k, v)[0], O.decode.attend_one(qf, k, np.abs(v))[0]
        noise = A * (2 * 16 * 2.0 ** -24 * _score_bound(qf[None], k) + p_err + 2.0 ** -18) * (1 + 2.0 ** -7)
        if dtype == E4M3 and far:
            noise += 2.0 ** -37 * np.abs(pv).sum(0).repeat(nq // nkv, 0)
        _check_bf16(_f64(o[b]).reshape(nq, d), want, noise)
        caught += (np.abs(_rounded_weights(qf, k, v, torch.bfloat16) - want) > 2.0 ** -8 * np.abs(want) + noise).sum()
    assert caught > 0 or p_err == 2.0 ** -11       # (one rounding to bf16 would be seen)


def test_attention_decode_shared_infinite_values_of_a_prefix():
    """Both ways of reading a prefix: an infinite value where every weight is above 0 is an infinite output of that column; a
    score of -inf is a weight of 0; keys of -inf alone in a run of tiles leave the others as they are."""
    g = _gen(22)
    n, nq, nkv, d, page, P = 9, 8, 1, 64, 64, 700
    cols = -(-P // page)
    cache = _pool(g, cols + n, nkv, page, d, BF16)
    for far in (False, True):
        bound = _far_bound(n, nkv, d, BF16) if far else P
        ptable = torch.full((1, -(-bound // page)), -1, dtype=torch.int32, device="cuda")
        ptable[0, :cols] = torch.arange(cols, device="cuda")
        table, lens = _i32([[cols + b] for b in range(n)]), [0, 1, 5, 64, 33, 0, 2, 9, 17]
        rnd = lambda ls: [torch.randn(x, nkv, d, device="cuda", generator=g) for x in ls]   # noqa: E731
        pk, pv = rnd([P])[0], rnd([P])[0]
        pv[17, 0, 5], pv[690, 0, 6] = float("inf"), float("-inf")
        pk[:140, 0, 0], pk[256:384, 0, 0], pk[699, 0, 0] = float("-inf"), float("-inf"), float("-inf")
        for masked in (False, True):
            k = pk.clone()
            if not masked:
                k[:, 0, 0] = 0
            v = pv.clone()
            if masked:
                v[17, 0, 5] = 0
            (kf, vf), = _fill(cache, ptable, [P], [k], [v])
            own = _fill(cache, table, lens, rnd(lens), rnd(lens))
            q = _randn(g, n, nq * d).abs() + 0.25
            o = torch.zeros(n, nq * d, device="cuda", dtype=torch.bfloat16)
            ws = torch.zeros(Q.h3enc_op_attention_decode_shared_workspace_bytes(n, nq, page), dtype=torch.uint8, device="cuda")
            Q.h3enc_op_attention_decode_shared(q, o, cache, ptable, _i32([P]), bound, table, _i32(lens), nq, page, ws)
            got, vf = _f64(o).reshape(n, nq, d), vf.copy()
            assert (got[..., 6] == -np.inf).all() and (masked or (got[..., 5] == np.inf).all())
            got[..., 6], vf[..., 6] = 0, 0
            seen = np.isfinite(kf[:, 0, 0])
            if not masked:
                got[..., 5], vf[..., 5] = 0, 0
            for b in range(n):
                kk, vv = np.concatenate([kf[seen], own[b][0]]), np.concatenate([vf[seen], own[b][1]])
                vv[..., 6] = 0
                if not masked:
                    vv[..., 5] = 0
                _check_cross(got[b][None], _f64(q[b]).reshape(1, nq, d), kk, vv, 2.0 ** -16 + 2.0 ** -18)


@pytest.mark.parametrize("far", [False, True])
def test_attention_decode_shared_of_groups_that_run_back(far):
    """Offsets of groups that overlap: reported, nothing written outside, and the workspace is fit for the next call (its arrival
    counters are zero again: every CTA has seen the same lengths).  Then one group of very many, and empty groups."""
    g = _gen(19)
    n, nq, nkv, d, page, P = 300, 4, 2, 64, 16, 64
    cache = _pool(g, 6 * 4 + n * 2, nkv, page, d, BF16)
    ids = torch.randperm(6 * 4 + n * 2, device="cuda", generator=g).to(torch.int32)
    far_cols = _far_bound(n, nkv, d, BF16) // page + 1 if far else 0
    ptable = torch.cat([ids[:24].view(6, 4), ids.new_full((6, far_cols), -1)], 1).contiguous()
    table, plens, lens = ids[24:].view(n, 2).contiguous(), [64, 1, 33, 0, 50, 17], [b % 30 for b in range(n)]

    def tokens(ls):
        return [torch.randn(x, nkv, d, device="cuda", generator=g) for x in ls], [torch.randn(x, nkv, d, device="cuda", generator=g) for x in ls]

    pre, own = _fill(cache, ptable, plens, *tokens(plens)), _fill(cache, table, lens, *tokens(lens))
    q, o = _randn(g, n, nq * d), torch.full((n + 2, nq * d), 7.0, device="cuda", dtype=torch.bfloat16)
    ws = torch.zeros(Q.h3enc_op_attention_decode_shared_workspace_bytes(n, nq, 32), dtype=torch.uint8, device="cuda")

    def run(rows):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Q.h3enc_op_attention_decode_shared(q, o[:n], cache, ptable, _i32(plens), P + page * far_cols, table, _i32(lens), nq, 32, ws,
                                           prefix_rows=_i32(rows), status=status)
        assert (o[n:] == 7).all() and not ws[:3 * 1024 * 4].any()
        return int(status.item())

    for rows in ([0, 300, 0, 300, 0, 300, 0], [300, 250, 200, 150, 100, 50, 0], [0, 200, 100, 250, 150, 300, 300],
                 [-5, 100, 2 ** 31 - 1, -(2 ** 31), 7, 250, 400]):
        assert run(rows) == 2
    for rows in ([0, 300, 300, 300, 300, 300, 300], [0, 0, 0, 299, 299, 299, 300], [3, 50, 100, 150, 200, 250, 290]):
        assert run(rows) == 0
        for b in [0, 2, 3, 49, 50, 151, 249, 250, 289, 290, 298, 299]:
            at = [i for i in range(6) if rows[i] <= b < rows[i + 1]]
            pk, pv = pre[at[0]] if at else (pre[0][0][:0], pre[0][1][:0])
            want, _ = O.decoder.attend_prefix(_f64(q[b]).reshape(nq, d), pk, pv, *own[b]) if len(pk) + lens[b] else (np.zeros((nq, d)), 0)
            # (|v| is at most 5 and each of the weights off by 2^-8 at most, and the output by half a step of values below 4)
            assert np.abs(_f64(o[b]).reshape(nq, d) - want).max() <= 5 * 2.0 ** -8 + 2.0 ** -7


@pytest.mark.parametrize("far", [False, True])
def test_attention_decode_shared_without_own_tokens_or_own_pages(far):
    """No own tokens at all: max_len 0 and a page table of no columns."""
    g = _gen(14)
    n, nq, nkv, d, page, P = 5, 4, 2, 64, 16, 50
    cache = _pool(g, 8, nkv, page, d, BF16)
    ptable = torch.full((1, 4 + (_far_bound(n, nkv, d, BF16) // page + 1 if far else 0)), -1, dtype=torch.int32, device="cuda")
    ptable[0, :4] = torch.randperm(8, device="cuda", generator=g)[:4].to(torch.int32)
    (k, v), = _fill(cache, ptable, [P], *([torch.randn(P, nkv, d, device="cuda", generator=g)] for _ in range(2)))
    q, o = _randn(g, n, nq * d), torch.zeros(n, nq * d, device="cuda", dtype=torch.bfloat16)
    ws = torch.zeros(Q.h3enc_op_attention_decode_shared_workspace_bytes(n, nq, 0), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Q.h3enc_op_attention_decode_shared(q, o, cache, ptable, _i32([P]), page * ptable.shape[1], ptable.new_zeros(n, 0), _i32([0] * n), nq,
                                       0, ws, status=status)
    assert int(status.item()) == 0
    _check_cross(_f64(o).reshape(n, nq, d), _f64(q).reshape(n, nq, d), k, v)


def test_attention_calls_on_two_streams_with_workspaces_of_their_own():
    """Cross attention and attention behind a prefix at once: each as alone."""
    g = _gen(15)
    nq, nkv, d, page, n, P = 8, 2, 128, 64, 40, 9000
    cache = _pool(g, P // page + 1 + n, nkv, page, d, BF16)
    for t in cache.tensors[:2]:
        t.copy_(_randn(g, *t.shape))
    ids = torch.arange(P // page + 1 + n, device="cuda", dtype=torch.int32)
    ptable, table = ids[:P // page + 1].view(1, -1), ids[P // page + 1:].view(n, 1)
    q1, q2, kv = _randn(g, n, nq * d), _randn(g, 900, nq * d), _randn(g, 1500, 2 * nkv * d)
    lens, outs = _i32([1 + i for i in range(n)]), []
    for _ in range(2):
        o1, o2 = torch.zeros_like(q1), torch.zeros_like(q2)
        ws1 = torch.zeros(Q.h3enc_op_attention_decode_shared_workspace_bytes(n, nq, page), dtype=torch.uint8, device="cuda")
        ws2 = _cross_ws(d)
        outs.append((o1, o2, ws1, ws2))
    plen = _i32([P])

    def shared(o, ws):
        Q.h3enc_op_attention_decode_shared(q1, o, cache, ptable, plen, page * ptable.shape[1], table, lens, nq, page, ws)

    def cross(o, ws):
        Q.h3enc_op_attention_cross(q2, kv[:, :nkv * d], kv[:, nkv * d:], o, nq, nkv, d, ws)

    shared(outs[0][0], outs[0][2])
    cross(outs[0][1], outs[0][3])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        with torch.cuda.stream(streams[0]):
            shared(outs[1][0], outs[1][2])
        with torch.cuda.stream(streams[1]):
            cross(outs[1][1], outs[1][3])
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ---------------------------------------------------------------- a run of them together

@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_decode_steps_of_a_decoder_that_reads_an_encoder(dtype):
    """Three steps of one captured graph: append (rotated by place), self attention behind a shared prompt, cross attention to the
    states of each sequence's own prompt.  The oracle follows the bf16 tensors between the calls."""
    g = _gen(13)
    n, nq, nkv, d, page, P = 6, 8, 2, 64, 16, 200
    plens, start = [P, 77], [0, 3, 15, 16, 40, 1]
    cache = _pool(g, 2 * 13 + n * 4, nkv, page, d, dtype)
    ids = torch.randperm(2 * 13 + n * 4, device="cuda", generator=g).to(torch.int32)
    ptable, table = ids[:26].view(2, 13).contiguous(), ids[26:].view(n, 4).contiguous()
    rnd = lambda ls: [torch.randn(x, nkv, d, device="cuda", generator=g) for x in ls]   # noqa: E731
    pre, own = _fill(cache, ptable, plens, rnd(plens), rnd(plens)), _fill(cache, table, start, rnd(start), rnd(start))
    klens = [1, 130, 77, 512, 0, 300]
    states = _randn(g, sum(klens), 2 * nkv * d)
    cu_k = np.concatenate([[0], np.cumsum(klens)])
    rope_args, rope = _rope("yarn", d)
    qkv, lens = torch.zeros(n, (nq + 2 * nkv) * d, device="cuda", dtype=torch.bfloat16), _i32(start)
    o1, o2 = (torch.zeros(n, nq * d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    rows, places = _i32([0, 4, 6]), torch.zeros(1, n, dtype=torch.int32, device="cuda")
    ws = torch.zeros(Q.h3enc_op_attention_decode_shared_workspace_bytes(n, nq, 64), dtype=torch.uint8, device="cuda")
    ws2, cuq, cuk = _cross_ws(d), _i32(list(range(n + 1))), _i32(cu_k)
    behind = _i32([P] * 4 + [77] * 2)
    plen_t, status = _i32(plens), torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        lens.add_(1)
        places[0].copy_(lens + behind - 1)         # a token's position counts its prefix
        Q.h3enc_op_rope_append(qkv, n, nq, nkv, d, None, None, 0.0, rope, places[0], qkv[:, :nq * d], cache=cache, page_table=table,
                               seq_lens=lens, max_len=64, status=status)
        Q.h3enc_op_attention_decode_shared(qkv[:, :nq * d], o1, cache, ptable, plen_t, P, table, lens, nq, 64, ws, prefix_rows=rows,
                                           status=status)
        Q.h3enc_op_attention_cross(o1, states[:, :nkv * d], states[:, nkv * d:], o2, nq, nkv, d, ws2, cuq, cuk, status)

    step()                                         # (warm-up outside the capture; undone)
    lens.copy_(_i32(start))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens.copy_(_i32(start))
    w, magnitude = O.decoder.frequencies(**{k: x for k, x in rope_args.items()})
    sf = _f64(states).reshape(-1, 2, nkv, d)
    p_err = 2.0 ** -8 if dtype == BF16 else 2.0 ** -11
    for i in range(3):
        rowsin = _randn(g, n, (nq + 2 * nkv) * d)
        qkv.copy_(rowsin)
        graph.replay()
        x = _f64(rowsin).reshape(n, nq + 2 * nkv, d)
        kp, vp, ks, vs = cache.tensors
        for b in range(n):
            at = start[b] + i
            angle = ((plens[0 if b < 4 else 1] + at) * w)[None]
            want_q = O.decoder.rotate(x[b:b + 1, :nq], angle, magnitude, False)[0]
            q = _f64(qkv[b, :nq * d]).reshape(nq, d)
            _check_bf16(q, want_q, 2.0 ** -19 * _pair_length(want_q, d, False))
            new = [_f64(_raw(t)[table[b, at // page].long(), :, at % page].view(t.dtype)) * (1 if sc is None else _f64(sc)[:, None])
                   for t, sc in ((kp, ks), (vp, vs))]
            want_k = O.decoder.rotate(x[b:b + 1, nq:nq + nkv], angle, magnitude, False)[0]
            step_size = 2.0 ** -8 * np.abs(want_k) if dtype == BF16 else 2.0 ** -4 * np.abs(want_k) + 2.0 ** -10 * _f64(ks)[:, None]
            assert (np.abs(new[0] - want_k) <= step_size * (1 + 2.0 ** -10) + 2.0 ** -19 * _pair_length(want_k, d, False)).all()
            own[b] = [np.concatenate([old, y[None]]) for old, y in zip(own[b], new)]
            pk, pv = pre[0 if b < 4 else 1]
            want, _ = O.decoder.attend_prefix(q, pk, pv, *own[b])
            A = O.decoder.attend_prefix(q, pk, np.abs(pv), own[b][0], np.abs(own[b][1]))[0]
            delta = 16 * 2.0 ** -24 * _score_bound(q[None], np.concatenate([pk, own[b][0]]))
            got = _f64(o1[b]).reshape(nq, d)
            _check_bf16(got, want, A * (2 * delta + p_err + 2.0 ** -15))
            s = sf[cu_k[b]:cu_k[b + 1]]
            _check_cross(_f64(o2[b:b + 1]).reshape(1, nq, d), got[None], s[:, 0], s[:, 1])
    assert int(status.item()) == 0
