"""A decoder that reads an encoder's states: rows rotated and appended to a paged cache, attention of one new token
behind shared prefixes, and cross attention, against the float64 oracle; their edges (empty and ragged
sequences, pages that end inside a tile, stale NaN behind a sequence, bad pages and lengths), graphs and streams, and
a run of them together.

Tolerances.  A bf16 output is rounded once: half a step, 2^-8 of the value, plus the fp32 noise of its terms.
Rotation: the angle is a 64-bit fraction of a turn, so cos and sin are off by less than 2^-21 of the magnitude (fp32
rounding of the fraction and of sincospi), and the norm's factor by 2^-21: at most 2^-19 of a pair's length.
An e4m3 value is off by half a step: 2^-4 of the value, 2^-10 at least.
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
