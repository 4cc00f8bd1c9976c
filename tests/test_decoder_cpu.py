"""A decoder that reads an encoder's states, without a GPU: the oracle against hand-made cases, and every
refusal of the entry points before they touch CUDA."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest

import oracle as O


@pytest.fixture(scope="module")
def Q():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import qwen3_vl_text_gb300
    return qwen3_vl_text_gb300


# ---------------------------------------------------------------- oracle pins

def test_frequencies_by_hand():
    w, m = O.decoder.frequencies(8, 16.0)
    assert np.allclose(w, [1, 0.5, 0.25, 0.125]) and m == 1
    assert np.allclose(O.decoder.frequencies(8, 16.0, "linear", 4.0)[0], w / 4)
    # 64 tokens: 10.2, 5.1, 2.5 and 1.3 turns; kept from 5, stretched whole below 2
    s = (32 * 0.25 / math.pi - 2) / 3
    got, m = O.decoder.frequencies(8, 16.0, "wavelength", 8.0, 64, 2.0, 5.0)
    assert np.allclose(got, [1, 0.5, 0.25 * (s + (1 - s) / 8), 0.125 / 8]) and m == 1
    # pair j turns 10.2 / 2^j times: 8 and 2 turns lie at j = 0.35 and 2.35, so the ramp runs from 0 to 3
    got, m = O.decoder.frequencies(8, 16.0, "yarn", 8.0, 64, 2.0, 8.0)
    assert np.allclose(got, [1, 0.5 * (2 / 3 + 1 / 24), 0.25 * (1 / 3 + 1 / 12), 0.125 / 8])
    assert m == pytest.approx(0.1 * math.log(8) + 1)
    assert O.decoder.frequencies(8, 16.0, "yarn", 8.0, 64, magnitude=1.0)[1] == 1


def test_axes_are_those_of_the_prefill_tables():
    section = (24, 20, 20)
    axes = [O.decoder.axis_of(j, section) for j in range(64)]
    assert axes == [0, 1, 2] * 20 + [0] * 4


def test_rotate_by_hand():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = np.full((1, 2), math.pi / 2)
    assert np.allclose(O.decoder.rotate(x, quarter, 1.0, False), [[[-3, -4, 1, 2, 5, 6, 7, 8]]])
    assert np.allclose(O.decoder.rotate(x, quarter, 2.0, True), [[[-4, 2, -8, 6, 5, 6, 7, 8]]])


def test_append_places_by_hand():
    assert O.decoder.append_places(6, [4, 9, 7], [0, 2, 2, 5]) == [(0, 2), (0, 3), (2, 4), (2, 5), (2, 6), None]
    assert O.decoder.append_places(3, [4, 1], None) == [(0, 3), (1, 0), None]


# ---------------------------------------------------------------- refusals

def _cache(Q, **kw):
    c = Q.KVCache.__new__(Q.KVCache)
    base = dict(k=4096, v=8192, k_scale=None, v_scale=None, page_stride=2 * 16 * 64, num_pages=4, page_size=16,
                n_kv_heads=2, head_dim=64, dtype=0)
    base.update(kw)
    for name, value in base.items():
        setattr(c, name, value)
    return c


BAD_CACHES = [(dict(k=None), 2), (dict(v=8), 2), (dict(dtype=1), 6), (dict(head_dim=96), 6), (dict(page_size=8), 6),
              (dict(page_size=48), 6), (dict(page_stride=2 * 16 * 64 - 8), 2), (dict(page_stride=2 * 16 * 64 + 4), 2),
              (dict(num_pages=0), 2), (dict(n_kv_heads=0), 2), (dict(dtype=2), 2), (dict(k_scale=64), 2)]


def _append(Q, cache=None, rope=None, **kw):
    a = dict(qkv=1 << 20, ld_qkv=512, T=3, nq=4, nkv=2, d=64, wq=16, wk=16, eps=1e-6, pos=None, ld_pos=3, q=1 << 24,
             ld_q=256, k=None, ld_k=128, table=16, ld_table=4, lens=16, cu=16, n=2, max_len=64)
    if cache is None:
        a.update(table=None, ld_table=0)
    a.update(kw)
    Q._check(Q.lib.h3enc_op_rope_append(
        a["qkv"], a["ld_qkv"], a["T"], a["nq"], a["nkv"], a["d"], a["wq"], a["wk"], a["eps"], rope, a["pos"], a["ld_pos"],
        a["q"], a["ld_q"], a["k"], a["ld_k"], cache, a["table"], a["ld_table"], a["lens"], a["cu"], a["n"], a["max_len"],
        None, None))


def _refused(Q, code, call, *args, **kw):
    with pytest.raises(Q.H3encError) as e:
        call(Q, *args, **kw)
    assert e.value.code == code, str(e.value)
    assert Q.h3enc_last_error(None)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused(Q, kw, code):
    _refused(Q, code, _append, _cache(Q, **kw))


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(nq=0), dict(nkv=0), dict(d=96), dict(qkv=None), dict(qkv=(1 << 20) + 8), dict(ld_qkv=511),
    dict(ld_qkv=508), dict(ld_qkv=516), dict(eps=-1.0), dict(wq=8), dict(q=None), dict(q=(1 << 24) + 2), dict(ld_q=252),
    dict(k=1 << 25, ld_k=64), dict(q=(1 << 20) + 16), dict(q=1 << 20, ld_q=520), dict(k=1 << 24, ld_k=128),
    dict(n=-1), dict(n=1025), dict(max_len=-1), dict(max_len=2 ** 30 + 1), dict(table=16), dict(lens=None),
    dict(lens=None, cu=None), dict(lens=None, n=0), dict(n=0), dict(pos=16, ld_pos=2)])
def test_rope_append_refuses(Q, kw):
    _refused(Q, 2, _append, **kw)


@pytest.mark.parametrize("kw", [dict(table=None), dict(ld_table=3), dict(ld_table=-1), dict(max_len=65), dict(nkv=1, ld_qkv=384),
                                dict(d=128, ld_qkv=1024, ld_q=512), dict(lens=None), dict(lens=None, n=0, cu=None)])
def test_rope_append_to_a_cache_refuses(Q, kw):
    _refused(Q, 2, _append, _cache(Q), **kw)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=40), dict(rotary_dim=144), dict(rotary_dim=-16), dict(theta=0.0),
    dict(theta=-2.0), dict(theta=math.inf), dict(theta=math.nan), dict(factor=0.0, scaling="linear"),
    dict(factor=math.nan, scaling="linear"), dict(magnitude=-1.0), dict(magnitude=math.nan), dict(magnitude=math.inf),
    dict(scaling="yarn", factor=4.0), dict(scaling="wavelength", factor=4.0, original_len=0),
    dict(scaling="yarn", factor=4.0, original_len=64, theta=1.0), dict(scaling="yarn", factor=4.0, original_len=64, theta=0.5),
    dict(scaling="wavelength", factor=4.0, original_len=64, low_turns=4.0, high_turns=4.0),
    dict(scaling="yarn", factor=4.0, original_len=64, low_turns=1.0), dict(section=(8, 8, 8)), dict(section=(40, -4, -4)),
    dict(section=(0, 0, 31)), dict(theta=1e-320)])
def test_rope_refuses_parameters(Q, kw):
    with pytest.raises(Q.H3encError) as e:
        Q.Rope(**{**dict(rotary_dim=64, theta=1e4), **kw})
    assert e.value.code == 2 and Q.h3enc_last_error(None)


def test_rope_plans(Q):
    """The frequencies of a plan are the oracle's, in turns; parameters and plans that are none are refused."""
    for kw in (dict(), dict(interleaved=True), dict(scaling="linear", factor=4.0), dict(scaling="wavelength", factor=8.0, original_len=8192),
               dict(scaling="yarn", factor=4.0, original_len=32768), dict(theta=0.5)):
        kw = {**dict(theta=5e5), **kw}
        plan = Q.Rope(96, **kw)
        kw.pop("interleaved", None)
        w, m = O.decoder.frequencies(96, **kw)
        turns = np.array(plan.turns[:48], np.float64) / 2.0 ** 64
        assert np.allclose(turns, w / (2 * math.pi) % 1, rtol=2.0 ** -50, atol=2.0 ** -52) and plan.magnitude == pytest.approx(m, rel=1e-7)
        assert (plan.rotary_dim, plan.axes, plan.axis1, plan.axis2) == (96, 1, 0, 0)
    plan = Q.Rope(128, 5e6, section=(24, 20, 20))
    assert plan.axes == 3 and [(plan.axis1 >> j & 1) + 2 * (plan.axis2 >> j & 1) for j in range(64)] == [O.decoder.axis_of(j, (24, 20, 20)) for j in range(64)]
    for scaling in (-1, 4):
        params = Q._RopeParams(64, 0, scaling, 0, 1e4, 1.0)
        with pytest.raises(Q.H3encError):
            Q.h3enc_rope_make(params, plan)
    for args in ((None, plan), (Q._RopeParams(64, 0, 0, 0, 1e4), None)):
        with pytest.raises(Q.H3encError):
            Q.h3enc_rope_make(*args)
    with pytest.raises(ValueError):
        Q.Rope(64, 1e4, scaling="ntk")
    with pytest.raises(ValueError):
        Q.Rope(64, 1e4, section=(16, 16))
    with pytest.raises(ValueError):
        Q.Rope(2 ** 32 + 64, 1e4)


def test_rope_append_refuses_plans(Q):
    _refused(Q, 2, _append, rope=Q.Rope(80, 1e4))          # more than a head
    for field, value in (("rotary_dim", 0), ("rotary_dim", 24), ("axes", 2), ("axes", 0)):
        r = Q.Rope(64, 1e4)
        setattr(r, field, value)
        _refused(Q, 2, _append, rope=r)
    r = Q.Rope(64, 1e4)
    r.axis1 = r.axis2 = 1
    _refused(Q, 2, _append, rope=r)


def test_rope_append_needs_positions_without_lengths(Q):
    _refused(Q, 2, _append, rope=Q.Rope(64, 1e4), lens=None, cu=None, n=0)


def test_rope_append_of_no_rows_does_nothing(Q):
    _append(Q, T=0)
    _append(Q, _cache(Q), Q.Rope(32, 1e4), T=0, n=0)
    _append(Q, T=0, q=1 << 20, ld_q=512, k=(1 << 20) + 512, ld_k=512)     # in place


# ---------------------------------------------------------------- what the Python calls check of their tensors

class _Record:
    """Stands in for the library: keeps a call's arguments and succeeds."""
    def __getattr__(self, name):
        def call(*args):
            self.args = args
            return 0
        return call


@pytest.fixture
def recorded(Q, monkeypatch):
    rec = _Record()
    monkeypatch.setattr(Q, "lib", rec)
    monkeypatch.setattr(Q, "_raw", (lambda: -1, lambda d: 77))     # the "device" of CPU tensors
    return rec


def _refuses(Q, call, args, name, tensor):
    with pytest.raises(Q.H3encError) as e:
        call(**{**args, name: tensor})
    assert e.value.code == 2 and name in str(e.value), str(e.value)


def _wrong(torch, t, rows):
    """Tensors that may not stand where t does: another type, fewer rows, rows that are too narrow, gaps."""
    out = [t.double() if t.dtype == torch.float32 else t.float(), t[:0] if rows else t[..., :0]]
    if t.dim() == 2:
        out += [t[:, :-1], torch.cat([t, t], 1)[:, ::2]]
    return out


@pytest.fixture
def plans(Q):
    return Q.Rope(64, 1e4, section=(12, 10, 10)), Q.Rope(64, 1e4)


def test_rope_append_checks_its_tensors(Q, plans, recorded):
    torch = pytest.importorskip("torch")
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    k = torch.zeros(5, 2, 16, 64, **bf)
    a = dict(qkv=torch.zeros(6, 512, **bf), T=6, n_heads=4, n_kv_heads=2, head_dim=64, w_q=torch.ones(64, **bf),
             w_k=torch.ones(64, **bf), eps=1e-6, rope=plans[0], positions=torch.zeros(3, 6, **i32),
             q_out=torch.zeros(6, 256, **bf), k_out=torch.zeros(6, 128, **bf), cache=Q.KVCache(k, k),
             page_table=torch.zeros(3, 4, **i32), seq_lens=torch.zeros(3, **i32), max_len=64, cu_rows=torch.zeros(4, **i32),
             status=torch.zeros(1, **i32))
    Q.h3enc_op_rope_append(**a)
    got = recorded.args
    assert got[:6] == (a["qkv"].data_ptr(), 512, 6, 4, 2, 64) and got[9].axes == 3 and got[11] == 6 and got[-1] == 77
    assert got[17:23] == (a["page_table"].data_ptr(), 4, a["seq_lens"].data_ptr(), a["cu_rows"].data_ptr(), 3, 64)
    for name in ("qkv", "w_q", "w_k", "positions", "q_out", "k_out", "page_table", "cu_rows", "status"):
        for bad in _wrong(torch, a[name], True):
            _refuses(Q, Q.h3enc_op_rope_append, a, name, bad)
    _refuses(Q, Q.h3enc_op_rope_append, a, "seq_lens", torch.zeros(3))
    _refuses(Q, Q.h3enc_op_rope_append, a, "positions", torch.zeros(6, **i32))     # three axes wanted
    _refuses(Q, Q.h3enc_op_rope_append, a, "page_table", torch.zeros(2, 4, **i32))
    a["rope"] = plans[1]
    a["positions"] = torch.zeros(6, **i32)
    Q.h3enc_op_rope_append(**a)
    a.update(rope=None, positions=None, cache=None, page_table=None, seq_lens=None, cu_rows=None, max_len=0, status=None)
    Q.h3enc_op_rope_append(**a)
    assert recorded.args[9:12] == (None, None, 0) and recorded.args[16:23] == (None, None, 0, None, None, 0, 0)


# ---------------------------------------------------------------- shared prefixes and cross attention: refusals

def test_attend_prefix_and_cross_by_hand():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((5, 6, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    o = O.decoder.cross(q, k, v)
    for t in range(5):
        one, p = O.decode.attend_one(q[t], k, v)
        assert np.allclose(o[t], one, rtol=1e-12, atol=1e-14)
        both, own = O.decoder.attend_prefix(q[t], k[:4], v[:4], k[4:], v[4:])
        assert np.allclose(both, one) and np.allclose(own, p[:, 4:])
    assert not O.decoder.cross(q, k[:0], v[:0]).any()


def _shared(Q, cache, **kw):
    a = dict(q=1 << 20, ld_q=256, o=1 << 24, ld_o=256, ptable=16, ld_p=4, plens=16, prows=16, groups=2, max_prefix=64,
             table=16, ld_table=4, lens=16, n=2, nq=4, max_len=64, w_in=None, w_out=None, ld_w=64, ws=256, ws_bytes=1 << 40)
    a.update(kw)
    Q._check(Q.lib.h3enc_op_attention_decode_shared(
        a["q"], a["ld_q"], a["o"], a["ld_o"], cache, a["ptable"], a["ld_p"], a["plens"], a["prows"], a["groups"],
        a["max_prefix"], a["table"], a["ld_table"], a["lens"], a["n"], a["nq"], a["max_len"], a["w_in"], a["w_out"],
        a["ld_w"], a["ws"], a["ws_bytes"], None, None))


def _cross(Q, **kw):
    a = dict(q=1 << 20, ld_q=256, k=1 << 22, ld_k=256, v=(1 << 22) + 256, ld_v=256, o=1 << 24, ld_o=256, Tq=5, Tk=7, nq=4, nkv=2,
             d=64, cu_q=16, cu_k=16, n=2, ws=256, ws_bytes=1 << 40)
    a.update(kw)
    Q._check(Q.lib.h3enc_op_attention_cross(
        a["q"], a["ld_q"], a["k"], a["ld_k"], a["v"], a["ld_v"], a["o"], a["ld_o"], a["Tq"], a["Tk"], a["nq"], a["nkv"],
        a["d"], a["cu_q"], a["cu_k"], a["n"], a["ws"], a["ws_bytes"], None, None))


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused_behind_prefixes(Q, kw, code):
    _refused(Q, code, _shared, _cache(Q, **kw))


@pytest.mark.parametrize("kw", [
    dict(groups=-1), dict(groups=1025), dict(max_prefix=-1), dict(max_prefix=65), dict(max_prefix=2 ** 30 + 1, ld_p=2 ** 27),
    dict(ld_p=-1), dict(ld_p=3), dict(prows=None), dict(plens=None), dict(ptable=None), dict(ld_q=1 << 39),
    dict(n=-1), dict(n=1025), dict(nq=0), dict(nq=3), dict(max_len=-1), dict(max_len=65), dict(q=None), dict(o=None),
    dict(q=(1 << 20) + 8), dict(ld_q=252), dict(ld_o=128), dict(table=None), dict(lens=None), dict(o=1 << 20), dict(w_in=16),
    dict(w_out=16, ld_w=63)])
def test_attention_decode_shared_refuses(Q, kw):
    _refused(Q, 2, _shared, _cache(Q), **kw)


def test_attention_decode_shared_of_no_sequences_does_nothing(Q):
    _shared(Q, _cache(Q), n=0)
    _shared(Q, _cache(Q), n=0, groups=0, prows=None, plens=None, ptable=None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), 6), (dict(Tq=-1), 2), (dict(Tk=-1), 2), (dict(Tq=2 ** 30 + 1), 2), (dict(nq=0), 2), (dict(nq=5), 2),
    (dict(nkv=0), 2), (dict(nq=65538), 2), (dict(n=-1), 2), (dict(n=1025), 2), (dict(cu_q=None), 2), (dict(cu_k=None), 2),
    (dict(q=None), 2), (dict(k=None), 2), (dict(v=None), 2), (dict(o=None), 2), (dict(q=(1 << 20) + 2), 2), (dict(k=(1 << 22) + 2), 2),
    (dict(v=(1 << 22) + 8), 2), (dict(o=(1 << 24) + 8), 2), (dict(ld_q=248), 2), (dict(ld_q=260), 2), (dict(ld_k=120), 2),
    (dict(ld_v=132), 2), (dict(ld_o=252), 2), (dict(ld_k=1 << 39), 2), (dict(ld_q=1 << 39), 2), (dict(o=1 << 20), 2),
    (dict(o=(1 << 20) + 512 * 4), 2), (dict(o=1 << 22), 2), (dict(o=(1 << 22) + 256), 2),
    (dict(Tq=2 ** 26, Tk=2 ** 26, q=0, o=1 << 50, k=1 << 55, v=1 << 56), 2), (dict(Tq=2 ** 26, Tk=2 ** 26, o=1 << 50, k=1 << 55, v=1 << 56), 6)])
def test_attention_cross_refuses(Q, kw, code):
    _refused(Q, code, _cross, **kw)


def test_attention_cross_takes_states_right_behind_its_output(Q):
    """o's own rows end where k begins, however many rows k has (refused for its workspace, after that check)."""
    with pytest.raises(Q.H3encError) as e:
        _cross(Q, o=1 << 24, k=(1 << 24) + 5 * 512, v=(1 << 24) + 5 * 512 + 256, Tk=700, ws=None)
    assert "overlap" not in str(e.value)


def test_attention_cross_of_nothing_does_nothing(Q):
    _cross(Q, Tq=0)
    _cross(Q, n=0)


def test_workspace_sizes_without_a_gpu_or_for_refused_sizes(Q):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        assert Q.h3enc_op_attention_decode_shared_workspace_bytes(1, 8, 100) == -1
        assert Q.h3enc_op_attention_cross_workspace_bytes(128) == -1
    assert Q.h3enc_op_attention_cross_workspace_bytes(96) == -1
    for bad in ((-1, 8, 100), (1025, 8, 100), (1, 0, 100), (1, 8, -1)):
        assert Q.h3enc_op_attention_decode_shared_workspace_bytes(*bad) == -1


def test_attention_decode_shared_checks_its_tensors(Q, recorded):
    torch = pytest.importorskip("torch")
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    k = torch.zeros(5, 2, 16, 64, **bf)
    a = dict(q=torch.zeros(3, 256, **bf), o=torch.zeros(3, 256, **bf), cache=Q.KVCache(k, k),
             prefix_table=torch.zeros(2, 5, **i32), prefix_lens=torch.zeros(2, **i32), max_prefix=80,
             page_table=torch.zeros(3, 4, **i32), seq_lens=torch.zeros(3, **i32), n_heads=4, max_len=64,
             workspace=torch.zeros(64, dtype=torch.uint8), prefix_rows=torch.zeros(3, **i32),
             weight_in=torch.zeros(3, 64), weight_out=torch.zeros(3, 64), status=torch.zeros(1, **i32))
    Q.h3enc_op_attention_decode_shared(**a)
    got = recorded.args
    assert got[5:11] == (a["prefix_table"].data_ptr(), 5, a["prefix_lens"].data_ptr(), a["prefix_rows"].data_ptr(), 2, 80)
    assert got[11:17] == (a["page_table"].data_ptr(), 4, a["seq_lens"].data_ptr(), 3, 4, 64) and got[21] == 64
    for name in ("q", "o", "prefix_table", "prefix_rows", "page_table", "weight_in", "weight_out", "status"):
        for bad in _wrong(torch, a[name], True):
            _refuses(Q, Q.h3enc_op_attention_decode_shared, a, name, bad)
    for name in ("prefix_lens", "seq_lens"):
        _refuses(Q, Q.h3enc_op_attention_decode_shared, a, name, a[name].float())
    _refuses(Q, Q.h3enc_op_attention_decode_shared, a, "workspace", torch.zeros(64, dtype=torch.uint8)[::2])


def test_attention_cross_checks_its_tensors(Q, recorded):
    torch = pytest.importorskip("torch")
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    kv = torch.zeros(9, 256, **bf)
    a = dict(q=torch.zeros(6, 256, **bf), k=kv[:, :128], v=kv[:, 128:], o=torch.zeros(6, 256, **bf), n_heads=4, n_kv_heads=2,
             head_dim=64, workspace=torch.zeros(64, dtype=torch.uint8), cu_q=torch.zeros(4, **i32), cu_k=torch.zeros(4, **i32),
             status=torch.zeros(1, **i32))
    Q.h3enc_op_attention_cross(**a)
    got = recorded.args
    assert got[1] == 256 and got[2:6] == (kv.data_ptr(), 256, kv.data_ptr() + 256, 256)
    assert got[8:16] == (6, 9, 4, 2, 64, a["cu_q"].data_ptr(), a["cu_k"].data_ptr(), 3)
    for name in ("q", "k", "v", "o"):
        for bad in (a[name].float(), a[name][:, :-1], torch.cat([a[name], a[name]], 1)[:, ::2]):
            _refuses(Q, Q.h3enc_op_attention_cross, a, name, bad)
    for name, bad in (("v", kv[:8, 128:]), ("o", a["o"][:5]), ("cu_k", torch.zeros(3, **i32)), ("cu_q", torch.zeros(4)),
                      ("cu_q", torch.zeros(0, **i32)), ("status", torch.zeros(1)), ("workspace", torch.zeros(64)[::2])):
        _refuses(Q, Q.h3enc_op_attention_cross, a, name, bad)
    a.update(cu_q=None, cu_k=None)
    Q.h3enc_op_attention_cross(**a)
    assert recorded.args[13:16] == (None, None, 1)


# ---------------------------------------------------------------- sound calls without a device

_WITHOUT_DEVICE = """
import sys
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import qwen3_vl_text_gb300 as Q
import test_decoder_cpu as T
for call in (lambda: T._append(Q), lambda: T._append(Q, T._cache(Q), Q.Rope(64, 1e4)), lambda: T._shared(Q, T._cache(Q)), lambda: T._cross(Q)):
    try:
        call()
    except Q.H3encError as e:
        assert e.code == 7, e
    else:
        raise AssertionError("no error")
print("all refused")
"""


def test_sound_calls_without_a_device_are_errors(Q):
    """In a process of its own, which sees no device wherever it runs: a division by its 0 SMs would end it."""
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", _WITHOUT_DEVICE.format(root=os.path.dirname(tests), tests=tests)], capture_output=True,
                       text=True, timeout=300, env={**os.environ, "CUDA_VISIBLE_DEVICES": "-1"})
    assert r.returncode == 0 and "all refused" in r.stdout, (r.returncode, r.stdout, r.stderr)
