"""Decoding from a paged key/value cache without a GPU: the oracle against the prefill oracle and
hand-made cases, and every refusal of the three entry points before they touch CUDA."""
import ctypes

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

def test_attend_one_is_the_last_row_of_causal_attention():
    rng = np.random.default_rng(0)
    S, nq, nkv, d = 13, 6, 2, 8
    q, k, v = rng.standard_normal((S, nq, d)), rng.standard_normal((S, nkv, d)), rng.standard_normal((S, nkv, d))
    for n in (1, 2, 13):
        o, p = O.decode.attend_one(q[n - 1], k[:n], v[:n])
        for h in range(nq):       # brute force, key by key
            s = [float(np.dot(q[n - 1, h], k[i, h // 3])) / d ** 0.5 for i in range(n)]
            z = sum(np.exp(x - max(s)) for x in s)
            want = sum(np.exp(x - max(s)) / z * v[i, h // 3] for i, x in enumerate(s))
            assert np.allclose(o[h], want, rtol=1e-12, atol=1e-14)
        assert np.allclose(p.sum(1), 1)
    assert not O.decode.attend_one(q[0], k[:0], v[:0])[0].any()


def test_head_norm_rope_is_a_rotation_of_a_unit_rms_vector():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 8)) * 5
    ang = rng.uniform(0, 6, (3, 4))
    y = O.decode.head_norm_rope(x, np.ones(8), 0.0, np.cos(ang), np.sin(ang))
    z = (y[..., :4] + 1j * y[..., 4:]) / ((x[..., :4] + 1j * x[..., 4:]) / np.sqrt((x * x).mean(-1, keepdims=True)))
    assert np.allclose(z, np.exp(1j * ang)[:, None], rtol=1e-12)
    assert np.array_equal(O.decode.head_norm_rope(x, None, 0.0, None, None), x)


def test_keep_heaviest_by_hand():
    nan = float("nan")
    w = [0.0, 5.0, 1.0, 3.0, 3.0, nan, 3.0, 0.5]
    assert O.decode.keep_heaviest(w, 8, 8, 1, 1) == list(range(8))
    assert O.decode.keep_heaviest(w, 8, 5, 1, 1) == [0, 1, 3, 4, 7]        # of three equal ones the earlier
    assert O.decode.keep_heaviest(w, 8, 2, 1, 1) == [0, 7]
    assert O.decode.keep_heaviest([-1.0, nan, -np.inf, -2.0], 4, 3, 0, 0) == [0, 2, 3]
    assert O.decode.keep_heaviest([0.0, -0.0, 0.0], 3, 2, 0, 0) == [0, 1]


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
              (dict(page_size=48), 6), (dict(page_size=512), 6), (dict(page_stride=2 * 16 * 64 - 8), 2),
              (dict(page_stride=2 * 16 * 64 + 4), 2), (dict(page_stride=1 << 40), 2), (dict(num_pages=0), 2),
              (dict(num_pages=1 << 28), 2), (dict(n_kv_heads=0), 2), (dict(n_kv_heads=65537, page_stride=65537 * 16 * 64), 2), (dict(dtype=2), 2),
              (dict(dtype=2, k_scale=64), 2), (dict(k_scale=64), 2), (dict(v_scale=64), 2)]


def _rope(Q, cache=None, **kw):
    a = dict(qkv=1 << 20, ld_qkv=512, T=3, nq=4, nkv=2, d=64, wq=16, wk=16, eps=1e-6, cos=16, sin=16, cs=0, q=1 << 24,
             ld_q=256, k=None, ld_k=128, slots=None)
    a.update(kw)
    Q._check(Q.lib.h3enc_op_qk_norm_rope(
        a["qkv"], a["ld_qkv"], a["T"], a["nq"], a["nkv"], a["d"], a["wq"], a["wk"], a["eps"], a["cos"], a["sin"],
        a["cs"], a["q"], a["ld_q"], a["k"], a["ld_k"], cache, a["slots"], None, None))


def _attend(Q, cache, **kw):
    a = dict(q=1 << 20, ld_q=256, o=1 << 24, ld_o=256, table=16, ld_table=4, lens=16, n=2, nq=4, max_len=64, w_in=None,
             w_out=None, ld_w=64, ws=256, ws_bytes=1 << 40)
    a.update(kw)
    Q._check(Q.lib.h3enc_op_attention_decode(
        a["q"], a["ld_q"], a["o"], a["ld_o"], cache, a["table"], a["ld_table"], a["lens"], a["n"], a["nq"],
        a["max_len"], a["w_in"], a["w_out"], a["ld_w"], a["ws"], a["ws_bytes"], None, None))


def _evict(Q, cache, **kw):
    a = dict(table=16, ld_table=4, table_out=None, ld_out=0, lens=16, n=2, max_len=64, budget=32, sink=4, recent=8,
             w=1 << 20, ld_w=64, w_out=1 << 24, ld_w_out=64, kept=16, ld_kept=32, new=16)
    a.update(kw)
    Q._check(Q.lib.h3enc_op_cache_evict(
        cache, a["table"], a["ld_table"], a["table_out"], a["ld_out"], a["lens"], a["n"], a["max_len"], a["budget"],
        a["sink"], a["recent"], a["w"], a["ld_w"], a["w_out"], a["ld_w_out"], a["kept"], a["ld_kept"], a["new"], None,
        None))


def _refused(Q, code, call, *args, **kw):
    with pytest.raises(Q.H3encError) as e:
        call(Q, *args, **kw)
    assert e.value.code == code, str(e.value)
    assert Q.h3enc_last_error(None)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused_by_every_entry(Q, kw, code):
    c = _cache(Q, **kw)
    _refused(Q, code, _rope, c, slots=16)
    _refused(Q, code, _attend, c)
    _refused(Q, code, _evict, c)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(nq=0), dict(nkv=0), dict(d=96), dict(qkv=None), dict(qkv=(1 << 20) + 8), dict(ld_qkv=511),
    dict(ld_qkv=508), dict(ld_qkv=516), dict(ld_qkv=1 << 62), dict(cos=None), dict(sin=None), dict(cos=20), dict(cs=2), dict(cs=-1),
    dict(eps=-1.0), dict(eps=float("nan")), dict(wq=8), dict(q=None), dict(q=(1 << 24) + 2), dict(ld_q=255),
    dict(ld_q=252), dict(k=1 << 25, ld_k=64), dict(q=(1 << 20) + 16),                # overlaps qkv, not in place
    dict(q=1 << 20, ld_q=520), dict(k=1 << 20, ld_k=512), dict(k=1 << 24, ld_k=128), dict(slots=16)])
def test_qk_norm_rope_refuses(Q, kw):
    _refused(Q, 2, _rope, **kw)


def test_qk_norm_rope_refuses_a_cache_of_other_heads_or_without_slots(Q):
    _refused(Q, 2, _rope, _cache(Q))
    _refused(Q, 2, _rope, _cache(Q, n_kv_heads=1, page_stride=4096), slots=16)
    _refused(Q, 2, _rope, _cache(Q, head_dim=128, page_stride=2 * 16 * 128), slots=16)


def test_qk_norm_rope_of_no_rows_does_nothing(Q):
    _rope(Q, T=0)
    _rope(Q, T=0, q=1 << 20, ld_q=512, k=(1 << 20) + 512, ld_k=512)     # in place


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=1025), dict(nq=0), dict(nq=3), dict(max_len=-1), dict(max_len=65), dict(ld_table=-1), dict(max_len=2 ** 30 + 1, ld_table=2 ** 27),
    dict(q=None), dict(o=None), dict(q=(1 << 20) + 8), dict(ld_q=252), dict(ld_q=260), dict(ld_q=1 << 62, ld_o=1 << 61), dict(ld_o=128), dict(table=None),
    dict(lens=None), dict(o=1 << 20), dict(o=(1 << 20) + 256), dict(w_in=16), dict(w_out=16, ld_w=63),
    dict(w_out=1 << 12, w_in=(1 << 12) + 4)])
def test_attention_decode_refuses(Q, kw):
    _refused(Q, 2, _attend, _cache(Q), **kw)


def test_attention_decode_of_no_sequences_does_nothing(Q):
    _attend(Q, _cache(Q), n=0)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=1025), dict(max_len=-1), dict(max_len=65), dict(max_len=2 ** 30 + 1, ld_table=2 ** 27, ld_w=2 ** 31, ld_w_out=2 ** 31), dict(budget=0), dict(sink=-1), dict(recent=-1),
    dict(sink=20, recent=13), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(table=None), dict(lens=None),
    dict(w=None), dict(w_out=None), dict(kept=None), dict(new=None), dict(ld_w=63), dict(ld_w_out=63),
    dict(ld_kept=31), dict(w_out=1 << 20), dict(w_out=(1 << 20) + 4), dict(table_out=16, ld_out=1)])
def test_cache_evict_refuses(Q, kw):
    _refused(Q, 2, _evict, _cache(Q), **kw)


def test_cache_evict_of_no_sequences_does_nothing(Q):
    _evict(Q, _cache(Q), n=0)


def test_workspace_size_without_a_gpu_or_for_refused_sizes(Q):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        assert Q.h3enc_op_attention_decode_workspace_bytes(1, 8, 100) == -1
    for bad in ((-1, 8, 100), (1025, 8, 100), (1, 0, 100), (1, 8, -1)):
        assert Q.h3enc_op_attention_decode_workspace_bytes(*bad) == -1


def test_kv_cache_checks_its_tensors(Q):
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    c = Q.KVCache(k, torch.zeros_like(k))
    assert (c.num_pages, c.n_kv_heads, c.page_size, c.head_dim, c.dtype, c.page_stride) == (3, 2, 16, 64, 0, 2048)
    both = torch.zeros(3, 2, 2, 16, 64, dtype=torch.bfloat16)             # K and V side by side
    assert Q.KVCache(both[:, 0], both[:, 1]).page_stride == 4096
    one = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)[:, :, :1].transpose(1, 2)     # one head: places 128 apart
    with pytest.raises(ValueError):
        Q.KVCache(one, one)
    one = torch.zeros(16, 1, 64, dtype=torch.bfloat16).as_strided((1, 1, 16, 64), (7, 5, 64, 1))   # strides of size 1
    assert Q.KVCache(one, one).page_stride == 16 * 64
    s = torch.ones(2)
    assert Q.KVCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn), s, s).dtype == 2
    for a, b, ks, vs in ((k, k[:2], None, None), (k.half(), k.half(), None, None), (k, k.float(), None, None),
                         (k.transpose(1, 2), k.transpose(1, 2), None, None), (k, k, s.double(), s), (k, k, s, s[:1])):
        with pytest.raises(ValueError):
            Q.KVCache(a, b, ks, vs)
    assert ctypes.sizeof(Q.KVCache) == 64


# ---------------------------------------------------------------- what the Python calls check of their tensors

class _Record:
    """Stands in for the library: keeps a call's arguments and succeeds."""
    def __getattr__(self, name):
        def call(*args):
            self.args = args
            return 0
        return call


@pytest.fixture
def on_cpu(Q, monkeypatch):
    """The calls with host tensors taken for the current device's, and nothing behind them."""
    torch = pytest.importorskip("torch")
    rec = _Record()
    monkeypatch.setattr(Q, "lib", rec)
    monkeypatch.setattr(Q, "_raw", (lambda: -1, lambda device: 0))
    return Q, torch, rec


def _tensors(torch, T=3, nq=4, nkv=2, d=64, page=16, max_len=40, budget=24):
    bf, i32 = torch.bfloat16, torch.int32
    n = T
    return dict(qkv=torch.zeros(T, (nq + 2 * nkv) * d, dtype=bf), w_q=torch.zeros(d, dtype=bf), w_k=torch.zeros(d, dtype=bf),
                cos=torch.zeros(T, d // 2), sin=torch.zeros(T, d // 2), q=torch.zeros(T, nq * d, dtype=bf),
                k=torch.zeros(T, nkv * d, dtype=bf), slots=torch.zeros(T, dtype=i32), status=torch.zeros(1, dtype=i32),
                o=torch.zeros(T, nq * d, dtype=bf), table=torch.zeros(n, 3, dtype=i32), lens=torch.zeros(n, dtype=i32),
                w=torch.zeros(n, max_len), w_out=torch.zeros(n, max_len), ws=torch.zeros(512, dtype=torch.uint8),
                table_out=torch.zeros(n, 2, dtype=i32), kept=torch.zeros(n, budget, dtype=i32),
                new=torch.zeros(n, dtype=i32), pool=torch.zeros(9, nkv, page, d, dtype=bf))


def _py_rope(Q, t, T=3, cs_stride=0):
    return Q.h3enc_op_qk_norm_rope(t["qkv"], T, 4, 2, 64, t["w_q"], t["w_k"], 1e-6, t["cos"], t["sin"], cs_stride, t["q"],
                                   t["k"], cache=Q.KVCache(t["pool"], t["pool"]), slots=t["slots"], status=t["status"])


def _py_attend(Q, t):
    return Q.h3enc_op_attention_decode(t["q"], t["o"], Q.KVCache(t["pool"], t["pool"]), t["table"], t["lens"], 4, 40,
                                       t["ws"], t["w"], t["w_out"], status=t["status"])


def _py_evict(Q, t):
    return Q.h3enc_op_cache_evict(Q.KVCache(t["pool"], t["pool"]), t["table"], t["lens"], 40, 24, t["w"], t["w_out"],
                                  t["kept"], t["new"], page_table_out=t["table_out"], status=t["status"])


PY_CALLS = [(_py_rope, ("qkv", "w_q", "w_k", "cos", "sin", "q", "k", "slots", "status")),
            (_py_attend, ("q", "o", "table", "lens", "w", "w_out", "status")),
            (_py_evict, ("table", "table_out", "lens", "w", "w_out", "kept", "new", "status"))]


@pytest.mark.parametrize("call,names", PY_CALLS)
def test_tensors_of_another_type_order_or_size_are_refused(on_cpu, call, names):
    Q, torch, rec = on_cpu
    call(Q, _tensors(torch))
    other = {torch.int32: torch.int64, torch.float32: torch.bfloat16, torch.bfloat16: torch.float32}
    for name in names:
        good = _tensors(torch)[name]
        bad = [good.to(other[good.dtype])]
        if name != "status":
            bad.append(good.new_zeros([2 * x for x in good.shape])[tuple([slice(None, None, 2)] * good.dim())])   # every other one
            if name != "lens":                                        # (its size is the number of sequences)
                bad.append(good[:-1])                                 # a row, or an element, too few
        if good.dim() == 2:
            bad.append(good.new_zeros(good.shape[::-1]).t())          # columns first
            wide = good.new_zeros(good.shape[0], good.shape[1] + 64)
            bad.append(wide[:, :good.shape[1] - 1])                   # the last column is not in the slice
        for t in bad:
            rec.args = None
            with pytest.raises(Q.H3encError) as e:
                call(Q, dict(_tensors(torch), **{name: t}))
            assert e.value.code == 2 and rec.args is None, (name, tuple(t.shape), t.stride())


@pytest.mark.parametrize("call,names", PY_CALLS)
def test_tensors_on_another_device_are_refused(on_cpu, call, names, monkeypatch):
    Q, torch, rec = on_cpu
    monkeypatch.setattr(Q, "_raw", (lambda: 0, lambda device: 0))
    t = _tensors(torch)
    with pytest.raises(Q.H3encError) as e:
        call(Q, t)                                                    # the cache too
    assert e.value.code == 2 and "current device" in str(e.value)
    monkeypatch.setattr(Q.KVCache, "device_index", property(lambda self: 0, lambda self, i: None), raising=False)
    with pytest.raises(Q.H3encError) as e:
        call(Q, t)
    assert e.value.code == 2 and "current device" in str(e.value)


@pytest.mark.parametrize("call", [_py_rope, _py_attend, _py_evict])
def test_sizes_may_be_any_integers(Q, call, monkeypatch):
    """numpy integers and tensors of one element, through the real argument types, up to the C entry's own refusal."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(Q, "_raw", (lambda: -1, lambda device: 0))
    t = _tensors(torch)
    for of in (int, np.int32, np.int64, torch.tensor):
        cache = Q.KVCache(t["pool"], t["pool"])
        with pytest.raises(Q.H3encError) as e:
            if call is _py_rope:
                Q.h3enc_op_qk_norm_rope(t["qkv"], of(3), of(4), of(2), of(64), t["w_q"], t["w_k"], -1e-6, t["cos"], t["sin"],
                                        of(0), t["q"], t["k"], cache=cache, slots=t["slots"])
            elif call is _py_attend:
                Q.h3enc_op_attention_decode(t["q"], t["o"], cache, t["table"], t["lens"], of(3), of(40), t["ws"])
            else:
                Q.h3enc_op_cache_evict(cache, t["table"], t["lens"], of(40), of(24), t["w"], t["w_out"], t["kept"], t["new"],
                                       sink=of(20), recent=of(5))
        assert e.value.code == 2


def test_numbers_beyond_a_32_bit_argument_are_refused(on_cpu):
    Q, torch, rec = on_cpu
    t = _tensors(torch)
    far = torch.empty_strided((3, 3), (2 ** 32 + 8, 1), dtype=torch.int32, device="meta")     # 8 if it is cut off
    c = Q.KVCache(t["pool"], t["pool"])
    for call in (lambda: _py_attend(Q, dict(t, table=far)), lambda: _py_evict(Q, dict(t, table=far)),
                 lambda: _py_evict(Q, dict(t, table_out=far)),
                 lambda: Q.h3enc_op_cache_evict(c, t["table"], t["lens"], 40, 24, t["w"], t["w_out"], t["kept"], t["new"],
                                                sink=2 ** 32 + 3),
                 lambda: Q.h3enc_op_cache_evict(c, t["table"], t["lens"], 40, 24, t["w"], t["w_out"], t["kept"], t["new"],
                                                recent=-2 ** 32 + 3),
                 lambda: Q.h3enc_op_cache_evict(c, t["table"], t["lens"], 40, 2 ** 32 + 24, t["w"], t["w_out"], t["kept"],
                                                t["new"]),
                 lambda: Q.h3enc_op_attention_decode(t["q"], t["o"], c, t["table"], t["lens"], 4, 2 ** 32 + 40, t["ws"]),
                 lambda: _py_rope(Q, t, T=2 ** 32 + 3)):
        rec.args = None
        with pytest.raises(Q.H3encError) as e:
            call()
        assert e.value.code == 2 and rec.args is None


def test_slices_single_rows_and_views_are_taken(on_cpu):
    Q, torch, rec = on_cpu
    t = _tensors(torch)
    wide = torch.zeros(5, 1024, dtype=torch.bfloat16)
    _py_rope(Q, dict(t, qkv=wide[:, 8:520], q=wide[:, 600:856]))      # slices of wider rows, more rows than needed
    assert rec.args[:3] == (wide.data_ptr() + 16, 1024, 3) and rec.args[12:14] == (wide.data_ptr() + 1200, 1024)
    assert rec.args[14:16] == (t["k"].data_ptr(), 128)
    _py_rope(Q, dict(t, q=t["q"].view(3, 4, 64)))                     # heads as a dimension
    assert rec.args[12:14] == (t["q"].data_ptr(), 256)
    one = dict(t, qkv=wide[4:, 8:520], q=wide[2:, 8:264])             # one row: its stride means nothing
    _py_rope(Q, one, T=1)
    assert rec.args[1] == 512 and rec.args[13] == 256
    _py_rope(Q, dict(t, qkv=wide[0, 8:520]), T=1)
    with pytest.raises(Q.H3encError):                                 # the row is short, although more rows follow
        _py_rope(Q, dict(t, q=torch.zeros(2, 128, dtype=torch.bfloat16)), T=1)
    for name, short in (("table", torch.zeros(4, 2, dtype=torch.int32)), ("w", torch.zeros(2, 39))):
        with pytest.raises(Q.H3encError):
            _py_attend(Q, dict(t, lens=t["lens"][:1], **{name: short}))
    _py_attend(Q, dict(t, lens=t["lens"][:1], table=torch.zeros(3, dtype=torch.int32)))
    grouped = torch.zeros(8, 32, 4)                                   # the row-interleaved tables
    _py_rope(Q, dict(t, cos=grouped, sin=grouped), cs_stride=32)
    with pytest.raises(Q.H3encError):
        _py_rope(Q, dict(t, cos=grouped[:7], sin=grouped), cs_stride=32)
    _py_rope(Q, t, T=0)
    table = torch.zeros(4, 7, dtype=torch.int32)
    _py_attend(Q, dict(t, table=table[1:, 2:]))
    assert rec.args[5:7] == (table.data_ptr() + 36, 7)
    _py_attend(Q, dict(t, w=t["w_out"]))                              # in place
    assert rec.args[11] == rec.args[12] == t["w_out"].data_ptr()
    with pytest.raises(ValueError):
        _py_attend(Q, dict(t, w=torch.zeros(3, 50)))
    _py_evict(Q, dict(t, new=t["lens"], kept=torch.zeros(3, 30, dtype=torch.int32)[:, :24]))
    assert rec.args[16] == 30 and rec.args[17] == t["lens"].data_ptr()
    Q.h3enc_op_attention_decode(t["q"], t["o"], Q.KVCache(t["pool"], t["pool"]), torch.zeros(3, 0, dtype=torch.int32),
                                t["lens"], 4, 0, t["ws"], None, torch.zeros(3, 0))     # no tokens, no pages
