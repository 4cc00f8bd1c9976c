"""Timing cases of the cached-decoding operators: the per-head q/k norm and rotation that fills a
paged key/value cache, the attention of one new token over it, and the eviction from it by
accumulated attention weight.

`run` computes an operator with elementary torch operations in 32 bits, or, where `own` is set, with
the library's call.  `exact` restates each operator in 64 bits.  Sizes follow the repository's
decoders: 64 query heads over 8 key/value heads of 128, 4 over 2 of 64 (the small model), and the
other head layouts the library takes.
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- cases

def _rope(name, T, nq, nkv, d, dtype, page, grouped, k_out, pad):
    """T rows of a QKV projection; grouped: the row-interleaved rotary tables; pad: every pad-th
    row is a padding row that gets no place in the cache (0: none)."""
    c = dict(op="rope", T=T, nq=nq, nkv=nkv, d=d, dtype=dtype, page=page, grouped=grouped, k_out=k_out, pad=pad)
    return dict(name=name, **c) if name else c


def _attn(name, n, nq, nkv, d, dtype, page, lo, hi, empty, weights):
    """n sequences of lengths spread over lo..hi (their logarithm), the first one empty if `empty`."""
    c = dict(op="attn", n=n, nq=nq, nkv=nkv, d=d, dtype=dtype, page=page, lo=lo, hi=hi, empty=empty, weights=weights)
    return dict(name=name, **c) if name else c


def _evict(name, n, nkv, d, dtype, page, lo, hi, budget, sink, recent):
    """n sequences of lengths lo..hi cut to `budget` tokens, copied into other pages of the pool."""
    c = dict(op="evict", n=n, nkv=nkv, d=d, dtype=dtype, page=page, lo=lo, hi=hi, budget=budget, sink=sink,
             recent=recent)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one new token of one sequence: the call between two projections of a single-user decode step
        _rope("rope-token", 1, 64, 8, 128, "bf16", 64, False, False, 0),
        # a decode step of a ragged batch padded to its slot count, e4m3 cache
        _rope("rope-batch-e4m3", 250, 64, 8, 128, "e4m3", 64, True, False, 5),
        # a prompt of the longest encode (8192 tokens): fills the cache behind the prefill
        _rope("rope-prompt", 8192, 64, 8, 128, "bf16", 64, True, True, 0),
        # the small model's heads, a prompt of odd length
        _rope("rope-small-heads", 4595, 4, 2, 64, "bf16", 16, False, True, 0),
        # one user's next token after a 1024-token prompt
        _attn("attn-one", 1, 64, 8, 128, "bf16", 64, 1025, 1025, False, False),
        # sixteen prompts of 77 to 512 tokens, one slot of the batch unused
        _attn("attn-prompts", 16, 64, 8, 128, "bf16", 16, 77, 512, True, False),
        # a serving batch deep into long answers: the cache alone is 1.7 GB
        _attn("attn-batch", 64, 64, 8, 128, "bf16", 64, 5000, 8192, False, False),
        # one long document, 8-bit cache
        _attn("attn-long-e4m3", 1, 64, 8, 128, "e4m3", 128, 130001, 130001, False, False),
        # a batch that also accumulates the attention weight of every cached token (for the eviction)
        _attn("attn-weights", 24, 64, 8, 128, "bf16", 64, 500, 4608, False, True),
        # few short sequences cut to a small budget
        _evict("evict-few", 4, 8, 128, "bf16", 64, 250, 321, 256, 4, 64),
        # a serving batch cut from up to 4608 tokens to 4096
        _evict("evict-batch", 32, 8, 128, "bf16", 64, 4000, 4608, 4096, 4, 256),
        # one long document cut to a quarter, 8-bit cache
        _evict("evict-long-e4m3", 1, 8, 128, "e4m3", 128, 65537, 65537, 16384, 16, 1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(64, 8, 128), (4, 2, 64), (32, 4, 128), (16, 16, 64), (24, 8, 128), (12, 1, 64), (40, 2, 128), (28, 4, 64)]


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "evict"])
    nq, nkv, d = rng.choice(_HEADS)
    dtype, page = rng.choice(["bf16", "bf16", "e4m3"]), rng.choice([16, 32, 64, 128, 256])
    if op == "rope":
        return _rope("", _log_int(rng, 1, 8192), nq, nkv, d, dtype, page, rng.random() < 0.5, rng.random() < 0.5,
                     rng.choice([0, 0, 3, 7]))
    if op == "attn":
        weights = rng.random() < 0.4
        hi = _log_int(rng, 20, 60000)
        lo = max(1, int(hi * rng.choice([1.0, 0.7, 0.1])))
        n = _log_int(rng, 1, max(1, min(100, 200000 // hi)))
        return _attn("", n, nq, nkv, d, dtype, page, lo, hi, n > 1 and rng.random() < 0.3, weights)
    hi = _log_int(rng, 40, 60000)
    lo = max(1, int(hi * rng.choice([1.0, 0.9, 0.5])))
    budget = max(16, int(hi * rng.uniform(0.1, 0.95)))
    n = _log_int(rng, 1, max(1, min(64, 100000 // hi)))
    return _evict("", n, nkv, d, dtype, page, lo, hi, budget, min(4, budget // 8), budget // rng.choice([4, 8, 16]))


def _lens(c):
    n, lo, hi = c["n"], c["lo"], c["hi"]
    v = [hi if n == 1 else int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]
    if c.get("empty"):
        v[0] = 0
    return v


def work(c):
    es = 1 if c["dtype"] == "e4m3" else 2
    nkv, d = c["nkv"], c["d"]
    if c["op"] == "rope":
        T, nq = c["T"], c["nq"]
        kept = T - (T // c["pad"] if c["pad"] else 0)
        b = T * (nq + 2 * nkv) * d * 2 + T * d * 4 + 4 * T + T * nq * d * 2 + kept * 2 * nkv * d * es
        b += T * nkv * d * 2 if c["k_out"] else 0
        return {"bytes": b, "flops": T * (nq + nkv) * d * 8}
    total = sum(_lens(c))
    if c["op"] == "attn":
        b = total * nkv * d * 2 * es + 4 * c["n"] * c["nq"] * d + 4 * (total // c["page"]) + 4 * c["n"]
        b += 8 * total if c["weights"] else 0
        return {"bytes": b, "flops": 4 * total * c["nq"] * d}
    kept = sum(min(x, c["budget"]) for x in _lens(c))
    b = 4 * total + kept * (4 * nkv * d * es + 8)
    return {"bytes": b, "flops": total}


# ---------------------------------------------------------------- inputs

def _pool(g, pages, c, fill):
    shape = (pages, c["nkv"], c["page"], c["d"])
    if not fill:
        x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    else:
        x = torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=g)
    return x if c["dtype"] == "bf16" else _to_e4m3(x)


def _to_e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = case
    nkv, d, page = c["nkv"], c["d"], c["page"]
    s = {"c": c}
    if c["dtype"] == "e4m3":
        s["k_scale"] = 0.02 + 0.01 * torch.rand(nkv, device="cuda", generator=g)
        s["v_scale"] = 0.02 + 0.01 * torch.rand(nkv, device="cuda", generator=g)
        if c["op"] != "rope":   # a filled cache of values of about 1
            s["k_scale"], s["v_scale"] = s["k_scale"] * 40, s["v_scale"] * 40
    else:
        s["k_scale"] = s["v_scale"] = None
    if c["op"] == "rope":
        _prepare_rope(s, g)
    else:
        lens = torch.tensor(_lens(c), device="cuda", dtype=torch.int32)
        order = torch.randperm(c["n"], generator=g, device="cuda")
        s["lens"] = lens[order].contiguous()
        s["cols"] = -(-c["hi"] // page)
        out_cols = -(-c["budget"] // page) if c["op"] == "evict" else 0
        pages = c["n"] * (s["cols"] + out_cols)
        s["k"], s["v"] = _pool(g, pages, c, True), _pool(g, pages, c, True)
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["table"] = ids[:c["n"] * s["cols"]].view(c["n"], s["cols"]).contiguous()
        if c["op"] == "attn":
            _prepare_attn(s, g)
        else:
            s["table_out"] = ids[c["n"] * s["cols"]:].view(c["n"], out_cols).contiguous()
            # weights as a run of decode steps leaves them: most tokens little, a few a lot
            s["weight"] = torch.empty(c["n"], c["hi"], device="cuda").exponential_(generator=g).pow_(3)
            s["weight_out"] = torch.zeros(c["n"], c["hi"], device="cuda")
            s["kept"] = torch.zeros(c["n"], c["budget"], dtype=torch.int32, device="cuda")
            s["new_lens"] = torch.zeros(c["n"], dtype=torch.int32, device="cuda")
    if own:
        import qwen3_vl_text_gb300 as Q
        s["Q"] = Q
        s["cache"] = Q.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if c["op"] == "attn":
            size = Q.h3enc_op_attention_decode_workspace_bytes(c["n"], c["nq"], c["hi"], c["weights"])
            s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return s


def _prepare_rope(s, g):
    c = s["c"]
    T, nq, nkv, d, page = c["T"], c["nq"], c["nkv"], c["d"], c["page"]
    dev = dict(device="cuda", generator=g)
    s["qkv"] = torch.randn(T, (nq + 2 * nkv) * d, dtype=torch.bfloat16, **dev)
    s["w_q"] = (1 + 0.1 * torch.randn(d, **dev)).to(torch.bfloat16)
    s["w_k"] = (1 + 0.1 * torch.randn(d, **dev)).to(torch.bfloat16)
    first = torch.randint(0, 4096, (1,), **dev)
    pos = (first + torch.arange(T, device="cuda")).to(torch.float64)
    ang = pos[:, None] * 5e6 ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    cos, sin = ang.cos().float(), ang.sin().float()
    s["stride"] = 0
    if c["grouped"]:   # [d/8][stride][4]: groups of four frequencies, rows one after another
        s["stride"] = -(-T // 32) * 32
        cos, sin = (torch.nn.functional.pad(t, (0, 0, 0, s["stride"] - T)).view(-1, d // 8, 4).transpose(0, 1)
                    .contiguous() for t in (cos, sin))
    s["cos"], s["sin"] = cos, sin
    pages = -(-T // page) + 1
    s["k"], s["v"] = _pool(g, pages, c, False), _pool(g, pages, c, False)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    if c["pad"]:
        slots[c["pad"] - 1::c["pad"]] = -1
    s["slots"] = slots.contiguous()
    s["q_out"] = torch.zeros(T, nq * d, dtype=torch.bfloat16, device="cuda")
    s["k_out"] = torch.zeros(T, nkv * d, dtype=torch.bfloat16, device="cuda") if c["k_out"] else None


def _prepare_attn(s, g):
    c = s["c"]
    # normed queries with a gain: rows attend to some keys much more than to others
    s["q"] = (2 * torch.randn(c["n"], c["nq"] * c["d"], device="cuda", generator=g)).to(torch.bfloat16)
    s["o"] = torch.zeros_like(s["q"])
    s["weight"] = s["weight_out"] = None
    if c["weights"]:
        s["weight"] = torch.rand(c["n"], c["hi"], device="cuda", generator=g)
        s["weight_out"] = torch.zeros_like(s["weight"])


# ---------------------------------------------------------------- one pass

def run(s):
    return {"rope": _run_rope, "attn": _run_attn, "evict": _run_evict}[s["c"]["op"]](s)


def _run_rope(s):
    c = s["c"]
    T, nq, nkv, d, page = c["T"], c["nq"], c["nkv"], c["d"], c["page"]
    out = {"q": s["q_out"], "k_cache": s["k"], "v_cache": s["v"]}
    if c["k_out"]:
        out["k"] = s["k_out"]
    if own:
        s["Q"].h3enc_op_qk_norm_rope(s["qkv"], T, nq, nkv, d, s["w_q"], s["w_k"], EPS, s["cos"], s["sin"], s["stride"],
                                     s["q_out"], s["k_out"], cache=s["cache"], slots=s["slots"])
        return out
    x = s["qkv"].view(T, nq + 2 * nkv, d)
    cos, sin = s["cos"], s["sin"]
    if s["stride"]:
        cos, sin = (t.transpose(0, 1).reshape(-1, d // 2)[:T] for t in (cos, sin))

    def norm_rope(h, w):
        h = h.float()
        h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * w.float()
        a, b = h[..., :d // 2], h[..., d // 2:]
        cs, sn = cos[:, None], sin[:, None]
        return torch.cat([a * cs - b * sn, b * cs + a * sn], -1)

    s["q_out"].view(T, nq, d).copy_(norm_rope(x[:, :nq], s["w_q"]))
    k = norm_rope(x[:, nq:nq + nkv], s["w_k"])
    if c["k_out"]:
        s["k_out"].view(T, nkv, d).copy_(k)
    # padding rows are sent to the slot of the first row, with the first row's vector
    slots = s["slots"].long()
    keep = slots >= 0
    at = torch.where(keep, slots, slots[:1])
    for src, pool, scale in ((k, s["k"], s["k_scale"]), (x[:, nq + nkv:].float(), s["v"], s["v_scale"])):
        src = torch.where(keep[:, None, None], src, src[:1])
        if scale is None:
            pool[at // page, :, at % page] = src.to(torch.bfloat16)
        else:
            pool.view(torch.uint8)[at // page, :, at % page] = _to_e4m3(src / scale[:, None]).view(torch.uint8)
    return out


def _run_attn(s):
    c = s["c"]
    n, nq, nkv, d, page = c["n"], c["nq"], c["nkv"], c["d"], c["page"]
    out = {"o": s["o"]}
    if c["weights"]:
        out["weight"] = s["weight_out"]
    if own:
        s["Q"].h3enc_op_attention_decode(s["q"], s["o"], s["cache"], s["table"], s["lens"], nq, c["hi"], s["workspace"],
                                         weight_in=s["weight"], weight_out=s["weight_out"])
        return out
    size = s["cols"] * page

    def gathered(pool, scale):   # [n, nkv, size, d] in 32 bits
        x = pool.view(torch.uint8)[s["table"].long()].view(pool.dtype) if scale is not None else pool[s["table"].long()]
        x = x.permute(0, 2, 1, 3, 4).reshape(n, nkv, size, d).float()
        return x if scale is None else x * scale[:, None, None]

    q = s["q"].view(n, nkv, nq // nkv, d).float()
    mask = torch.arange(size, device="cuda")[None] < s["lens"][:, None]
    sc = torch.matmul(q, gathered(s["k"], s["k_scale"]).transpose(2, 3)) / math.sqrt(d)
    sc = sc.masked_fill(~mask[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - top.masked_fill(top == -math.inf, 0))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    s["o"].view(n, nkv, nq // nkv, d).copy_(torch.matmul(p, gathered(s["v"], s["v_scale"])))
    if c["weights"]:
        w = s["weight"] + p.sum((1, 2))[:, :c["hi"]]
        s["weight_out"].copy_(torch.where(mask[:, :c["hi"]], w, s["weight_out"]))
    return out


def _run_evict(s):
    c = s["c"]
    page, budget, hi = c["page"], c["budget"], c["hi"]
    out = {"kept": s["kept"], "lens": s["new_lens"], "weight": s["weight_out"], "k": s["k"], "v": s["v"]}
    if own:
        s["Q"].h3enc_op_cache_evict(s["cache"], s["table"], s["lens"], hi, budget, s["weight"], s["weight_out"],
                                    s["kept"], s["new_lens"], page_table_out=s["table_out"], sink=c["sink"],
                                    recent=c["recent"])
        return out
    lens = s["lens"][:, None]
    idx = torch.arange(hi, device="cuda")[None]
    live = idx < lens
    key = torch.where((idx < c["sink"]) | (idx >= lens - c["recent"]), math.inf, s["weight"])
    key = torch.where(live, key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    top = torch.where(torch.gather(live.expand(c["n"], hi), 1, order), order, hi)[:, :budget]
    kept = torch.sort(top, dim=1).values
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[1]), value=hi)
    valid = kept < hi
    s["kept"].copy_(torch.where(valid, kept, -1))
    s["new_lens"].copy_(valid.sum(1))
    src = torch.where(valid, kept, 0)
    w = torch.where(valid, torch.gather(s["weight"], 1, src), 0)
    s["weight_out"].copy_(torch.nn.functional.pad(w, (0, hi))[:, :hi])
    sp, so = torch.gather(s["table"].long(), 1, src // page), src % page
    dst = torch.arange(budget, device="cuda").expand(c["n"], budget)
    dp, do = torch.gather(s["table_out"].long(), 1, dst // page), dst % page
    for pool in (s["k"], s["v"]):
        raw = pool.view(torch.uint8) if pool.element_size() == 1 else pool
        raw[dp, :, do] = torch.where(valid[..., None, None], raw[sp, :, so], raw[dp, :, do])
    return out


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """From the definitions, a row or a sequence at a time, in float64."""
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "evict": _exact_evict}[case["op"]](s)


def _exact_rope(s):
    c = s["c"]
    T, nq, nkv, d, page = c["T"], c["nq"], c["nkv"], c["d"], c["page"]
    half = d // 2
    rows = torch.arange(T, device="cuda")
    j = torch.arange(half, device="cuda")
    if s["stride"]:
        at = ((j[None] // 4) * s["stride"] + rows[:, None]) * 4 + j[None] % 4
    else:
        at = rows[:, None] * half + j[None]
    turn = torch.complex(s["cos"].double().reshape(-1)[at], s["sin"].double().reshape(-1)[at])
    x = s["qkv"].double()
    heads = []
    for h in range(nq + nkv):
        w = (s["w_q"] if h < nq else s["w_k"]).double()
        v = x[:, h * d:(h + 1) * d]
        v = v * w * (v.square().sum(1, keepdim=True) / d + EPS).rsqrt()
        z = torch.complex(v[:, :half], v[:, half:]) * turn
        heads.append(torch.cat([z.real, z.imag], 1))
    k = torch.stack(heads[nq:], 1)
    v = x[:, (nq + nkv) * d:].view(T, nkv, d)
    out = {"q": torch.cat(heads[:nq], 1)}
    live = torch.nonzero(s["slots"] >= 0).flatten()
    slot = s["slots"][live].long()
    for name, pool, val, scale in (("k_cache", s["k"], k, s["k_scale"]), ("v_cache", s["v"], v, s["v_scale"])):
        flat = pool.double().transpose(1, 2).reshape(-1, nkv, d)
        flat[slot] = val[live] if scale is None else (val[live] / scale.double()[:, None]).clamp(-448, 448)
        out[name] = flat.view(-1, page, nkv, d).transpose(1, 2).contiguous()
    if c["k_out"]:
        out["k"] = k.reshape(T, nkv * d)
    return out


def _exact_attn(s):
    c = s["c"]
    n, nq, nkv, d = c["n"], c["nq"], c["nkv"], c["d"]
    g = nq // nkv
    o = torch.zeros(n, nq, d, dtype=torch.float64, device="cuda")
    weight = None if not c["weights"] else s["weight_out"].double()
    for b, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        pages = s["table"][b, :-(-length // c["page"])].long()
        for h in range(nkv):
            k = s["k"][pages, h].double().reshape(-1, d)[:length]
            v = s["v"][pages, h].double().reshape(-1, d)[:length]
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            q = s["q"][b].view(nq, d)[h * g:(h + 1) * g].double()
            p = torch.softmax(k @ q.T * d ** -0.5, dim=0)
            o[b, h * g:(h + 1) * g] = p.T @ v
            if c["weights"]:
                weight[b, :length] += p.sum(1) if h else s["weight"][b, :length].double() + p.sum(1)
    out = {"o": o.view(n, nq * d)}
    if c["weights"]:
        out["weight"] = weight
    return out


def _exact_evict(s):
    c = s["c"]
    page = c["page"]
    out = {"kept": torch.full_like(s["kept"], -1), "lens": torch.zeros_like(s["new_lens"]),
           "weight": torch.zeros_like(s["weight_out"], dtype=torch.float64), "k": s["k"].clone(), "v": s["v"].clone()}
    for b, length in enumerate(s["lens"].tolist()):
        w = s["weight"][b, :length].cpu().double().numpy()
        ranked = sorted(range(length), key=lambda i: (not (i < c["sink"] or i >= length - c["recent"]), -w[i], i)
                        if not (i < c["sink"] or i >= length - c["recent"]) else (False, 0.0, i))
        keep = torch.tensor(sorted(ranked[:c["budget"]]), dtype=torch.long, device="cuda")
        m = len(keep)
        out["kept"][b, :m], out["lens"][b] = keep.int(), m
        out["weight"][b, :m] = s["weight"][b, keep].double()
        to = torch.arange(m, device="cuda")
        for name in ("k", "v"):
            raw, old = out[name].view(torch.uint8), s[name].view(torch.uint8)
            raw[s["table_out"][b, to // page].long(), :, to % page] = old[s["table"][b, keep // page].long(), :, keep % page]
    out["k"], out["v"] = out["k"].float(), out["v"].float()
    return out
