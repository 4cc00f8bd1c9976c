"""Timing cases of the operators of a decoder that reads an encoder's states: new rows rotated and appended to a
paged cache, the attention of one new token of sequences that share a prefix, and cross attention.

`run` computes an operator with elementary torch operations in 32 bits (angles in 64), or, where `own` is set, with
the library's call.  `exact` restates each operator in 64 bits.  Sizes follow the repository's decoders: 64
query heads over 8 key/value heads of 128, 4 over 2 of 64 (the small model), prompts of 77 to 512 tokens,
sequences of 1024 and 8192, and the other head layouts the library takes.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 5e6
ORIGINAL = 4096      # tokens of the contexts that the scalings stretch


# ---------------------------------------------------------------- cases

def _append(name, n, lo, hi, start, nq, nkv, d, dtype, page, rot, inter, scaling, factor, axes, norm, k_out, pad):
    """lo..hi new rows of each of n sequences that hold up to `start` tokens; the first `rot` elements of a head
    rotated, pairs side by side if `inter`; `pad` rows behind the last sequence."""
    c = dict(op="append", n=n, lo=lo, hi=hi, start=start, nq=nq, nkv=nkv, d=d, dtype=dtype, page=page, rot=rot,
             inter=inter, scaling=scaling, factor=factor, axes=axes, norm=norm, k_out=k_out, pad=pad)
    return dict(name=name, **c) if name else c


def _shared(name, groups, n, plo, phi, lo, hi, nq, nkv, d, dtype, page, weights):
    """n sequences of lo..hi tokens of their own behind `groups` prefixes of plo..phi tokens."""
    c = dict(op="shared", groups=groups, n=n, plo=plo, phi=phi, lo=lo, hi=hi, nq=nq, nkv=nkv, d=d, dtype=dtype,
             page=page, weights=weights)
    return dict(name=name, **c) if name else c


def _cross(name, n, qlo, qhi, klo, khi, nq, nkv, d, empty):
    """n sequences of qlo..qhi queries over klo..khi states; `empty`: the second one has no states."""
    c = dict(op="cross", n=n, lo=qlo, hi=qhi, klo=klo, khi=khi, nq=nq, nkv=nkv, d=d, empty=empty)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one new token of one sequence far into a stretched context: between two projections of a decode step
        _append("append-token", 1, 1, 1, 40000, 64, 8, 128, "bf16", 64, 128, False, "yarn", 16.0, 1, True, False, 0),
        # a decode step of a ragged batch padded to its slot count, 8-bit cache, half of each head rotated in pairs
        _append("append-batch-e4m3", 200, 1, 1, 3000, 64, 8, 128, "e4m3", 64, 64, True, "linear", 4.0, 1, False, False, 50),
        # image prompts of 77 to 512 tokens at three-axis positions behind what their conversations hold already
        _append("append-prompts", 24, 77, 512, 900, 64, 8, 128, "bf16", 16, 128, False, "none", 1.0, 3, True, True, 0),
        # the small model's heads, one long prompt of odd length, half of each head rotated
        _append("append-small-heads", 1, 4595, 4595, 13, 4, 2, 64, "bf16", 16, 32, False, "wavelength", 8.0, 1, False,
                True, 0),
        # four answers sampled to one short question
        _shared("shared-few", 1, 4, 1000, 1000, 20, 60, 64, 8, 128, "bf16", 64, False),
        # a serving batch behind one long instruction
        _shared("shared-batch", 1, 64, 8192, 8192, 100, 1024, 64, 8, 128, "bf16", 64, False),
        # sixteen questions about one long document, 8-bit cache
        _shared("shared-long-e4m3", 1, 16, 65537, 65537, 300, 2000, 64, 8, 128, "e4m3", 128, False),
        # three tenants' instructions, and the weight of every own token accumulated for the eviction
        _shared("shared-groups", 3, 48, 500, 4097, 50, 700, 64, 8, 128, "bf16", 16, True),
        # one decoder token over the states of one 1024-token prompt
        _cross("cross-token", 1, 1, 1, 1024, 1024, 64, 8, 128, False),
        # a decode step of 64 sequences over prompts of 77 to 512 tokens
        _cross("cross-tokens", 64, 1, 1, 77, 512, 64, 8, 128, False),
        # the patches of one picture over the states of its 1024-token prompt
        _cross("cross-picture", 1, 4096, 4096, 1024, 1024, 64, 8, 128, False),
        # sixteen ragged rows of patches over prompts of 77 to 512 tokens, every head its own; one prompt is missing
        _cross("cross-prompts", 16, 500, 2305, 77, 512, 40, 40, 128, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(64, 8, 128), (4, 2, 64), (32, 4, 128), (18, 18, 64), (28, 4, 128), (12, 1, 64), (40, 2, 128), (20, 4, 64),
          (40, 40, 128)]


def draw(rng):
    op = rng.choice(["append", "shared", "cross"])
    nq, nkv, d = rng.choice(_HEADS)
    if op == "append":
        dtype, page = rng.choice(["bf16", "bf16", "e4m3"]), rng.choice([16, 32, 64, 128, 256])
        rot, inter = rng.choice([d, d, d // 2, d // 4]), rng.random() < 0.4
        scaling = rng.choice(["none", "linear", "wavelength", "yarn"])
        factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0])
        hi = rng.choice([1, 1, _log_int(rng, 2, 2700)])
        n = _log_int(rng, 1, max(1, min(256, int(2e8 / ((2 * nq + 5 * nkv) * d * 2)) // hi)))
        lo = max(1, int(hi * rng.choice([1.0, 0.5, 0.1])))
        axes = 3 if scaling == "none" and rot == d and rng.random() < 0.5 else 1
        return _append("", n, lo, hi, _log_int(rng, 1, 100000 // n), nq, nkv, d, dtype, page, rot, inter, scaling,
                       factor, axes, rng.random() < 0.5, rng.random() < 0.4, rng.choice([0, 0, 5, 37]))
    if op == "shared":
        dtype, page = rng.choice(["bf16", "bf16", "e4m3"]), rng.choice([16, 32, 64, 128, 256])
        n = _log_int(rng, 1, 128)
        groups = rng.choice([1, 1, 1, 2, 5])
        most = min(65000, int(4e9 / (n * nq * d)), 350000 // (nkv * groups))
        phi = _log_int(rng, 1, most)
        hi = _log_int(rng, 1, max(2, 350000 // (nkv * n)))
        return _shared("", groups, n, max(1, int(phi * rng.choice([1.0, 0.6, 0.1]))), phi,
                       max(1, int(hi * rng.choice([1.0, 0.5, 0.1]))), hi, nq, nkv, d, dtype, page, rng.random() < 0.3)
    n = rng.choice([1, _log_int(rng, 1, 64)])
    khi = _log_int(rng, 1, min(32768, 8000000 // (n * nkv * d)))
    qhi = rng.choice([1, _log_int(rng, 2, max(3, min(int(8e7 / (nq * d * n)), int(3e10 / (nq * d * n * khi)))))])
    return _cross("", n, max(1, int(qhi * rng.choice([1.0, 0.7, 0.1]))), qhi, max(1, int(khi * rng.choice([1.0, 0.7, 0.1]))),
                  khi, nq, nkv, d, n > 2 and rng.random() < 0.3)


def _spread(n, lo, hi):
    """n numbers from lo to hi, even in their logarithm."""
    return [hi if n == 1 else int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _key_lens(c):
    v = _spread(c["n"], c["klo"], c["khi"])
    if c["empty"]:
        v[1] = 0
    return v


def _groups(c):
    """First sequence of each group, and the end: sizes that differ, the last group empty where they do not suffice."""
    n, g = c["n"], c["groups"]
    return [min(n, n * i * (i + 1) // (g * (g + 1)) + (1 if 0 < i < g else 0)) for i in range(g)] + [n]


def work(c):
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    if c["op"] == "cross":
        pairs = list(zip(_spread(c["n"], c["lo"], c["hi"]), _key_lens(c)))
        b = sum(4 * q * nq * d + 4 * k * nkv * d for q, k in pairs)
        return {"bytes": b, "flops": sum(4 * q * k for q, k in pairs) * nq * d}
    es = 1 if c["dtype"] == "e4m3" else 2
    total = sum(_spread(c["n"], c["lo"], c["hi"]))
    if c["op"] == "append":
        b = total * ((2 * nq + 2 * nkv) * d * 2 + 2 * nkv * d * es + 4 * c["axes"])
        b += total * nkv * d * 2 if c["k_out"] else 0
        return {"bytes": b, "flops": total * (nq + nkv) * d * 8}
    first = _groups(c)
    plens = _spread(c["groups"], c["plo"], c["phi"])
    keys = total + sum(p for p, a, b in zip(plens, first, first[1:]) if b > a)
    flops = 4 * nq * d * (total + sum(p * (b - a) for p, a, b in zip(plens, first, first[1:])))
    b = keys * nkv * d * 2 * es + 4 * c["n"] * nq * d + 4 * (keys // c["page"]) + 4 * c["n"]
    return {"bytes": b + (8 * total if c["weights"] else 0), "flops": flops}


# ---------------------------------------------------------------- inputs

def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _pool(g, pages, c, fill):
    shape = (pages, c["nkv"], c["page"], c["d"])
    x = (torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=g) if fill
         else torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))
    return x if c["dtype"] == "bf16" else _e4m3(x)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": case}
    if own:
        import qwen3_vl_text_gb300 as Q
        s["Q"] = Q
    {"append": _prepare_append, "shared": _prepare_shared, "cross": _prepare_cross}[case["op"]](s, g)
    if own and "k" in s and case["op"] != "cross":
        s["cache"] = s["Q"].KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


def _scales(s, g, size):
    s["k_scale"] = s["v_scale"] = None
    if s["c"]["dtype"] == "e4m3":
        s["k_scale"], s["v_scale"] = (size * (1 + torch.rand(s["c"]["nkv"], device="cuda", generator=g)) for _ in range(2))


def _section(rot):
    return [rot // 2 - 2 * (rot * 5 // 32), rot * 5 // 32, rot * 5 // 32]      # 24, 20, 20 of 64


def _prepare_append(s, g):
    c = s["c"]
    n, nq, nkv, d, page = c["n"], c["nq"], c["nkv"], c["d"], c["page"]
    dev = dict(device="cuda", generator=g)
    rows = torch.tensor(_spread(n, c["lo"], c["hi"]), device="cuda")[torch.randperm(n, **dev)]
    held = torch.randint(0, c["start"] + 1, (n,), **dev)
    live, T = int(rows.sum()), int(rows.sum()) + c["pad"]
    s["T"], s["live"] = T, live
    s["cu"] = torch.cat([rows.new_zeros(1), rows.cumsum(0)]).to(torch.int32)
    s["lens"] = (held + rows).to(torch.int32)                  # the new rows counted in
    s["max_len"] = c["start"] + c["hi"]
    cols = -(-s["max_len"] // page)
    # the pages of the new rows lie anywhere in the pool, earlier ones are not touched by this call
    need = torch.zeros(n, cols, dtype=torch.bool, device="cuda")
    col = torch.arange(cols, device="cuda")[None]
    need = (col >= held[:, None] // page) & (col <= (held + rows - 1)[:, None] // page)
    pages = sum(-(-m // page) + 1 for m in _spread(n, c["lo"], c["hi"]))
    s["table"] = torch.zeros(n, cols, dtype=torch.int32, device="cuda")
    s["table"][need] = torch.randperm(pages, **dev)[:int(need.sum())].to(torch.int32)
    _scales(s, g, 0.02)
    s["k"], s["v"] = _pool(g, pages, c, False), _pool(g, pages, c, False)
    s["qkv"] = torch.randn(T, (nq + 2 * nkv) * d, dtype=torch.bfloat16, **dev)
    s["w_q"], s["w_k"] = ((1 + 0.1 * torch.randn(d, **dev)).to(torch.bfloat16) if c["norm"] else None for _ in range(2))
    s["positions"] = None
    if c["axes"] == 3:     # an image's rows and columns within the text's positions
        s["positions"] = torch.randint(0, 8192, (3, T), **dev).to(torch.int32)
    s["q_out"] = torch.zeros(T, nq * d, dtype=torch.bfloat16, device="cuda")
    s["k_out"] = torch.zeros(T, nkv * d, dtype=torch.bfloat16, device="cuda") if c["k_out"] else None
    s["one"] = c["lo"] == c["hi"] == 1 and c["pad"] == 0       # a row per sequence: no row offsets needed
    if own:
        s["rope"] = s["Q"].Rope(c["rot"], theta=THETA, interleaved=c["inter"], scaling=c["scaling"], factor=c["factor"],
                                original_len=ORIGINAL, section=_section(c["rot"]) if c["axes"] == 3 else None)


def _prepare_shared(s, g):
    c = s["c"]
    n, page, groups = c["n"], c["page"], c["groups"]
    lens = torch.tensor(_spread(n, c["lo"], c["hi"]), device="cuda", dtype=torch.int32)
    s["lens"] = lens[torch.randperm(n, generator=g, device="cuda")].contiguous()
    s["first"] = _groups(c)
    s["prefix_rows"] = torch.tensor(s["first"], device="cuda", dtype=torch.int32) if groups > 1 else None
    s["prefix_lens"] = torch.tensor(_spread(groups, c["plo"], c["phi"]), device="cuda", dtype=torch.int32)
    cols, pcols = -(-c["hi"] // page), -(-c["phi"] // page)
    pages = n * cols + groups * pcols
    _scales(s, g, 0.8)                                         # a filled cache of values of about 1
    s["k"], s["v"] = _pool(g, pages, c, True), _pool(g, pages, c, True)
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["table"] = ids[:n * cols].view(n, cols).contiguous()
    s["prefix_table"] = ids[n * cols:].view(groups, pcols).contiguous()
    # normed queries with a gain: rows attend to some keys much more than to others
    s["q"] = (2 * torch.randn(n, c["nq"] * c["d"], device="cuda", generator=g)).to(torch.bfloat16)
    s["o"] = torch.zeros_like(s["q"])
    s["weight"] = s["weight_out"] = None
    if c["weights"]:
        s["weight"] = torch.rand(n, c["hi"], device="cuda", generator=g)
        s["weight_out"] = torch.zeros_like(s["weight"])
    if own:
        size = s["Q"].h3enc_op_attention_decode_shared_workspace_bytes(n, c["nq"], c["hi"], c["weights"])
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")


def _prepare_cross(s, g):
    c = s["c"]
    n, nq, nkv, d = c["n"], c["nq"], c["nkv"], c["d"]
    dev = dict(device="cuda", generator=g)
    order = torch.randperm(n, **dev).tolist()
    spread_q, spread_k = _spread(n, c["lo"], c["hi"]), _key_lens(c)
    s["qlens"], s["klens"] = [spread_q[i] for i in order], [spread_k[i] for i in order]
    s["cu_q"], s["cu_k"] = (torch.tensor([sum(v[:i]) for i in range(n + 1)], device="cuda", dtype=torch.int32)
                            if n > 1 else None for v in (s["qlens"], s["klens"]))
    s["q"] = (2 * torch.randn(sum(s["qlens"]), nq * d, **dev)).to(torch.bfloat16)
    kv = torch.randn(sum(s["klens"]), 2 * nkv * d, dtype=torch.bfloat16, **dev)    # one packed projection of the states
    s["k"], s["v"] = kv[:, :nkv * d], kv[:, nkv * d:]
    s["o"] = torch.zeros_like(s["q"])
    if own:
        size = s["Q"].h3enc_op_attention_cross_workspace_bytes(d)
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- one pass

def run(s):
    return {"append": _run_append, "shared": _run_shared, "cross": _run_cross}[s["c"]["op"]](s)


def _frequencies(c):
    """The scaled rotary frequencies [rot / 2] in 64 bits, and the factor on cos and sin."""
    rot, f = c["rot"], c["factor"]
    j = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    w = THETA ** (-2 * j / rot)
    if c["scaling"] == "linear":
        return w / f, 1.0
    if c["scaling"] == "wavelength":     # whole above 4 turns in the original context, stretched below 1
        keep = ((ORIGINAL * w / (2 * math.pi) - 1) / 3).clamp(0, 1)
        return w * (keep + (1 - keep) / f), 1.0
    if c["scaling"] == "yarn":           # whole for the dimensions of more than 32 turns, stretched below 1
        def dim(turns):
            return rot * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(THETA))
        low, high = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), rot - 1)
        ramp = ((j - low) / max(high - low, 1e-3)).clamp(0, 1)
        return w * (1 - ramp) + w / f * ramp, 0.1 * math.log(f) + 1
    return w, 1.0


def _run_append(s):
    c = s["c"]
    T, live, nq, nkv, d, page, rot = s["T"], s["live"], c["nq"], c["nkv"], c["d"], c["page"], c["rot"]
    out = {"q": s["q_out"], "k_cache": s["k"], "v_cache": s["v"]}
    if c["k_out"]:
        out["k"] = s["k_out"]
    if own:
        s["Q"].h3enc_op_rope_append(s["qkv"], T, nq, nkv, d, s["w_q"], s["w_k"], EPS, s["rope"], s["positions"],
                                    s["q_out"], s["k_out"], cache=s["cache"], page_table=s["table"],
                                    seq_lens=s["lens"], max_len=s["max_len"], cu_rows=None if s["one"] else s["cu"])
        return out
    cu = s["cu"].long()
    t = torch.arange(live, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    place = s["lens"].long()[seq] - cu[seq + 1] + t
    w, magnitude = _frequencies(c)
    if c["axes"] == 3:
        j, sec = torch.arange(rot // 2, device="cuda"), _section(rot)
        axis = torch.where((j % 3 == 1) & (j < 3 * sec[1]), 1, torch.where((j % 3 == 2) & (j < 3 * sec[2]), 2, 0))
        angle = s["positions"][:, :live].double().T[:, axis] * w
    else:
        angle = place.double()[:, None] * w
    cos, sin = (magnitude * angle.cos()).float()[:, None], (magnitude * angle.sin()).float()[:, None]

    def rotate(x, weight):
        x = x.float()
        if weight is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
        y = x.clone()
        a, b = (x[..., :rot:2], x[..., 1:rot:2]) if c["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        if c["inter"]:
            y[..., :rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y

    x = s["qkv"].view(T, nq + 2 * nkv, d)[:live]
    s["q_out"][:live].view(live, nq, d).copy_(rotate(x[:, :nq], s["w_q"]))
    k = rotate(x[:, nq:nq + nkv], s["w_k"])
    if c["k_out"]:
        s["k_out"][:live].view(live, nkv, d).copy_(k)
    pages, at = s["table"].long()[seq, place // page], place % page
    for src, pool, scale in ((k, s["k"], s["k_scale"]), (x[:, nq + nkv:].float(), s["v"], s["v_scale"])):
        if scale is None:
            pool[pages, :, at] = src.to(torch.bfloat16)
        else:
            pool.view(torch.uint8)[pages, :, at] = _e4m3(src / scale[:, None]).view(torch.uint8)
    return out


def _gathered(pool, scale, table, c):
    """[rows of the table, nkv, places, d] in 32 bits."""
    x = pool.view(torch.uint8)[table.long()].view(pool.dtype) if scale is not None else pool[table.long()]
    x = x.permute(0, 2, 1, 3, 4).reshape(table.shape[0], c["nkv"], -1, c["d"]).float()
    return x if scale is None else x * scale[:, None, None]


def _run_shared(s):
    c = s["c"]
    n, nq, nkv, d = c["n"], c["nq"], c["nkv"], c["d"]
    out = {"o": s["o"]}
    if c["weights"]:
        out["weight"] = s["weight_out"]
    if own:
        s["Q"].h3enc_op_attention_decode_shared(s["q"], s["o"], s["cache"], s["prefix_table"], s["prefix_lens"], c["phi"],
                                                s["table"], s["lens"], nq, c["hi"], s["workspace"],
                                                prefix_rows=s["prefix_rows"], weight_in=s["weight"],
                                                weight_out=s["weight_out"])
        return out
    q = s["q"].view(n, nkv, nq // nkv, d).float() / math.sqrt(d)
    k, v = (_gathered(s[x], s[x + "_scale"], s["table"], c) for x in "kv")
    mask = torch.arange(k.shape[2], device="cuda")[None] < s["lens"][:, None]
    own_scores = torch.matmul(q, k.transpose(2, 3)).masked_fill(~mask[:, None, None], -math.inf)
    pk, pv = (_gathered(s[x], s[x + "_scale"], s["prefix_table"], c) for x in "kv")
    for i, (a, b) in enumerate(zip(s["first"], s["first"][1:])):
        if a == b:
            continue
        # the prefix's keys are read once for all rows of the group
        rows = q[a:b].transpose(0, 1).reshape(nkv, -1, d)
        there = torch.arange(pk.shape[2], device="cuda") < s["prefix_lens"][i]
        sc = torch.matmul(rows, pk[i].transpose(1, 2)).masked_fill(~there, -math.inf)
        mine = own_scores[a:b].transpose(0, 1).reshape(nkv, rows.shape[1], -1)
        top = torch.maximum(sc.amax(-1, keepdim=True), mine.amax(-1, keepdim=True))
        p, pm = torch.exp(sc - top), torch.exp(mine - top)
        total = p.sum(-1, keepdim=True) + pm.sum(-1, keepdim=True)
        pm = (pm / total).view(nkv, b - a, nq // nkv, -1).transpose(0, 1)
        o = torch.matmul(p / total, pv[i]).view(nkv, b - a, nq // nkv, d).transpose(0, 1) + torch.matmul(pm, v[a:b])
        s["o"][a:b].view(b - a, nkv, nq // nkv, d).copy_(o)
        if c["weights"]:
            w = s["weight"][a:b] + pm.sum((1, 2))[:, :c["hi"]]
            s["weight_out"][a:b] = torch.where(mask[a:b, :c["hi"]], w, s["weight_out"][a:b])
    return out


def _run_cross(s):
    c = s["c"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    if own:
        s["Q"].h3enc_op_attention_cross(s["q"], s["k"], s["v"], s["o"], nq, nkv, d, s["workspace"], cu_q=s["cu_q"],
                                        cu_k=s["cu_k"])
        return {"o": s["o"]}
    group, q0, k0 = nq // nkv, 0, 0
    for m, length in zip(s["qlens"], s["klens"]):
        q = s["q"][q0:q0 + m].view(m, nkv, group, d).permute(1, 2, 0, 3).reshape(nkv, group * m, d).float() / math.sqrt(d)
        k, v = (x[k0:k0 + length].view(length, nkv, d).transpose(0, 1).float() for x in (s["k"], s["v"]))
        if length:
            sc = torch.matmul(q, k.transpose(1, 2))
            p = torch.exp(sc - sc.amax(-1, keepdim=True))
            o = torch.matmul(p / p.sum(-1, keepdim=True), v)
        else:
            o = torch.zeros_like(q)
        s["o"][q0:q0 + m].view(m, nkv, group, d).copy_(o.view(nkv, group, m, d).permute(2, 0, 1, 3))
        q0, k0 = q0 + m, k0 + length
    return {"o": s["o"]}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """From the definitions, a head or a sequence at a time, in float64."""
    return {"append": _exact_append, "shared": _exact_shared, "cross": _exact_cross}[case["op"]](prepare(case, seed))


def _exact_append(s):
    c = s["c"]
    nq, nkv, d, page, rot = c["nq"], c["nkv"], c["d"], c["page"], c["rot"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    rows = [(b, lens[b] - (cu[b + 1] - t)) for b in range(c["n"]) for t in range(cu[b], cu[b + 1])]
    place = torch.tensor([p for _, p in rows], device="cuda")
    freq, magnitude = [], 1.0
    for j in range(rot // 2):
        w = math.exp(-math.log(THETA) * 2 * j / rot)
        if c["scaling"] == "linear":
            w /= c["factor"]
        elif c["scaling"] == "wavelength":
            turns = ORIGINAL / (2 * math.pi / w)
            if turns < 1:
                w /= c["factor"]
            elif turns < 4:
                w = (turns - 1) / 3 * w + (4 - turns) / 3 * w / c["factor"]
        elif c["scaling"] == "yarn":
            ends = [rot / 2 * math.log(ORIGINAL / (2 * math.pi * turns), THETA) for turns in (32, 1)]
            low, high = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rot - 1)
            part = min(max((j - low) / (high - low if high > low else 1e-3), 0.0), 1.0)
            w *= part / c["factor"] + 1 - part
            magnitude = 1 + math.log(c["factor"]) / 10
        freq.append(w)
    if c["axes"] == 3:
        sec = _section(rot)
        axis = [j % 3 if j % 3 and j < 3 * sec[j % 3] else 0 for j in range(rot // 2)]
        angle = torch.stack([s["positions"][a, :s["live"]].double() * w for a, w in zip(axis, freq)], 1)
    else:
        angle = torch.stack([place.double() * w for w in freq], 1)
    turn = torch.polar(torch.full_like(angle, magnitude), angle)
    x = s["qkv"][:s["live"]].double()
    heads = []
    for h in range(nq + nkv):
        v = x[:, h * d:(h + 1) * d].clone()
        w = s["w_q"] if h < nq else s["w_k"]
        if w is not None:
            v = v * w.double() * (v.square().sum(1, keepdim=True) / d + EPS).rsqrt()
        if c["inter"]:
            z = torch.view_as_complex(v[:, :rot].reshape(-1, rot // 2, 2).contiguous()) * turn
            v[:, :rot] = torch.view_as_real(z).reshape(-1, rot)
        else:
            z = torch.complex(v[:, :rot // 2].contiguous(), v[:, rot // 2:rot].contiguous()) * turn
            v[:, :rot] = torch.cat([z.real, z.imag], 1)
        heads.append(v)
    out = {"q": torch.zeros(s["T"], nq * d, dtype=torch.float64, device="cuda")}
    out["q"][:s["live"]] = torch.cat(heads[:nq], 1)
    k, v = torch.stack(heads[nq:], 1), x[:, (nq + nkv) * d:].view(-1, nkv, d)
    at = torch.tensor([b for b, _ in rows], device="cuda")
    flat_at = s["table"][at, place // page].long() * page + place % page
    for name, pool, val, scale in (("k_cache", s["k"], k, s["k_scale"]), ("v_cache", s["v"], v, s["v_scale"])):
        flat = pool.double().transpose(1, 2).reshape(-1, nkv, d)
        flat[flat_at] = val if scale is None else (val / scale.double()[:, None]).clamp(-448, 448)
        out[name] = flat.view(-1, page, nkv, d).transpose(1, 2).contiguous()
    if c["k_out"]:
        out["k"] = torch.zeros(s["T"], nkv * d, dtype=torch.float64, device="cuda")
        out["k"][:s["live"]] = k.reshape(-1, nkv * d)
    return out


def _exact_shared(s):
    c = s["c"]
    nq, nkv, d, page = c["nq"], c["nkv"], c["d"], c["page"]
    m = nq // nkv
    o = torch.zeros(c["n"], nq, d, dtype=torch.float64, device="cuda")
    weight = s["weight_out"].double() if c["weights"] else None
    lens, plens = s["lens"].tolist(), s["prefix_lens"].tolist()

    def tokens(table, length, h, name):
        x = s[name][table[:-(-length // page)].long(), h].double().reshape(-1, d)[:length]
        return x if s[name + "_scale"] is None else x * s[name + "_scale"][h].double()

    for i, (a, e) in enumerate(zip(s["first"], s["first"][1:])):
        for h in range(nkv):
            pk, pv = (tokens(s["prefix_table"][i], plens[i], h, x) for x in "kv")
            for b in range(a, e):
                k, v = (torch.cat([p, tokens(s["table"][b], lens[b], h, x)]) for p, x in ((pk, "k"), (pv, "v")))
                p = torch.softmax(k @ s["q"][b].view(nq, d)[h * m:(h + 1) * m].double().T * d ** -0.5, dim=0)
                o[b, h * m:(h + 1) * m] = p.T @ v
                if c["weights"]:
                    weight[b, :lens[b]] = (weight if h else s["weight"].double())[b, :lens[b]] + p[plens[i]:].sum(1)
    out = {"o": o.view(c["n"], nq * d)}
    if c["weights"]:
        out["weight"] = weight
    return out


def _exact_cross(s):
    c = s["c"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for m, length in zip(s["qlens"], s["klens"]):
        for h in range(nq if length else 0):
            g = h // (nq // nkv)
            k, v = (x[k0:k0 + length, g * d:(g + 1) * d].double() for x in (s["k"], s["v"]))
            q = s["q"][q0:q0 + m, h * d:(h + 1) * d].double()
            o[q0:q0 + m, h * d:(h + 1) * d] = torch.softmax(q @ k.T * d ** -0.5, dim=1) @ v
        q0, k0 = q0 + m, k0 + length
    return {"o": o}
