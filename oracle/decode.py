"""Decoding from a key/value cache, restated for the CPU oracle in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).  The pages stop at the
prefill: the norm and rotation restate ``MiniMaxH3Qwen3VLTextAttention.forward``
(page "vllm-omni vllm_omni/diffusion/models/minimax_h3/encoder.py"); the cache,
the attention of a single token and the eviction are this library's own, defined
in ``include/h3enc_ops.h``.  Pinned by ``tests/test_decode_cpu.py``.
"""
from __future__ import annotations

import numpy as np

__all__ = ["head_norm_rope", "attend_one", "keep_heaviest"]


def head_norm_rope(x, w, eps, cos, sin):
    """x [T, heads, d]: RMSNorm over d with weight w (None: none), then the rotation by the
    tables cos / sin [T, d/2] (None: none)."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    if cos is not None:
        h = x.shape[-1] // 2
        c, s = np.asarray(cos, np.float64)[:, None], np.asarray(sin, np.float64)[:, None]
        a, b = x[..., :h], x[..., h:]
        x = np.concatenate([a * c - b * s, b * c + a * s], axis=-1)
    return x


def attend_one(q, k, v):
    """One token's q [nq, d] over k, v [L, nkv, d]: (o [nq, d], p [nq, L]); L = 0 gives zeros."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    nq, d = q.shape
    n, nkv = k.shape[:2]
    o, p = np.zeros((nq, d)), np.zeros((nq, n))
    for h in range(nq if n else 0):
        g = h // (nq // nkv)
        s = k[:, g] @ q[h] / np.sqrt(d)
        e = np.exp(s - s.max())
        p[h] = e / e.sum()
        o[h] = p[h] @ v[:, g]
    return o, p


def keep_heaviest(weight, length, budget, sink, recent):
    """The kept indices, ascending: all if length <= budget, else the first `sink`, the last
    `recent` and the heaviest of the others (ties: the earlier; NaN: the lightest)."""
    if length <= budget:
        return list(range(length))
    held = set(range(sink)) | set(range(length - recent, length))
    rest = [i for i in range(length) if i not in held]
    rest.sort(key=lambda i: (-weight[i] if weight[i] == weight[i] else np.inf, weight[i] != weight[i], i))
    return sorted(held | set(rest[:budget - len(held)]))
