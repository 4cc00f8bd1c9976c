"""The steps of a decoder that reads an encoder's states, restated for the CPU oracle in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Rotary frequencies and their scalings, rows
appended to a cache, attention behind a shared prefix and cross attention are this library's own,
defined in ``include/h3enc_ops.h``.  Pinned by ``tests/test_decoder_cpu.py``.
"""
from __future__ import annotations

import math

import numpy as np

from .decode import attend_one

__all__ = ["frequencies", "axis_of", "rotate", "append_places", "attend_prefix", "cross"]


def frequencies(rot, theta, scaling="none", factor=1.0, original_len=0, low_turns=0.0, high_turns=0.0, magnitude=0.0):
    """(w [rot / 2], the factor on cos and sin)."""
    if not low_turns and not high_turns:
        low_turns, high_turns = 1.0, 32.0 if scaling == "yarn" else 4.0
    out = []
    for j in range(rot // 2):
        w = theta ** (-2.0 * j / rot)
        if scaling == "linear":
            w = w / factor
        elif scaling == "wavelength":
            turns = original_len * w / (2 * math.pi)
            s = min(max((turns - low_turns) / (high_turns - low_turns), 0.0), 1.0)
            w = s * w + (1 - s) * w / factor
        elif scaling == "yarn":
            a, e = (rot * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (high_turns, low_turns))
            a, e = max(math.floor(a), 0), min(math.ceil(e), rot - 1)
            s = min(max((j - a) / max(e - a, 0.001), 0.0), 1.0)
            w = (1 - s) * w + s * w / factor
        out.append(w)
    if not magnitude:
        magnitude = 0.1 * math.log(factor) + 1 if scaling == "yarn" and factor > 1 else 1.0
    return np.array(out), magnitude


def axis_of(j, section):
    """Which of the three axes of the positions pair j goes by."""
    return j % 3 if j % 3 and j < 3 * section[j % 3] else 0


def rotate(x, angle, magnitude, interleaved):
    """x [T, heads, d], angle [T, rot / 2]: the first rot elements of every head rotated."""
    y = np.array(x, np.float64)
    half = angle.shape[1]
    turn = (magnitude * np.exp(1j * angle))[:, None]
    if interleaved:
        z = (y[..., 0:2 * half:2] + 1j * y[..., 1:2 * half:2]) * turn
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
    else:
        z = (y[..., :half] + 1j * y[..., half:2 * half]) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def append_places(T, seq_lens, cu_rows):
    """(sequence, place) of every row, or None for a row of no sequence."""
    out = [None] * T
    for b, length in enumerate(seq_lens):
        first, end = (b, b + 1) if cu_rows is None else (cu_rows[b], cu_rows[b + 1])
        for t in range(first, min(end, T)):
            out[t] = b, length - (end - t)
    return out


def attend_prefix(q, prefix_k, prefix_v, k, v):
    """One token's q [nq, d] over a prefix and its own tokens: (o, the weights of the own tokens [nq, L])."""
    o, p = attend_one(q, np.concatenate([prefix_k, k]), np.concatenate([prefix_v, v]))
    return o, p[:, len(prefix_k):]


def cross(q, k, v):
    """q [M, nq, d] over k, v [L, nkv, d]: every query sees every state; L = 0 gives zeros."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    (_, nq, d), (n, nkv, _) = q.shape, k.shape
    o = np.zeros(q.shape)
    for h in range(nq if n else 0):
        g = h // (nq // nkv)
        s = q[:, h] @ k[:, g].T / math.sqrt(d)
        e = np.exp(s - s.max(1, keepdims=True))
        o[:, h] = e @ v[:, g] / e.sum(1, keepdims=True)
    return o
