"""Rotary positions and latent attention in float64.

A plain restatement of the definitions in ``include/attn.h``, in NumPy.  It
shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from . import paged_ref as P


def frequencies(rot, base=10000.0, scaling="NONE", factor=1.0, trained_len=1, turns=(1.0, 32.0)):
    """Radians a position of every pair."""
    out = []
    for p in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "BASE" else base
        f = b ** (-2.0 * p / rot)
        if scaling == "LINEAR":
            f /= factor
        if scaling == "TURNS":
            t = trained_len * f / (2 * math.pi)
            w = min(1.0, max(0.0, (t - turns[0]) / (turns[1] - turns[0])))
            f *= w + (1 - w) / factor
        out.append(f)
    return np.array(out)


def rope_table(rope_len, freq, magnitude=1.0):
    ang = np.arange(rope_len, dtype=np.float64)[:, None] * freq
    return magnitude * np.cos(ang), magnitude * np.sin(ang)


def turn(x, cos, sin, start=0, interleaved=False, inverse=False):
    """x [tokens, heads, d]; cos, sin [tokens, rot / 2]: the rot coordinates from
    `start` on turned by each token's angles (back, if inverse)."""
    half = cos.shape[1]
    y = np.array(x, np.float64)
    s = -sin if inverse else sin
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        a, b = x[..., start + i], x[..., start + j]
        y[..., start + i] = a * cos[:, p, None] - b * s[:, p, None]
        y[..., start + j] = b * cos[:, p, None] + a * s[:, p, None]
    return y


def expand(kv, k_rope, cos, sin, d_n, interleaved=False):
    """K [tokens, H, d_n + d_r], V [tokens, H, d_v]."""
    pe = turn(k_rope[:, None], cos, sin, interleaved=interleaved)
    k = np.concatenate([kv[..., :d_n], np.repeat(pe, kv.shape[1], axis=1)], -1)
    return k, np.array(kv[..., d_n:])


def expand_bwd(dk, dv, cos, sin, d_n, interleaved=False):
    """Gradients of kv and k_rope."""
    dkv = np.concatenate([dk[..., :d_n], dv], -1)
    pe = dk[..., d_n:].sum(1, keepdims=True)
    return dkv, turn(pe, cos, sin, interleaved=interleaved, inverse=True)[:, 0]


def attend(q, rows_of, d_c, seq_lens, cu, scale, **kw):
    """q [tokens, H, d_c + d_r]; rows_of(s): [len, d_c + d_r] of sequence s.  As
    paged_ref.attend with one KV head whose value is the key's first part."""
    return P.attend(q, lambda s: rows_of(s)[None], lambda s: rows_of(s)[None, :, :d_c], seq_lens,
                    cu, scale, **kw)
