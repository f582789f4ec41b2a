"""The paged KV cache in float64: rotation, E4M3 pages with a power-of-two
scale for each page and head, and attention over the pages.

A plain restatement of the definitions in ``include/attn.h``, token by token,
in NumPy.  It shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

MIN_EXP = -64
E4M3_MAX = 448.0


def e4m3_round(x):
    """Nearest E4M3 value (ties to even): three bits behind the leading one,
    steps of 2^-9 below 2^-6; infinities and NaN become NaN."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    _, e = np.frexp(np.maximum(a, 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    r = np.copysign(np.minimum(np.rint(a / step) * step, E4M3_MAX), x)
    return np.where(np.isfinite(x), r, np.nan)


def e4m3_values():
    """Values of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * np.exp2(e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def page_scale(x):
    """Smallest 2^e, e >= MIN_EXP, that brings every finite value to 448 or less."""
    a = np.abs(x)[np.isfinite(x)]
    amax = a.max() if a.size else 0.0
    e = MIN_EXP
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x, cos, sin, interleaved):
    """x [heads, dim]; cos, sin [rot / 2]: pair p turned by its angle."""
    half = len(cos)
    y = np.array(x, np.float64)
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        y[:, i] = x[:, i] * cos[p] - x[:, j] * sin[p]
        y[:, j] = x[:, j] * cos[p] + x[:, i] * sin[p]
    return y


def new_rows(seq_lens, cu):
    """[(sequence, row, position)] of every new token."""
    out = []
    for s, n in enumerate(np.diff(cu)):
        out += [(s, cu[s] + i, seq_lens[s] - n + i) for i in range(n)]
    return out


def append(cache, scale, page_table, page, seq_lens, cu, x):
    """Writes x [tokens, Hkv, dim] (rotated already) into `cache` [pages, Hkv,
    page, dim] in place: values, or E4M3 code values when `scale` [pages, Hkv]
    is given."""
    for s, n in enumerate(np.diff(cu)):
        lo = seq_lens[s] - n
        for col in range(lo // page, (seq_lens[s] - 1) // page + 1 if n else 0):
            a, b = max(lo, col * page), min(seq_lens[s], (col + 1) * page)
            rows = x[cu[s] + a - lo:cu[s] + b - lo].transpose(1, 0, 2)
            pid, slot = page_table[s][col], a - col * page
            for h in range(cache.shape[1]):
                if scale is None:
                    cache[pid, h, slot:slot + b - a] = rows[h]
                    continue
                fit = page_scale(rows[h])
                if slot:
                    fit = max(fit, scale[pid, h])
                    cache[pid, h, :slot] = e4m3_round(cache[pid, h, :slot] * scale[pid, h] / fit)
                cache[pid, h, slot:slot + b - a] = e4m3_round(rows[h] / fit)
                scale[pid, h] = fit


def gather(cache, scale, table_row, page, length):
    """[Hkv, length, dim] values of one sequence."""
    hkv, dim = cache.shape[1], cache.shape[3]
    out = np.zeros((hkv, length, dim))
    for j in range(length):
        pid = table_row[j // page]
        v = cache[pid, :, j % page]
        out[:, j] = v if scale is None else v * scale[pid][:, None]
    return out


def attend(q, k_of, v_of, seq_lens, cu, scale, causal=True, window=-1, sink=None):
    """q [tokens, Hq, d]; k_of(s), v_of(s): [Hkv, len, dim] of sequence s.
    Returns O, LSE [Hq, tokens], and for error bounds A = sum_j P |V| and
    D = max_j sum_d |q k| * scale; rows of no sequence are NaN."""
    T, hq, _ = q.shape
    d_v = v_of(0).shape[2]
    o = np.full((T, hq, d_v), np.nan)
    lse = np.full((hq, T), np.nan)
    A, D = np.zeros((T, hq, d_v)), np.zeros((T, hq))
    for s, n in enumerate(np.diff(cu)):
        if n == 0:
            continue
        k, v = k_of(s), v_of(s)
        g = hq // k.shape[0]
        for i in range(n):
            row, pos = cu[s] + i, seq_lens[s] - n + i
            hi = min(seq_lens[s], pos + 1) if causal else seq_lens[s]
            lo = max(0, pos - window) if window >= 0 else 0
            for h in range(hq):
                kk, vv = k[h // g, lo:max(lo, hi)], v[h // g, lo:max(lo, hi)]
                sc = kk @ q[row, h] * scale
                logits = sc if sink is None else np.append(sc, sink[h])
                if logits.size == 0:
                    o[row, h], lse[h, row] = 0.0, -np.inf
                    continue
                m = logits.max()
                z = np.exp(logits - m).sum()
                p = np.exp(sc - m) / z
                o[row, h], lse[h, row] = p @ vv, m + np.log(z)
                if sc.size:
                    A[row, h] = p @ np.abs(vv)
                    D[row, h] = (np.abs(kk) @ np.abs(q[row, h])).max() * scale
    return o, lse, A, D
