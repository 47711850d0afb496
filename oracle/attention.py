"""Attention before the MoE layer (oracle; test infrastructure only): position
rotation, the paged key-value cache and masked softmax attention.

Rotation follows the operator's stated arithmetic (fp32 products and sums,
each rounded, then one rounding to bf16), so its results are exact bit
patterns; attention is float64 from the definition.  The FP8 cache holds, per
128 elements (or per row of a 64-element head), E4M3 codes and the power-of-
two scale of quant.act_quant.
"""

import numpy as np

from . import formats


def rotate(x, cos_sin, positions, offset=0, interleaved=False):
    """x [tokens, heads, dim] bf16 values (float) -> rotated, rounded to bf16
    (float32 values).  cos_sin [n, rot] float32; a position outside it gives NaN."""
    x = np.asarray(x, np.float32)
    n, rot = cos_sin.shape
    half = rot // 2
    positions = np.asarray(positions, np.int64)
    known = (positions >= 0) & (positions < n)
    row = np.where(known[:, None], cos_sin[np.where(known, positions, 0)], np.float32(np.nan)).astype(np.float32)
    c, s = row[:, None, :half], row[:, None, half:]
    part = x[..., offset:offset + rot]
    first = slice(0, None, 2) if interleaved else slice(0, half)
    second = slice(1, None, 2) if interleaved else slice(half, None)
    a, b = part[..., first], part[..., second]
    y = x.copy()
    z = y[..., offset:offset + rot]
    z[..., first] = a * c - b * s
    z[..., second] = b * c + a * s
    return formats.bf16_decode(formats.bf16_encode(y)).astype(np.float32) if not np.isnan(y).any() else _bf16_nan(y)


def _bf16_nan(y):
    bad = np.isnan(y)
    r = formats.bf16_decode(formats.bf16_encode(np.where(bad, np.float32(0), y))).astype(np.float32)
    return np.where(bad, np.float32(np.nan), r)


def cache_rows(pages, table, length):
    """Positions 0 .. length of a sequence: pages [n, heads, size, ...] -> [heads, length, ...]."""
    size = pages.shape[2]
    at = np.asarray(table[:-(-length // size)], np.int64)
    rows = np.moveaxis(pages[at], 1, 0)
    return rows.reshape(pages.shape[1], -1, *pages.shape[3:])[:, :length]


def fp8_values(codes, scales):
    """E4M3 codes [..., dim] and E8M0 bytes [..., groups] -> float64."""
    v = formats.e4m3_decode(codes)
    s = np.ldexp(1.0, np.asarray(scales).astype(np.int64) - 127)
    return (v.reshape(*s.shape, -1) * s[..., None]).reshape(v.shape)


def attend(q, k, v, first, scale, causal=True, window=0, hidden=None):
    """One sequence.  q [rows, heads, dim] at positions first + i; k, v
    [kv_heads, keys, dim]; hidden: keys left out for every row.  Returns out,
    lse, the sums sum_j p_j |v_j| and max_j scale sum_d |q_d k_jd| over kept j
    (for error bounds)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    rows, heads, dim = q.shape
    group = heads // k.shape[0]
    n = k.shape[1]
    out, absv = np.zeros(q.shape), np.zeros(q.shape)
    lse, size = np.full((rows, heads), -np.inf), np.zeros((rows, heads))
    pos = first + np.arange(rows)[:, None]
    j = np.arange(n)[None, :]
    keep = np.ones((rows, n), bool)
    if causal:
        keep &= j <= pos
    if window:
        keep &= j > pos - window
    if hidden is not None:
        keep &= ~hidden[None, :]
    for h in range(heads):
        kh, vh = k[h // group], v[h // group]
        s = scale * (q[:, h] @ kh.T)
        a = abs(scale) * (np.abs(q[:, h]) @ np.abs(kh).T)
        for i in range(rows):
            kept = keep[i]
            if not kept.any():
                continue
            m = s[i, kept].max()
            e = np.exp(s[i, kept] - m)
            t = e.sum()
            lse[i, h] = m + np.log(t)
            out[i, h] = (e / t) @ vh[kept]
            absv[i, h] = (e / t) @ np.abs(vh[kept])
            size[i, h] = a[i, kept].max()
    return out, lse, absv, size
