"""fp64 oracle of the serving operators: rotary positions, the paged cache and attention over it.

Plain numpy in fp64, written from the definitions; it shares no code with the CUDA path.  A cache is
given as numpy arrays: codes as fp64 values [pages, h_kv, page_size, d] with fp64 scales
[pages, h_kv, page_size] (or None), a page table and lengths as integers.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -60


def inv_freq(rot, base=10000.0, scaling="none", factor=1.0, original_context=0.0, beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair, and the factor on the rotated values."""
    out, att = [], 1.0
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
        f = b ** (-2 * i / rot)
        if scaling == "linear":
            f = f / factor
        if scaling == "yarn":
            r = original_context * f / (2 * math.pi)
            g = min(1.0, max(0.0, (r - beta_slow) / (beta_fast - beta_slow)))
            f = g * f + (1 - g) * f / factor
            att = 0.1 * math.log(factor) + 1.0
        out.append(f)
    return np.array(out), att


def rotate(x, positions, freqs, interleaved=False, factor=1.0, inverse=False):
    """x [b, h, s, d] at positions [b, s].  Returns (y, reach): reach is |a| + |b| of each rotated
    element's pair (0 for the others), the scale of its fp32 rounding errors."""
    y, reach = x.copy(), np.zeros_like(x)
    n = len(freqs)
    t = positions[:, None, :, None] * freqs * (-1.0 if inverse else 1.0)
    c, s = factor * np.cos(t), factor * np.sin(t)
    ia = np.arange(n) * 2 if interleaved else np.arange(n)
    ib = ia + (1 if interleaved else n)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    reach[..., ia] = reach[..., ib] = (np.abs(a) + np.abs(b)) * abs(factor)
    return y, reach


def row_scale(x):
    """Scale of each row of an E4M3 cache (NaN where a row holds one, infinite where an infinity)."""
    amax = np.abs(x).max(-1)
    return np.where(amax < AMAX_MIN, AMAX_MIN, amax) / E4M3_MAX


def slots(page_table, page_size, num_pages, lens_kv, lens_q, s):
    """(sequence, row, page, slot) of every row that a write stores."""
    out = []
    for i in range(len(lens_kv)):
        n = min(max(lens_kv[i], 0), page_table.shape[1] * page_size)
        m = min(max(lens_q[i], 0), s) if lens_q is not None else s
        for r in range(m):
            pos = n - m + r
            if 0 <= pos < n and 0 <= page_table[i, pos // page_size] < num_pages:
                out.append((i, r, int(page_table[i, pos // page_size]), pos % page_size))
    return out


def dense(values, scales, page_table, i, n):
    """Positions 0..n-1 of sequence i as [h, n, d] in fp64, and which of them exist."""
    pages, h, ps, d = values.shape
    at = np.arange(n)
    page = page_table[i, at // ps]
    live = (page >= 0) & (page < pages)
    x = values[np.where(live, page, 0), :, at % ps]                    # [n, h, d]
    if scales is not None:
        x = x * scales[np.where(live, page, 0), :, at % ps][..., None]
    return np.where(live[:, None, None], x, 0.0).transpose(1, 0, 2), live


def attend(q, k_values, v_values, k_scales, v_scales, page_table, lens_kv, lens_q, scale, causal=False, tree=None):
    """O, LSE, spread = sum_j P_j |v_j| (the scale of O's weight errors) of q [b, h_q, s, d], and reach =
    sum_j P_j |scale| sum_d |q_d k_jd|, the scale of LSE's errors from the sums of the scores.
    tree: bool [b, s, s] (row i sees drafted token j), or None."""
    b, h_q, s, d = q.shape
    h_kv, ps = k_values.shape[1], k_values.shape[2]
    o, spread = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((b, h_q, s), -np.inf)
    reach = np.zeros((b, h_q, s))
    for i in range(b):
        n = min(max(lens_kv[i], 0), page_table.shape[1] * ps)
        m = min(max(lens_q[i], 0), s) if lens_q is not None else s
        if n == 0:
            continue
        k, live = dense(k_values, k_scales, page_table, i, n)
        v, _ = dense(v_values, v_scales, page_table, i, n)
        j = np.arange(n) - (n - m)
        for r in range(m):
            see = live.copy()
            if causal:
                see &= j <= r
            if tree is not None:
                see &= (j < 0) | tree[i, r, np.clip(j, 0, s - 1)]
            if not see.any():
                continue
            for h in range(h_q):
                x = scale * (k[h * h_kv // h_q][see] @ q[i, h, r])
                big = x.max()
                p = np.exp(x - big)
                l = p.sum()
                vv = v[h * h_kv // h_q][see]
                o[i, h, r] = p @ vv / l
                spread[i, h, r] = p @ np.abs(vv) / l
                lse[i, h, r] = big + math.log(l)
                reach[i, h, r] = abs(scale) * (p @ (np.abs(k[h * h_kv // h_q][see]) @ np.abs(q[i, h, r]))) / l
    return o, lse, spread, reach
