"""Float64 oracle of the serving operators (paged 8-bit cache, attention over it, low-rank adapters),
in plain numpy from their definitions.  Shares no code with the library."""
from __future__ import annotations

import numpy as np


def rotate(x, cos, sin, interleaved):
    """x [T, H, D] float64; cos, sin [T, half]: the pairs of the first 2 * half values turned."""
    x = np.asarray(x, dtype=np.float64)
    half = cos.shape[1]
    out = x.copy()
    a = np.arange(half) * (2 if interleaved else 1)
    b = a + 1 if interleaved else a + half
    c, s = np.asarray(cos, np.float64)[:, None], np.asarray(sin, np.float64)[:, None]
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def append(codes, scale, x, page_table, start, cu):
    """One half (keys, already rotated, or values) appended to copies of codes [pages, heads, page,
    dim] and scale [pages, heads].  Returns (ideal, new scale): ideal holds, in float64, what each
    written code is the rounding of (clipped to +-127) and the codes elsewhere."""
    ideal, scale = np.asarray(codes, np.float64).copy(), np.asarray(scale, np.float64).copy()
    before = scale.copy()
    page = codes.shape[2]
    for b in range(len(start)):
        n, s = int(cu[b + 1] - cu[b]), int(start[b])
        if n <= 0:
            continue
        for j in range(s // page, (s + n - 1) // page + 1):
            if j >= page_table.shape[1]:
                continue
            p = int(page_table[b, j])
            if p < 0 or p >= codes.shape[0]:
                continue
            lo, hi = max(s, j * page), min(s + n, (j + 1) * page)
            new = np.asarray(x[cu[b] + lo - s:cu[b] + hi - s], np.float64).transpose(1, 0, 2)   # [heads, t, dim]
            had = before[p] if j * page < s else np.zeros_like(before[p])
            mag = np.where(np.isfinite(new), np.abs(new), 0.0)
            unit = np.maximum(had, mag.max((1, 2)) / 127.0)
            with np.errstate(all="ignore"):
                fresh = np.clip(np.where(unit[:, None, None] > 0, new / unit[:, None, None], 0.0), -127, 127)
            fresh[np.isnan(new)] = 0.0
            keep = slice(0, max(s - j * page, 0))
            grow = unit > had
            ratio = np.divide(had, unit, out=np.zeros_like(unit), where=unit > 0)
            ideal[p, grow, keep] *= ratio[grow, None, None]
            ideal[p, :, lo - j * page:hi - j * page] = fresh
            scale[p] = unit
    return ideal, scale


def values(codes, scale, page_table, b, length):
    """Cached values [length, heads, dim] of sequence b and which tokens are present."""
    page = codes.shape[2]
    out = np.zeros((length, codes.shape[1], codes.shape[3]))
    there = np.zeros(length, bool)
    for t in range(length):
        j = t // page
        p = int(page_table[b, j]) if j < page_table.shape[1] else -1
        if 0 <= p < codes.shape[0]:
            out[t] = codes[p, :, t % page].astype(np.float64) * scale[p].astype(np.float64)[:, None]
            there[t] = True
    return out, there


def attention(q, k_codes, v_codes, k_scale, v_scale, page_table, kv_len, cu, scale, causal=True, window=0):
    """(out, weight, most): out [T, Hq, D]; weight = sum_j p_j |v_j| and most [T, Hq] = the largest
    sum_d |q_d k_d| * scale that a query meets (both bound the error of finite arithmetic)."""
    q = np.asarray(q, np.float64)
    group = q.shape[1] // k_codes.shape[1]
    out, weight, most = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2])
    for b in range(len(kv_len)):
        n, length = int(cu[b + 1] - cu[b]), int(kv_len[b])
        if n <= 0 or length <= 0:
            continue
        k, there = values(k_codes, k_scale, page_table, b, length)
        v, _ = values(v_codes, v_scale, page_table, b, length)
        pos = np.arange(length)
        for i in range(n):
            at = length - n + i
            see = there.copy()
            if causal:
                see &= pos <= at
            if window > 0:
                see &= pos > at - window
            if not see.any():
                continue
            kk, vv = k[see], v[see]
            for h in range(q.shape[1]):
                row = q[cu[b] + i, h]
                s = kk[:, h // group] @ row * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[cu[b] + i, h] = p @ vv[:, h // group]
                weight[cu[b] + i, h] = p @ np.abs(vv[:, h // group])
                most[cu[b] + i, h] = (np.abs(kk[:, h // group]) @ np.abs(row)).max() * abs(scale)
    return out, weight, most


def lora(y, x, a, b, scale, ids):
    """(out, low weight): y + scale * B (A x), and scale * |B| (|A| |x|)."""
    y, x, a, b = (np.asarray(t, np.float64) for t in (y, x, a, b))
    out, weight = y.copy(), np.zeros_like(y)
    for m, i in enumerate(ids):
        if 0 <= i < a.shape[0]:
            out[m] += float(scale[i]) * (b[i] @ (a[i] @ x[m]))
            weight[m] = abs(float(scale[i])) * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[m])))
    return out, weight
