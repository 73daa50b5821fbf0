"""fp64 numpy oracle of the operators around the attention kernels: the per-head RMS norm with the position
rotation (forward and backward), the paged key-value cache, and one-token attention over it.  Written from the
definitions, sharing no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def _angles(cos_sin, positions, rot):
    cs = np.asarray(cos_sin, np.float64)[np.asarray(positions)]
    return cs[:, None, :rot // 2], cs[:, None, rot // 2:]


def _pair_index(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def norm_rope(x, weight, cos_sin, positions, eps, interleaved):
    """R(pos) diag(weight) x / rms(x) for x [tokens, heads, d]; padding (pos < 0) gives 0, pos >= max_pos NaN."""
    x = np.asarray(x, np.float64)
    pos, rot = np.asarray(positions), cos_sin.shape[1]
    inside = (pos >= 0) & (pos < cos_sin.shape[0])
    y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    c, s = _angles(cos_sin, np.where(inside, pos, 0), rot)
    a, b = _pair_index(rot, interleaved)
    out = y.copy()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    out[pos >= cos_sin.shape[0]] = np.nan
    out[pos < 0] = 0.0
    return out


def norm_rope_grad(x, weight, cos_sin, positions, dout, eps, interleaved):
    """(dx, dweight, sum of the absolute products dweight is made of) of sum(norm_rope(x) * dout).  The last counts the rotation's two
    products apart, since rounding errors scale with them even where they cancel."""
    x, dout, w = (np.asarray(t, np.float64) for t in (x, dout, weight))
    pos, rot, d = np.asarray(positions), cos_sin.shape[1], x.shape[-1]
    keep = (pos >= 0)[:, None, None]
    c, s = _angles(cos_sin, np.maximum(pos, 0), rot)
    a, b = _pair_index(rot, interleaved)
    g = dout.copy()
    g[..., a] = dout[..., a] * c + dout[..., b] * s
    g[..., b] = dout[..., b] * c - dout[..., a] * s
    size = np.abs(dout)
    size[..., a] = np.abs(dout[..., a] * c) + np.abs(dout[..., b] * s)
    size[..., b] = np.abs(dout[..., b] * c) + np.abs(dout[..., a] * s)
    rms = np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    terms, size = np.where(keep, g * x / rms, 0.0), np.where(keep, size * np.abs(x) / rms, 0.0)
    h = g * w
    dx = np.where(keep, h / rms - x * (h * x).sum(-1, keepdims=True) / (d * rms ** 3), 0.0)
    return dx, terms.sum((0, 1)), size.sum((0, 1))


def e4m3_values():
    """The non-negative finite e4m3 values in code order (code 0 .. 126)."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


def quantise_row(row):
    """(codes uint8 [d], byte) of one row: the smallest n >= -126 with max|x| <= 448 * 2^n, nearest codes, ties to even."""
    row = np.asarray(row, np.float64)
    if not np.isfinite(row).all():
        return np.full(row.shape, 0x7f, np.uint8), 127
    top, n = np.abs(row).max(), -126
    while top > 448.0 * 2.0 ** n:
        n += 1
    grid, codes = e4m3_values(), np.zeros(row.shape, np.uint8)
    for i, x in enumerate(row):
        z = abs(x) / 2.0 ** n
        dist = np.abs(grid - z)
        best = np.flatnonzero(dist == dist.min())
        code = best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]
        codes[i] = code | (0x80 if np.signbit(x) else 0)
    return codes, n + 127


def stored_values(codes, byte):
    """What codes [..., d] with exponent bytes [...] stand for; byte 0, which no write stores, stands for 0."""
    codes = np.asarray(codes)
    mag = np.append(e4m3_values(), np.nan)[codes & 0x7f]
    return np.where(codes & 0x80, -mag, mag) * np.where(np.asarray(byte) == 0, 0.0, 2.0 ** (np.asarray(byte, np.float64) - 127))[..., None]


def gather_rows(values, page_table_row, start, end):
    """Rows [start, end) of one sequence, [n, hkv, d], of values [pages, hkv, page, d]."""
    page = values.shape[2]
    rows = [values[page_table_row[j // page], :, j % page] for j in range(start, end)]
    return np.stack(rows) if rows else np.zeros((0, values.shape[1], values.shape[3]))


def decode(q, k, v, scale, sink=None):
    """One token's attention: q [hq, d], k, v [n, hkv, d] -> out [hq, d], lse [hq], sum_j p_j |v_j| [hq, d], and
    max_j sum_i |scale q_i k_ji| [hq] (what rounding errors of the scores scale with)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    hq, d = q.shape
    g = hq // k.shape[1]
    out, lse, mass, size = np.zeros((hq, d)), np.full(hq, -np.inf), np.zeros((hq, d)), np.zeros(hq)
    for h in range(hq):
        kh, vh = k[:, h // g], v[:, h // g]
        z = scale * kh @ q[h]
        zs = z if sink is None else np.append(z, sink[h])
        if len(zs) == 0:
            continue
        m = zs.max()
        lse[h] = m if np.isinf(m) else m + np.log(np.exp(zs - m).sum())
        if len(z):
            p = np.exp(z - lse[h])
            out[h], mass[h] = p @ vh, p @ np.abs(vh)
            size[h] = np.abs(scale) * (np.abs(kh) @ np.abs(q[h])).max()
    return out, lse, mass, size
