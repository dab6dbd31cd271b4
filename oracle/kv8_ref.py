"""float64 CPU oracle of the 8-bit cache operators (test infrastructure only).

Plain numpy restatements of the definitions: it shares no code, table or constant with the
CUDA path.  Caches are dense arrays here, values[b, h, position, 128]; paging is the
tests' business.
"""
from __future__ import annotations

import numpy as np

FMAX = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values():
    """The finite values of the 8-bit format with 4 exponent and 3 mantissa bits (bias 7),
    by byte: byte 0x7F and 0xFF are NaN."""
    out = np.empty(256)
    for byte in range(256):
        s, e, m = byte >> 7, byte >> 3 & 15, byte & 7
        if e == 15 and m == 7:
            v = np.nan
        elif e == 0:
            v = m / 8 * 2.0 ** -6
        else:
            v = (1 + m / 8) * 2.0 ** (e - 7)
        out[byte] = -v if s else v
    return out


def block_scale(a, fmt):
    """The smallest power of two S >= 2^-126 with a <= FMAX * S, elementwise."""
    a = np.asarray(a, np.float64)
    e = np.full(a.shape, -126)
    for _ in range(260):
        short = a > FMAX[fmt] * np.ldexp(1.0, e)
        if not short.any():
            break
        e = e + short
    return np.ldexp(1.0, e)


def round8(x, fmt):
    """Nearest value of the format, ties to even, the largest for anything beyond."""
    x = np.asarray(x, np.float64)
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127)
    _, e = np.frexp(np.abs(x))                      # |x| = m 2^e, 1/2 <= m < 1
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.rint(x / step) * step, -448, 448)


def append(stored, scale, new, start, fmt, block):
    """One sequence and kv head: stored [L, d] format values, scale [L / block]; rows new
    [n, d] at start.  Returns the new (stored, scale)."""
    stored, scale = stored.copy(), scale.copy()
    end = start + len(new)
    if len(new) == 0:
        return stored, scale
    for j in range(start // block, (end - 1) // block + 1):
        p0, p1 = max(start, j * block), min(end, (j + 1) * block)
        rows = new[p0 - start:p1 - start]
        a = np.abs(rows)
        s = float(block_scale(np.max(np.where(np.isfinite(a), a, 0.0)), fmt))
        if start > j * block:
            old = scale[j]
            if old > s:
                s = old
            if s != old:
                was = stored[j * block:start]
                stored[j * block:start] = round8(was * old / s, fmt)
        scale[j] = s
        stored[p0:p1] = round8(rows / s, fmt)
    return stored, scale


def attention(q, K, V, pos):
    """One query head over positions pos (in any order, repeats counted): (out, p).  Empty:
    zeros."""
    if len(pos) == 0:
        return np.zeros(V.shape[-1]), np.zeros(0)
    s = K[pos] @ q / np.sqrt(len(q))
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ V[pos], p


def evict_select(w, length, budget, sink, recent):
    """Positions of one (batch, kv head) that stay, ascending."""
    if length <= budget:
        return np.arange(length)
    keep = set(range(sink)) | set(range(length - recent, length))
    mid = [(-np.inf if np.isnan(w[p]) else w[p], p) for p in range(sink, length - recent)]
    mid.sort(key=lambda t: (-t[0], t[1]))
    keep |= {p for _, p in mid[:budget - sink - recent]}
    return np.array(sorted(keep), dtype=np.int64)


def requantise(values, fmt, block):
    """Rows [n, d] as block-scaled format values: (stored, scale per block)."""
    n = len(values)
    stored = np.empty_like(values)
    scale = np.empty(-(-n // block))
    for j in range(len(scale)):
        rows = values[j * block:(j + 1) * block]
        scale[j] = block_scale(np.abs(rows).max(), fmt)
        stored[j * block:(j + 1) * block] = round8(rows / scale[j], fmt)
    return stored, scale
