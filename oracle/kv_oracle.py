"""The paged cache and its attention in float64, from the definitions (numpy, no GPU code shared).

Cached values are decoded float64 arrays [n_pages, n_kv, page_tokens, d] (8-bit codes already times
their page's scale); a sequence is its row of the page table and its length.
"""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The 256 values of OCP E4M3: exponent bias 7, no infinities, 0x7F and 0xFF are NaN."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        out[c] = s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        if c & 0x7F == 0x7F:
            out[c] = np.nan
    return out


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Codes of x (|x| <= 448), to nearest, ties to the even code; NaN and infinities to 0x7F."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    a = np.where(fin, np.abs(x), 0.0)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    e = np.where(a >= np.exp2(e + 1), e + 1, np.where((a < np.exp2(e)) & (e > -6), e - 1, e))
    q = np.round(a / np.exp2(e - 3))  # numpy rounds ties to even; q <= 16
    code = np.where(q < 8, q, (e + 7) * 8 + (q - 8)).astype(np.int64)  # q = 16 carries into the exponent
    return np.where(fin, code + np.where(np.signbit(x), 128, 0), 0x7F).astype(np.uint8)


def least_scale(a: float) -> float:
    """The least power of two s >= 2^-118 with a <= 448 s."""
    s = 2.0 ** -118
    while a > 448 * s:
        s *= 2
    return s


def rotate(x: np.ndarray, pos: np.ndarray, inv_freq: np.ndarray, style: str) -> np.ndarray:
    """x [rows, heads, d] with row i at position pos[i]."""
    x = np.array(x, np.float64)
    for j, f in enumerate(np.asarray(inv_freq, np.float64)):
        a, b = (j, j + len(inv_freq)) if style == "halves" else (2 * j, 2 * j + 1)
        c, s = np.cos(pos * f)[:, None], np.sin(pos * f)[:, None]
        u, v = x[:, :, a].copy(), x[:, :, b].copy()
        x[:, :, a], x[:, :, b] = u * c - v * s, v * c + u * s
    return x


def append_fp8(values, scale, table, first, new):
    """Values (units of the scale) and scales of one 8-bit cache after one sequence's tokens `new`
    [n, n_kv, d] from position `first`, unrounded. `values` [n_pages, n_kv, pt, d] are codes' values."""
    pt = values.shape[2]
    values, scale = values.copy(), scale.astype(np.float64)
    n_pages = values.shape[0]
    by_page = {}
    for i in range(len(new)):
        p = first + i
        if p < 0 or p // pt >= len(table):
            continue
        page = int(table[p // pt])
        if 0 <= page < n_pages:
            by_page.setdefault(page, []).append((p % pt, i))
    for page, items in by_page.items():
        for h in range(values.shape[1]):
            x = np.stack([new[i, h] for _, i in items])
            need = least_scale(np.abs(x[np.isfinite(x)]).max(initial=0.0))
            s0 = items[0][0]
            old = scale[page, h]
            scale[page, h] = need if s0 == 0 else max(old, need)
            values[page, h, :s0] *= old / scale[page, h]
            for slot, i in items:
                values[page, h, slot] = new[i, h] / scale[page, h]
    return values, scale


def visible(p: int, n: int, window: int, sinks: int, listed=None, entry_tokens: int = 1) -> np.ndarray:
    """Which of the first n positions the query at p sees; `listed` entries for the top-k form."""
    s = np.arange(n)
    if listed is None:
        see = np.ones(n, bool) if window == 0 else (s > p - window) | (s < sinks)
    else:
        see = np.isin(s // entry_tokens, [e for e in listed if e >= 0]) | (s < sinks)
        if window > 0:
            see |= s > p - window
    return see & (s <= p)


def rows_of(cache: np.ndarray, table: np.ndarray, n: int, h: int):
    """(values [n, d], there [n]) of the first n positions; a bad page holds no tokens."""
    n_pages, _, pt, d = cache.shape
    out, there = np.zeros((n, d)), np.zeros(n, bool)
    for s in range(0, n, pt):
        if s // pt >= len(table):
            break
        page = int(table[s // pt])
        if 0 <= page < n_pages:
            m = min(pt, n - s)
            out[s:s + m], there[s:s + m] = cache[page, h, :m], True
    return out, there


def attend_row(q, K, V, see, scale):
    """One query row: (out [d], lse, sum_s P_s |V_s| [d], largest sum |q_i K_si| * scale of a seen key)."""
    d = len(q)
    if not see.any():
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    k, v = K[see], V[see]
    x = k @ q * scale
    with np.errstate(invalid="ignore"):
        m = x.max()
        p = np.exp(x - m)
        l = p.sum()
        return p @ v / l, m + np.log(l), p @ np.abs(v) / l, float((np.abs(k) @ np.abs(q)).max() * abs(scale))
