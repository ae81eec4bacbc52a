"""The paged 8-bit K/V cache, written out as its definition (test infrastructure, see package docstring; no page has a
cache).  Pages ``[n_pages, 2, Hkv, P, D]`` of e4m3 codes, scales ``[n_pages, 2, Hkv]`` powers of two, tables ``[B, per]``.
"""
from __future__ import annotations

import numpy as np

MIN_EXP = -110


def e4m3_values():
    """float64 value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = np.nan if c & 127 == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        out[c] = -v if c & 128 else v
    return out


def e4m3_codes(x):
    """Codes of float64 values, |x| <= 448, to the nearest, ties to the even code; not finite: 0x7f."""
    x = np.asarray(x, np.float64)
    pos = e4m3_values()[:127]
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    down, up = a - pos[lo], pos[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isfinite(x), code | np.where(np.signbit(x), 128, 0), 127).astype(np.uint8)


def scale_exponent(amax: float) -> int:
    """The least e >= MIN_EXP with amax <= 448 * 2^e."""
    e = MIN_EXP
    while amax > np.ldexp(448.0, e):
        e += 1
    return e


def rotate(x, pos, cos, sin, interleaved: bool):
    """Rows ``[..., n, D]`` at positions ``pos [n]``, rotated and rounded once to float32; ``cos`` None: as they are."""
    x = np.array(x, np.float64)
    if cos is None:
        return x.astype(np.float32)
    R = 2 * cos.shape[1]
    i = np.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    c, s = cos[pos].astype(np.float64), sin[pos].astype(np.float64)
    out = x.copy()
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    with np.errstate(over="ignore"):
        return out.astype(np.float32)


def kv8_append(k, v, pages, scales, table, lens=None, counts=None, cos=None, sin=None, interleaved=False):
    """Store rows ``[B, Hkv, n, D]`` behind ``lens`` tokens, in place."""
    B, Hkv, n, _ = k.shape
    P, per = pages.shape[3], table.shape[1]
    value = e4m3_values()
    for b in range(B):
        at = 0 if lens is None else int(lens[b])
        m = n if counts is None else min(int(counts[b]), n)
        m = min(m, per * P - at) if at >= 0 else 0
        for page_no in range(at // P if m > 0 else 0, -(-(at + m) // P) if m > 0 else 0):
            page = table[b, page_no]
            if not 0 <= page < len(pages):
                continue
            t0, t1 = max(at, page_no * P), min(at + m, (page_no + 1) * P)
            pos = np.minimum(np.arange(t0, t1), (1 << 60) if cos is None else len(cos) - 1)
            for half, rows in ((0, rotate(k[b, :, t0 - at:t1 - at], pos, cos, sin, interleaved)),
                               (1, v[b, :, t0 - at:t1 - at].astype(np.float32))):
                for h in range(Hkv):
                    x = rows[h].astype(np.float64)
                    e = scale_exponent(np.abs(x[np.isfinite(x)]).max(initial=0.0))
                    old = t0 - page_no * P
                    if old:
                        was = int(np.frexp(scales[page, half, h])[1]) - 1
                        if e > was:
                            there = value[pages[page, half, h, :old]] * 2.0 ** (was - e)
                            pages[page, half, h, :old] = e4m3_codes(there)
                        e = max(e, was)
                    pages[page, half, h, old:t1 - page_no * P] = e4m3_codes(np.ldexp(x, -e))
                    scales[page, half, h] = np.ldexp(1.0, e)


def kv8_values(pages, scales, table, n):
    """float64 K, V ``[Hkv, n, D]`` of the first n tokens of one sequence (``table [per]``); 0 where there is no page."""
    P = pages.shape[3]
    value = e4m3_values()
    out = np.zeros((2, pages.shape[2], n, pages.shape[4]))
    for t in range(0, n, P):
        page = table[t // P]
        if 0 <= page < len(pages):
            cnt = min(P, n - t)
            out[:, :, t:t + cnt] = value[pages[page, :, :, :cnt]] * scales[page].astype(np.float64)[..., None, None]
    return out[0], out[1]
