"""Accumulated key weights, the 4-bit K/V cache and eviction, as their definitions, in fp64.

Test infrastructure (see package docstring); none of this is on the pages.  Codes, scales and records
follow the format that the library's header describes; the functions here decode and encode it element by
element, with exact rational arithmetic where a rounding is decided.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .attention import _group

GROUP = 32


def visible(Sq: int, Sk: int, mask: str, n: int | None = None) -> np.ndarray:
    """Boolean ``[Sq, Sk]``: does row i see key j?  ``n``: only the first n keys are valid (the rows
    are then the last of n tokens under ``bottom_right``)."""
    i, j = np.arange(Sq)[:, None], np.arange(Sk)[None, :]
    n = Sk if n is None else n
    if mask == "top_left" and Sq > 1:
        return (j <= i) & (j < n)
    if mask == "bottom_right":
        return (j <= i + n - Sq) & (j < n)
    return np.broadcast_to(j < n, (Sq, Sk))


def key_weights(Q, K, lse, mask: str = "none", scale: float | None = None) -> np.ndarray:
    """``w[B, Hkv, Sk]``: column sums of ``exp(Q K^T scale - lse)`` over each kv head's query heads."""
    Q, K, lse = (np.asarray(a, dtype=np.float64) for a in (Q, K, lse))
    B, Hq, Sq, D = Q.shape
    Hkv, Sk = K.shape[1], K.shape[2]
    G = _group(Hq, Hkv)
    scale = D ** -0.5 if scale is None else scale
    seen = visible(Sq, Sk, mask)
    out = np.zeros((B, Hkv, Sk))
    for b in range(B):
        for h in range(Hq):
            S = (Q[b, h] @ K[b, h // G].T) * scale
            z = lse[b, h][:, None]
            with np.errstate(invalid="ignore", over="ignore"):
                P = np.where(seen & (z != -np.inf), np.exp(S - z), 0.0)
            out[b, h // G] += P.sum(0)
    return out


# ---------------------------------------------------------------------------------- 4-bit records
def _bf16(x) -> float:
    """The bfloat16 nearest to x towards zero, exactly (x a Fraction or float)."""
    f = np.float32(float(x))
    bits = int(np.array(f, np.float32).view(np.uint32)) & 0xFFFF0000
    v = float(np.array(bits, np.uint32).view(np.float32))
    if abs(Fraction(v)) > abs(Fraction(x)):   # float32 rounded away past a bfloat16
        v = float(np.array(bits - 0x10000, np.uint32).view(np.float32))
    return v


def _next(v: float, up: bool) -> float:
    """The bfloat16 above (or below) the bfloat16 v."""
    if v == 0.0:
        return float(np.array(0x00010000 if up else 0x80010000, np.uint32).view(np.float32))
    bits = int(np.array(v, np.float32).view(np.uint32))
    away = (v > 0) == up
    return float(np.array(bits + (0x10000 if away else -0x10000), np.uint32).view(np.float32))


def quantise_group(x):
    """``(codes, scale, minimum)`` of one group: exact rational arithmetic."""
    x = [Fraction(float(v)) for v in x]
    lo, hi = min(x), max(x)
    m = _bf16(lo)
    if Fraction(m) > lo:
        m = _next(m, up=False)
    rng = hi - Fraction(m)
    s = _bf16(rng / 15)
    if Fraction(s) * 15 < rng:
        s = _next(s, up=True)
    if s == 0.0:
        return [0] * len(x), 0.0, m
    # round() of a Fraction is half to even
    return [round((v - Fraction(m)) / Fraction(s)) for v in x], s, m


def records(K, V) -> np.ndarray:
    """uint8 records ``[..., 1.25 D]`` of rows ``K[..., D]``, ``V[..., D]`` (finite values)."""
    K, V = np.asarray(K, np.float64), np.asarray(V, np.float64)
    D = K.shape[-1]
    rec = np.zeros((int(np.prod(K.shape[:-1])), D + D // 4), np.uint8)
    for row, (k, v) in enumerate(zip(K.reshape(-1, D), V.reshape(-1, D))):
        for half, x in enumerate((k, v)):
            for g in range(D // GROUP):
                codes, s, m = quantise_group(x[g * GROUP:(g + 1) * GROUP])
                for c, code in enumerate(codes):
                    w = (g * GROUP + c) // 8
                    byte = half * (D // 2) + 4 * ((w % 4) * (D // GROUP) + w // 4) + (c % 8) // 2
                    rec[row, byte] |= code << (4 * (c % 2))
                pair = np.array([s, m], np.float32).view(np.uint32) >> 16
                at = D + half * (D // 8) + 4 * g
                rec[row, at:at + 4] = pair.astype(np.uint16).view(np.uint8)
    return rec.reshape(*K.shape[:-1], D + D // 4)


def record_values(rec):
    """``(K, V)`` fp64 values ``[..., D]`` that records stand for, and ``(|K|, |V|)`` bounds of the terms
    they are summed from (``|minimum| + scale * code``)."""
    rec = np.asarray(rec)
    D = rec.shape[-1] * 4 // 5
    out, mag = [], []
    c = np.arange(D)
    w = c // 8
    for half in range(2):
        byte = half * (D // 2) + 4 * ((w % 4) * (D // GROUP) + w // 4) + (c % 8) // 2
        code = ((rec[..., byte] >> (4 * (c % 2)).astype(np.uint8)) & 15).astype(np.float64)
        at = D + half * (D // 8)
        pair = np.ascontiguousarray(rec[..., at:at + D // 8]).view(np.uint16).astype(np.uint32) << np.uint32(16)
        pair = pair.view(np.float32).astype(np.float64)
        s, m = pair[..., 0::2][..., c // GROUP], pair[..., 1::2][..., c // GROUP]
        out.append(s * code + m)
        mag.append(np.abs(s * code) + np.abs(m))
    return out, mag


def attention_records(Q, rec, lens=None, mask: str = "none", scale: float | None = None):
    """Attention of ``Q[B, Hq, Sq, D]`` over ``rec[B, Hkv, S, 1.25 D]``: ``(O, lse, w, A)`` with the key
    weights ``w[B, Hkv, S]`` and ``A = sum_j P_j |V_j|``, the size of the terms O is summed from."""
    Q = np.asarray(Q, np.float64)
    B, Hq, Sq, D = Q.shape
    Hkv, S = rec.shape[1], rec.shape[2]
    G = _group(Hq, Hkv)
    scale = D ** -0.5 if scale is None else scale
    O, A = np.zeros(Q.shape), np.zeros(Q.shape)
    lse, w = np.full((B, Hq, Sq), -np.inf), np.zeros((B, Hkv, S))
    for b in range(B):
        n = S if lens is None else int(min(max(lens[b], 0), S))
        (K, V), (_, Vm) = record_values(rec[b, :, :n])
        for h in range(Hq):
            g = h // G
            s = np.where(visible(Sq, n, mask, n), (Q[b, h] @ K[g].T) * scale, -np.inf)
            for i in range(Sq):
                if n == 0 or np.all(s[i] == -np.inf):
                    continue
                m = s[i].max()
                e = np.exp(s[i] - m)
                p = e / e.sum()
                lse[b, h, i] = m + np.log(e.sum())
                live = p > 0
                O[b, h, i] = p[live] @ V[g][live]
                A[b, h, i] = p[live] @ Vm[g][live]
                w[b, g, :n] += p
    return O, lse, w, A


def evict(weights, n: int, budget: int, sinks: int, recent: int) -> np.ndarray:
    """Positions kept of one row of n valid keys, ascending."""
    if n <= budget:
        return np.arange(n)
    lo, hi = sinks, n - recent
    mid = sorted(range(lo, hi), key=lambda j: (-(float("-inf") if np.isnan(weights[j]) else float(weights[j])), j))
    nan_last = [j for j in mid if not np.isnan(weights[j])] + [j for j in mid if np.isnan(weights[j])]
    kept = nan_last[:budget - sinks - recent]
    return np.array(sorted(list(range(sinks)) + kept + list(range(hi, n))), dtype=np.int64)
