"""Attention under a sliding window with sinks and its gradients, written out as their definition, in fp64.

Test infrastructure (see package docstring).  The pages' attention ([Q3] "自注意力原理", "GQA") with another mask: the Sq
rows are the last of Sk tokens, row ``i`` stands at position ``p = i + Sk - Sq`` and sees key ``j`` where ``j <= p`` and
(``p - j < window`` or ``j < sinks``).
"""
from __future__ import annotations

import numpy as np

from .attention import _group


def window_mask(Sq: int, Sk: int, window: int, sinks: int):
    """``[Sq, Sk]`` truth values: whether a row sees a key (``window`` 0: no window)."""
    p, j = np.arange(Sq)[:, None] + Sk - Sq, np.arange(Sk)[None, :]
    return (j <= p) & (((p - j < window) | (j < sinks)) if window else True)


def attention_window(Q, K, V, window: int, sinks: int = 0, scale: float | None = None, dO=None):
    """``(O, lse, size)`` and, with ``dO``, ``(dQ, dK, dV)`` and their rounding errors' sizes too, of ``[B, H, S, D]``
    arrays.  ``size`` is ``sum_j P_ij |V_j|``, what rounding errors of P and of sums are relative to.  The sizes of the
    gradients' errors are a triple of pairs ``(near, far)``: ``near`` what one rounding of P, dS = P (dP - D) and of O
    (in D = dO . O) is relative to, ``far`` what errors of the sums dP and D are relative to."""
    Q, K, V = (np.asarray(a, dtype=np.float64) for a in (Q, K, V))
    B, Hq, Sq, D = Q.shape
    Hkv, Sk = K.shape[1], K.shape[2]
    G = _group(Hq, Hkv)
    scale = D ** -0.5 if scale is None else scale
    see = window_mask(Sq, Sk, window, sinks)
    O, size, lse = np.zeros_like(Q), np.zeros_like(Q), np.full((B, Hq, Sq), -np.inf)
    grads = tuple(np.zeros_like(a) for a in (Q, K, V))
    sizes = tuple((np.zeros_like(a), np.zeros_like(a)) for a in (Q, K, V))
    for b in range(B):
        for h in range(Hq):
            k, v = K[b, h // G], V[b, h // G]
            S = np.where(see, Q[b, h] @ k.T * scale, -np.inf)
            m = S.max(1, initial=-np.inf, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            E = np.exp(S - m)
            L = E.sum(1, keepdims=True)
            with np.errstate(divide="ignore", invalid="ignore"):
                P = np.where(L > 0, E / L, 0.0)
                lse[b, h] = np.where(L > 0, m + np.log(L), -np.inf)[:, 0]
            O[b, h], size[b, h] = P @ v, P @ np.abs(v)
            if dO is not None:
                g = np.asarray(dO[b, h], dtype=np.float64)
                dP = g @ v.T
                dS = P * (dP - (dP * P).sum(1, keepdims=True)) * scale
                grads[0][b, h] = dS @ k
                grads[1][b, h // G] += dS.T @ Q[b, h]
                grads[2][b, h // G] += P.T @ g
                of_d = P * np.abs(g * O[b, h]).sum(1, keepdims=True) * scale
                near, far = of_d + np.abs(dS), of_d + P * (np.abs(g) @ np.abs(v).T) * scale
                for i, e in enumerate((near, far)):
                    sizes[0][i][b, h] = e @ np.abs(k)
                    sizes[1][i][b, h // G] += e.T @ np.abs(Q[b, h])
                    sizes[2][i][b, h // G] += P.T @ np.abs(g)
    return (O, lse, size) if dO is None else (O, lse, size, *grads, sizes)
