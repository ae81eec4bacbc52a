"""Attention over 4-bit records whose V scales and values lie far apart, against the fp64 oracle.

Tolerances, with u = 2^-24 (float32) and h = 2^-8 (bfloat16), the half steps relative to a value; A of a channel is
sum p (|minimum| + scale * code):
  score         a sum of D products in float32, each operand exact: |ds| <= 2 (D + 8) u scale sum |q| |k|; the
                factor 2 allows the tensor core to truncate
  p             relative error e = ds + 4 u (|score| + 12) + 2^-21: the score's rounding, the exponent's, 2^x
  sum           n terms in float32, 2 n u (again with truncation)
  O             A (2 e + 2 (n + 8) u) + u |O|: p and the denominator, float32 products; a bfloat16 result + h |O|
  bfloat16 queries with D 64 or 128: p * scale in 11 bits, + 2^-11 A; and, where every scale of a tile is at least
                2^-6 of the largest met, in float16 whose least step is 2^-38 of that one's next power of two 2^e: at
                most 15 codes times 2^(e - 39) of a key, where the row's largest p is at least 2^-5 (references are
                whole numbers, 4 above): n 15 2^-34 2^e / sum exp(s - max s), and 2^e <= 2^7 of the smallest scale
  lse           ds + 4 u (|score| + |lse| + 12) + 2^-21 + n u: the denominator, its logarithm and their sum
"""
import numpy as np
import pytest

import oracle
from test_gpu_kv4 import H, U, check_attention, ints, random_cache, rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def pairs(rec, D, half):
    """The (scale, minimum) pairs of one half (0: K, 1: V) of numpy records, float32 [..., D / 32, 2]."""
    at = D + half * (D // 8)
    bits = np.ascontiguousarray(rec[..., at:at + D // 8]).view(np.uint16).astype(np.uint32) << np.uint32(16)
    return bits.view(np.float32).reshape(*rec.shape[:-1], D // 32, 2).copy()


def set_pairs(rec, D, half, p):
    at = D + half * (D // 8)
    bits = np.ascontiguousarray(p.astype(np.float32)).view(np.uint32) >> np.uint32(16)
    rec[..., at:at + D // 8] = bits.astype(np.uint16).reshape(*rec.shape[:-1], -1).view(np.uint8)


def set_codes(rec, D, half, group, code, where):
    """Codes of the V or K channels of a group, of the records `where` selects."""
    for t in range(4):
        byte = half * (D // 2) + 4 * (t * (D // 32) + group)
        rec[(*where, slice(byte, byte + 4))] = code * 17


def weight_sum(q, rec, lens, mask, scale):
    """sum exp(s - max s) of every row, at least 1."""
    B, Hq, Sq, _ = q.shape
    Hkv, S = rec.shape[1], rec.shape[2]
    (K, _), _ = oracle.record_values(rec)
    out = np.ones((B, Hq, Sq))
    for b in range(B):
        n = S if lens is None else lens[b]
        for h in range(Hq):
            s = np.where(oracle.kv_cache.visible(Sq, n, mask, n), (q[b, h] @ K[b, h * Hkv // Hq, :n].T) * scale, -np.inf)
            out[b, h] = np.maximum(np.exp(s - np.maximum(s.max(-1, keepdims=True, initial=-np.inf), -1e300)).sum(-1), 1)
    return out


def check(osf, q, rec, lens=None, mask="none", scale=None, what=""):
    qv = q.double().cpu().numpy()
    B, Hq, Sq, D = qv.shape
    Hkv, S = rec.shape[1], rec.shape[2]
    G = Hq // Hkv
    lse = torch.empty(B, Hq, Sq, device="cuda")
    out = osf.osf_attn_kv4(q, torch.from_numpy(rec).cuda(), lens=None if lens is None else ints(lens), mask=mask, scale=scale, lse=lse)
    O, L, _, A = oracle.attention_records(qv, rec, lens, mask, scale)
    sc = D ** -0.5 if scale is None else scale
    _, (Km, _) = oracle.record_values(rec)
    top = max((np.abs(qv[b, h]) @ Km[b, h // G].T).max() for b in range(B) for h in range(Hq)) * sc
    ds = 2 * (D + 8) * U * top
    e = ds + 4 * U * (top + 12) + 2.0 ** -21
    tol = A * (2 * e + 2 * (S + 8) * U) + U * np.abs(O)
    if q.dtype == torch.bfloat16:
        tol = tol + H * np.abs(O)
    if q.dtype == torch.bfloat16 and D in (64, 128):
        sv = pairs(rec, D, 1)[..., 0]
        least = sv[sv > 0].min() if np.any(sv > 0) else 0.0
        tol = tol + 2.0 ** -11 * A + S * 15 * 2.0 ** -27 * least / weight_sum(qv, rec, lens, mask, sc)[..., None]
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(np.isfinite(got)), what
    excess = (np.abs(got - O) - tol) / np.maximum(A, 1e-300)
    assert np.max(excess) <= 0, f"{what}: O off by {np.max(excess):.3e} of its terms past the tolerance"
    seen = np.isfinite(L)
    assert np.array_equal(np.isneginf(gl), ~seen)
    lt = ds + 4 * U * (top + np.abs(L[seen]) + 12) + 2.0 ** -21 + S * U
    worst = np.max(np.abs(gl[seen] - L[seen]) - lt)
    assert worst <= 0, f"{what}: lse off by {worst:.3e} past its tolerance"


KINDS = [("bf16", 64), ("bf16", 128), ("bf16", 96), ("f32", 128)]


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("ratio", [10, 16, 24, 28, 32, 40, 60])
def test_groups_whose_scales_differ(osf, dtype, D, ratio):
    """The second group's values are 2^ratio below the first's."""
    for n, sharp, lens in ((64, 0.0, None), (64, 6.0, None), (4400, 0.0, None), (4400, 6.0, [4400, 77])):
        B = 1 if lens is None else 2
        _, rec = random_cache(B, 2, n, D, ratio + n)
        for zero in (False, True):   # with the minima that quantised values have, and without
            p = pairs(rec, D, 1)
            p[..., 1, :] *= 2.0 ** -ratio
            if zero:
                p[..., 1] = 0
            r = rec.copy()
            set_pairs(r, D, 1, p)
            q, _ = rows((B, 4, 1, D), n, dtype)
            check(osf, q * sharp, r, lens=lens, what=f"n={n} sharp={sharp} zero={zero}")


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("ratio", [10, 16, 24, 28, 32, 40, 60])
def test_a_key_whose_scale_is_far_above_the_others(osf, dtype, D, ratio):
    """One record's V scales are 2^ratio above the others': with a weight like theirs, where its codes are zero; with a
    weight that vanishes; and hidden by the mask from most rows."""
    q, _ = rows((1, 4, 4, D), ratio, dtype)
    for n in (70, 3000):
        _, rec = random_cache(1, 2, n, D, ratio + n)
        p = pairs(rec, D, 1)
        p[..., 1] = 0
        at = n // 2
        p[:, :, at, :, 0] *= 2.0 ** ratio
        set_pairs(rec, D, 1, p)
        for g in range(D // 32):
            set_codes(rec, D, 1, g, 0, (slice(None), slice(None), at))
        check(osf, q * 0, rec, what=f"codes of zero, n={n}")
        check(osf, q * 0.25, rec, what=f"codes of zero, n={n}, uneven weights")
        for g in range(D // 32):
            set_codes(rec, D, 1, g, 9, (slice(None), slice(None), at))
        pk = pairs(rec, D, 0)
        pk[:, :, at, :, 0] = 0
        pk[:, :, at, :, 1] = -30.0   # queries of ones: a score of -30 sqrt(D)
        low = rec.copy()
        set_pairs(low, D, 0, pk)
        check(osf, torch.ones_like(q) * 0.125, low, what=f"low score, n={n}")
        late = np.roll(rec, n - 1 - at, axis=2)   # the last key: only the last row sees it
        check(osf, q * 0.25, late, mask="bottom_right", what=f"hidden, n={n}")


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("exponent", [-100, -70, 0, 70, 100])
def test_scores_do_not_depend_on_the_values(osf, dtype, D, exponent):
    """lse and O with V constant in every group (scale 0) and with V scales of 2^exponent, few keys and many; keys 2^-18
    below the largest still count."""
    for n in (1, 3, 15, 100):
        _, rec = random_cache(1, 2, n, D, n)
        q, _ = rows((1, 4, 4, D), n, dtype)
        for const in (True, False):
            p = pairs(rec, D, 1)
            p[..., 0] = 0 if const else p[..., 0] * 2.0 ** exponent
            p[..., 1] *= 2.0 ** exponent
            r = rec.copy()
            set_pairs(r, D, 1, p)
            check(osf, q * 2.0 ** -6, r, what=f"n={n} const={const}")
    n = 4000
    _, rec = random_cache(1, 1, n, D, 5)
    pk, pv = pairs(rec, D, 0), pairs(rec, D, 1)
    pk[..., 0] = 0
    pk[..., 1] = -1
    pk[:, :, 700, :, 1] = 0.5
    pv[..., :] *= 2.0 ** exponent
    set_pairs(rec, D, 0, pk)
    set_pairs(rec, D, 1, pv)
    # scores 0.5 and -1 times scale * D: 18 ln 2 apart
    check(osf, torch.ones(1, 2, 1, D, device="cuda", dtype=torch.bfloat16 if dtype == "bf16" else torch.float32), rec,
          scale=float(np.float32(12 * np.log(2) / D)), what="one key above the others")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(1, 1, 1), (4, 1, 1), (6, 2, 3), (16, 1, 1), (8, 2, 5)])
@pytest.mark.parametrize("S", [1, 17, 100, 1000, 5000])
def test_ordinary_records_keep_eleven_bits(osf, D, Hq, Hkv, Sq, S):
    _, rec = random_cache(2, Hkv, S, D, S + Hq)
    q, _ = rows((2, Hq, Sq, D), S, "bf16")
    check(osf, q, rec, lens=[S, S // 2], mask="bottom_right")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(16, 1, 1), (8, 2, 4), (24, 1, 1), (4, 1, 5)])
@pytest.mark.parametrize("S", [50, 4600])
def test_scales_far_apart_with_many_rows_and_weights(osf, D, Hq, Hkv, Sq, S):
    """Groups 2^20 and keys 2^12 apart under 16 and more rows, with the records' weights, a mask and ragged lengths."""
    _, rec = random_cache(3, Hkv, S, D, S + Hq)
    p = pairs(rec, D, 1)
    p[..., 1, :] *= 2.0 ** -20
    p[:, :, ::7] *= 2.0 ** 12
    set_pairs(rec, D, 1, p)
    q, _ = rows((3, Hq, Sq, D), S, "bf16")
    lens = [S, S // 2, 3]
    check(osf, q, rec, lens=lens, mask="bottom_right")
    check_attention(osf, 3, Hq, Hkv, Sq, S, D, "bf16", lens=lens, mask="bottom_right", q=q, cache=torch.from_numpy(rec).cuda())
