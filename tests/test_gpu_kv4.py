"""The 4-bit K/V cache on the GPU: stored records byte for byte, values read back, and attention over
records against the fp64 oracle.

Tolerances, with u = 2^-24 (float32) and h = 2^-8 (bfloat16), the half steps relative to a value:
  read back     one rounding of the exact value to float32, one more to bfloat16
  score         a sum of D products in float32, each operand exact: |ds| <= 2 (D + 8) u scale sum |q| |k|, |k| taken as
                |minimum| + scale * code; the factor 2 allows the tensor core to truncate
  weight p      relative error e = ds + (|lse| + 8) 4 u + 4 (2^-22), from the exponent and the 2^x approximation
  O, float32    sum p |v| (2 e + (n + D) u);  bfloat16: + h for P, + h for V, + h |O| for the result
  lse           max ds + 16 u (|lse| + 1) + 2^-21
  weights       relative e + (rows + 64) u
"""
import numpy as np
import pytest

import oracle
import seeded_inputs as si
from conftest import bf16_tensor, f32_tensor

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U, H = 2.0 ** -24, 2.0 ** -8


def rows(shape, seed, dtype):
    """(GPU tensor, fp64 values) of normal rows with an offset and a width per channel."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape) * rng.uniform(0.5, 1.5, shape[-1]) + rng.standard_normal(shape[-1]) * 0.5
    if dtype == "bf16":
        bits = si.f32_to_bf16_bits(x.astype(np.float32))
        return bf16_tensor(bits), si.bf16_bits_to_f32(bits).astype(np.float64)
    x = x.astype(np.float32)
    return f32_tensor(x), x.astype(np.float64)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def random_cache(B, Hkv, S, D, seed):
    """A cache of records with random codes and plausible scales and minima (the oracle's exact
    quantiser is too slow for long caches)."""
    rng = np.random.default_rng(seed)
    rec = rng.integers(0, 256, (B, Hkv, S, D + D // 4), dtype=np.uint8)
    pairs = np.empty((B, Hkv, S, 2 * (D // 32), 2), np.float32)
    pairs[..., 0] = rng.uniform(0.05, 0.4, pairs.shape[:-1])
    pairs[..., 1] = -7.5 * pairs[..., 0] + 0.3 * rng.standard_normal(pairs.shape[:-1])
    rec[..., D:] = (pairs.view(np.uint32) >> 16).astype(np.uint16).reshape(B, Hkv, S, -1).view(np.uint8)
    return torch.from_numpy(rec).cuda(), rec


# ------------------------------------------------------------------------------------------ store, read
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 256])
def test_append_writes_the_oracle_records(osf, dtype, D):
    B, Hkv, n, S = 2, 3, 5, 11
    k, kv = rows((B, Hkv, n, D), D, dtype)
    v, vv = rows((B, Hkv, n, D), D + 1, dtype)
    cache = torch.full((B, Hkv, S, osf.osf_kv4_record_bytes(D)), 0xA5, dtype=torch.uint8, device="cuda")
    lens = [6, 1]
    osf.osf_kv4_append(k, v, cache, lens=ints(lens))
    got, want = cache.cpu().numpy(), oracle.records(kv, vv)
    for b in range(B):
        assert np.array_equal(got[b, :, lens[b]:lens[b] + n], want[b])
        rest = np.delete(got[b], np.s_[lens[b]:lens[b] + n], axis=1)
        assert np.all(rest == 0xA5)   # no other record is touched
    # read back: one rounding of the exact values
    (K, V), _ = oracle.record_values(want)
    for dt, tol in ((torch.float32, U), (torch.bfloat16, H)):
        ko, vo = osf.osf_kv4_read(cache, D, n, starts=ints(lens), dtype=dt)
        for g, w in ((ko, K), (vo, V)):
            err = np.abs(g.double().cpu().numpy() - w)
            assert np.all(err <= tol * (1 + 2 * U) * np.abs(w) + U * np.abs(w))
    assert osf.osf_device_status() == osf.OSF_OK


def test_append_of_values_next_to_ties(osf):
    """Groups whose values sit on, just above and just below the ties of a code, wide ranges, constants,
    subnormals and both zeros: every code is the exact one."""
    rng = np.random.default_rng(3)
    g = []
    for s, m in ((1.0, 0.0), (0.0078125, -3.0), (2.0 ** -120, 2.0 ** -118), (3.0 * 2.0 ** -131, 0.0), (2.0 ** 100, -2.0 ** 103),
                 (1.015625, 1000.0)):
        ties = m + s * (np.arange(15) + 0.5)
        x = np.concatenate([[m, m + 15 * s], ties, np.nextafter(ties.astype(np.float32), np.float32(np.inf))[:15]])
        g += [x[:32], np.concatenate([[m, m + 15 * s], np.nextafter(ties.astype(np.float32), np.float32(-np.inf)), ties])[:32]]
    g += [np.full(32, 0.1), np.zeros(32), np.concatenate([np.full(16, -0.0), np.zeros(16)]), np.full(32, 1e-45),
          np.concatenate([[1e30, -1e-30], rng.standard_normal(30)]), np.concatenate([[2.5e38, 1.0], np.full(30, 1e38)])]
    x = np.array(g, np.float64).astype(np.float32)
    x = np.concatenate([x, np.zeros((-len(x) % 4, 32), np.float32)]).reshape(1, 1, -1, 128)
    n = x.shape[2]
    cache = torch.zeros(1, 1, n, osf.osf_kv4_record_bytes(128), dtype=torch.uint8, device="cuda")
    osf.osf_kv4_append(f32_tensor(x), f32_tensor(x[:, :, ::-1]), cache)
    diff = np.argwhere(cache.cpu().numpy() != oracle.records(x, x[:, :, ::-1]))
    assert len(diff) == 0, diff[:20].tolist()


def test_append_of_bfloat16_values_of_all_magnitudes(osf):
    """Magnitudes spread over 2^-30 .. 2^4, tiny minima under coarse values, offsets far from zero: the codes
    of bfloat16 groups are the exact ones too."""
    rng = np.random.default_rng(4)
    n = 48
    x = rng.standard_normal((1, 1, n, 128)) * 2.0 ** rng.uniform(-30, 4, (1, 1, n, 128))
    x[0, 0, :12] = np.abs(np.round(rng.standard_normal((12, 128)) * 8) / 8) + 0.125      # coarse, with exact ties
    x[0, 0, :6, ::32] = 2.0 ** rng.uniform(-30, -12, (6, 4))                               # under a tiny minimum
    x[0, 0, 6:12, 1::32] = 2.0 ** rng.uniform(-30, -12, (6, 4)) * rng.choice([-1, 1], (6, 4))
    x[0, 0, 12:20] = 300 + np.round(rng.standard_normal((8, 128)) * 8)
    x[0, 0, 20:24, :64] = 0
    bits = si.f32_to_bf16_bits(x.astype(np.float32))
    xv = si.bf16_bits_to_f32(bits)
    cache = torch.zeros(1, 1, n, 160, dtype=torch.uint8, device="cuda")
    osf.osf_kv4_append(bf16_tensor(bits), bf16_tensor(bits[:, :, ::-1].copy()), cache)
    diff = np.argwhere(cache.cpu().numpy() != oracle.records(xv, xv[:, :, ::-1]))
    assert len(diff) == 0, diff[:20].tolist()


def test_append_counts_strides_and_bounds(osf):
    B, Hkv, n, D, S = 4, 2, 6, 64, 16
    # [B, n, H, D] projections seen as [B, H, n, D], padded rows poisoned
    k, _ = rows((B, n, Hkv, D), 5, "bf16")
    v, _ = rows((B, n, Hkv, D), 6, "bf16")
    counts, lens = [6, 0, 2, 5], [0, 3, 15, 8]
    for b, c in enumerate(counts):
        k[b, c:] = float("nan")
        v[b, c:] = float("nan")
    kt, vt = k.transpose(1, 2), v.transpose(1, 2)
    cache = torch.zeros(B, Hkv, S, 80, dtype=torch.uint8, device="cuda")
    osf.osf_kv4_append(kt, vt, cache, lens=ints(lens), counts=ints(counts))
    assert osf.osf_device_status() == osf.OSF_ERR_INVALID   # sequence 2: one of its two tokens does not fit
    assert osf.osf_device_status() == osf.OSF_OK
    got = cache.cpu().numpy()
    want = np.zeros_like(got)
    for b in range(B):
        c = min(counts[b], S - lens[b])
        if c:
            want[b, :, lens[b]:lens[b] + c] = oracle.records(kt[b, :, :c].float().cpu().numpy(), vt[b, :, :c].float().cpu().numpy())
    assert np.array_equal(got, want)
    before = cache.clone()
    for bad_lens, bad_counts in (([-1] * 4, None), ([0] * 4, [-2] * 4), ([17] * 4, [1] * 4)):
        osf.osf_kv4_append(kt, vt, cache, lens=ints(bad_lens), counts=None if bad_counts is None else ints(bad_counts))
        assert osf.osf_device_status() == osf.OSF_ERR_INVALID
        assert torch.equal(cache, before)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_group_with_a_non_finite_value_reads_nan(osf, bad):
    k, _ = rows((1, 1, 2, 64), 7, "f32")
    v = k.clone()
    k[0, 0, 0, 40] = bad
    cache = torch.zeros(1, 1, 2, 80, dtype=torch.uint8, device="cuda")
    osf.osf_kv4_append(k, v, cache)
    ko, vo = osf.osf_kv4_read(cache, 64, 2, dtype=torch.float32)
    nan = torch.isnan(ko)
    assert bool(nan[0, 0, 0, 32:].all()) and int(nan.sum()) == 32 and not bool(torch.isnan(vo).any())


def test_read_positions_behind_the_length_are_zero(osf):
    cache, rec = random_cache(2, 1, 9, 64, 8)
    k, v = osf.osf_kv4_read(cache, 64, 12, starts=ints([-2, 4]), lens=ints([9, 6]), dtype=torch.float32)
    (K, V), _ = oracle.record_values(rec)
    for got, ref in ((k, K), (v, V)):
        got = got.cpu().numpy()
        assert np.all(got[0, :, :2] == 0) and np.all(got[0, :, 11:] == 0) and np.all(got[1, :, 2:] == 0)
        assert np.allclose(got[0, :, 2:11], ref[0], rtol=2 * U, atol=0) and np.allclose(got[1, :, :2], ref[1, :, 4:6], rtol=2 * U, atol=0)
    assert osf.osf_device_status() == osf.OSF_OK


# ------------------------------------------------------------------------------------------ attention
def check_attention(osf, B, Hq, Hkv, Sq, S, D, dtype, lens=None, mask="none", seed=0, q=None, weights=True, cache=None, scale=None):
    if cache is None:
        cache, rec = random_cache(B, Hkv, S, D, seed)
    else:
        rec = cache.cpu().numpy()
    if q is None:
        q, qv = rows((B, Hq, Sq, D), seed + 1, dtype)
    else:
        qv = q.double().cpu().numpy()
    lse = torch.full((B, Hq, Sq), float("nan"), device="cuda")
    w = torch.full((B, Hkv, S), float("nan"), device="cuda") if weights else None
    lt = None if lens is None else ints(lens)
    out = osf.osf_attn_kv4(q, cache, lens=lt, mask=mask, lse=lse, weights=w, scale=scale)
    O, L, W, A = oracle.attention_records(qv, rec, lens, mask, scale)
    sc = D ** -0.5 if scale is None else scale
    _, (Km, _) = oracle.record_values(rec)
    G = Hq // Hkv
    # the largest possible error of a score of each kv head
    ds = 2 * (D + 8) * U * sc * np.array([[max((np.abs(qv[b, h]) @ Km[b, h // G].T).max() if S else 0.0 for h in range(g * G, g * G + G))
                                          for g in range(Hkv)] for b in range(B)])
    finite = np.isfinite(L)
    big = np.abs(L[finite]).max() if finite.any() else 0.0
    e = ds.max() + (big + 8) * 4 * U + 2.0 ** -20
    n = S
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    tol = A * (2 * e + (n + D) * U) + U * np.abs(O)
    if dtype == "bf16":
        tol = tol + 2 * H * A + H * np.abs(O)
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - O) - tol) if got.size else 0
    assert worst <= 0, f"O off by {worst:.3e} past its tolerance"
    assert np.array_equal(np.isneginf(gl), ~finite)
    assert np.all(got[~finite] == 0)
    assert np.all(np.abs(gl[finite] - L[finite]) <= ds.max() + 16 * U * (np.abs(L[finite]) + 1) + 2.0 ** -20)
    if weights:
        gw = w.double().cpu().numpy()
        assert np.all(np.abs(gw - W) <= W * (e + (G * Sq + 64) * U) + 1e-30)
        # adding to what is there
        base = torch.rand(B, Hkv, S, device="cuda")
        acc = base.clone()
        osf.osf_attn_kv4(q, cache, lens=lt, mask=mask, weights=acc, accumulate=True, scale=scale)
        assert np.all(np.abs(acc.double().cpu().numpy() - base.double().cpu().numpy() - W) <= W * (e + (G * Sq + 64) * U) + 4 * U * (1 + W))
        if lens is not None:
            for b, n_ in enumerate(lens):
                assert torch.equal(acc[b, :, max(n_, 0):], base[b, :, max(n_, 0):])
    assert osf.osf_device_status() == osf.OSF_OK
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("S", [1, 15, 16, 17, 33, 300])
def test_attention_lengths_and_head_dims(osf, dtype, D, S):
    check_attention(osf, 1, 4, 2, 1, S, D, dtype, seed=S + D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(1, 1, 1), (3, 3, 1), (8, 1, 1), (5, 1, 1), (4, 2, 4), (12, 4, 3), (16, 1, 1), (8, 2, 5), (9, 1, 2),
                                       (32, 2, 1), (4, 1, 11)])
def test_attention_row_counts(osf, D, Hq, Hkv, Sq):
    check_attention(osf, 2, Hq, Hkv, Sq, 203, D, "bf16", lens=[203, 87], mask="bottom_right", seed=Hq * 10 + Sq)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 64), ("bf16", 96)])
def test_attention_ragged_lengths(osf, dtype, D):
    lens = [0, 1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 1000, 1024]
    check_attention(osf, len(lens), 4, 2, 3, 1024, D, dtype, lens=lens, mask="bottom_right", seed=D)
    check_attention(osf, len(lens), 2, 2, 1, 1024, D, dtype, lens=lens, seed=D + 1)
    check_attention(osf, len(lens), 2, 1, 2, 1024, D, dtype, lens=lens, seed=D + 2)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_long_cache(osf, D):
    check_attention(osf, 1, 2, 1, 1, 40000, D, "bf16", seed=D)
    check_attention(osf, 2, 4, 1, 4, 20011, D, "bf16", lens=[20011, 7], mask="bottom_right", seed=D + 1)


def test_attention_records_behind_the_length_do_not_matter(osf):
    """Records behind a length hold NaN and infinite scales: they meet no output."""
    for D in (64, 128, 96):
        S, lens = 100, [37, 100, 0]
        cache, _ = random_cache(3, 2, S, D, D)
        clean = cache.clone()
        for b, n in enumerate(lens):
            cache[b, :, n:, D:] = 0xFF
            clean[b, :, n:] = 0
        q, _ = rows((3, 4, 2, D), 1, "bf16")
        w = [torch.zeros(3, 2, S, device="cuda") for _ in range(2)]
        a = osf.osf_attn_kv4(q, cache, lens=ints(lens), mask="bottom_right", weights=w[0])
        b = osf.osf_attn_kv4(q, clean, lens=ints(lens), mask="bottom_right", weights=w[1])
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b) and torch.equal(w[0], w[1])


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_attention_nan_records_that_the_mask_hides(osf, dtype, D):
    """A NaN record is met by the rows that see it, and by no other row of the call."""
    S, Sq = 700, 4
    q, _ = rows((1, 4, Sq, D), 51, dtype)
    clean, _ = random_cache(1, 2, S, D, 52)
    want = osf.osf_attn_kv4(q, clean, mask="bottom_right")
    for part in (slice(D, D + D // 8), slice(D + D // 8, D + D // 4), slice(D, None)):   # pairs of K, of V, of both
        bad = clean.clone()
        bad[0, :, S - 2, part] = 0xFF        # seen by rows 2 and 3
        got = osf.osf_attn_kv4(q, bad, mask="bottom_right")
        assert torch.equal(got[:, :, :2], want[:, :, :2])
        assert bool(torch.isnan(got[:, :, 2:]).all())
    bad = clean.clone()
    bad[0, :, S - 2, D + D // 8:D + D // 8 + 4] = 0xFF   # the first group of V alone
    got = osf.osf_attn_kv4(q, bad, mask="bottom_right")
    assert torch.equal(got[:, :, :2], want[:, :, :2]) and torch.equal(got[..., 32:], want[..., 32:])
    assert bool(torch.isnan(got[:, :, 2:, :32]).all())


@pytest.mark.parametrize("D,tile", [(64, 64), (128, 32)])
@pytest.mark.parametrize("B,Hkv", [(1, 2), (10, 8)])
@pytest.mark.parametrize("tiles", [48, 49, 64, 65])
def test_attention_around_the_cut_of_the_work(osf, D, tile, B, Hkv, tiles):
    """Lengths at which items begin to be shared among CTAs, whole batches and ragged ones."""
    S = tiles * tile
    lens = [max(S - 7 * b * tile, 0) for b in range(B)]   # 48 tiles less 7 * 9 would be a negative length, which is recorded
    check_attention(osf, B, 2 * Hkv, Hkv, 1, S, D, "bf16", lens=lens, seed=tiles, weights=B == 1)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_large_ragged_batch(osf, D):
    lens = [int(x) for x in np.random.default_rng(D).integers(0, 1501, 75)]
    lens[:40] = [0] * 40
    check_attention(osf, 75, 2, 1, 1, 1500, D, "bf16", lens=lens, seed=53)
    check_attention(osf, 75, 4, 2, 2, 1500, D, "bf16", lens=lens[::-1], mask="bottom_right", seed=54, weights=False)


def test_attention_strided_queries_and_outputs(osf):
    B, Hq, Hkv, Sq, S, D = 2, 4, 2, 3, 90, 128
    cache, _ = random_cache(B, Hkv, S, D, 11)
    x, _ = rows((B, Sq, Hq, D + 8), 12, "bf16")
    q = x[..., :D].transpose(1, 2)
    out = torch.full((B, Sq, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    osf.osf_attn_kv4(q, cache, out=out.transpose(1, 2), mask="bottom_right")
    want = osf.osf_attn_kv4(q.contiguous(), cache, mask="bottom_right")
    assert torch.equal(out.transpose(1, 2), want)
    # a broadcast query, and one that starts at an odd element
    one = q[:1].expand(B, -1, -1, -1)
    assert torch.equal(osf.osf_attn_kv4(one, cache), osf.osf_attn_kv4(one.contiguous(), cache))
    odd = x[..., 1:D + 1].transpose(1, 2)
    assert torch.equal(osf.osf_attn_kv4(odd, cache), osf.osf_attn_kv4(odd.contiguous(), cache))


@pytest.mark.parametrize("D", [64, 128])
def test_attention_sharp_scores_and_query_magnitudes(osf, D):
    """One key far above the others, scores that climb along the cache, tiny, huge and zero query rows."""
    q, _ = rows((1, 4, 1, D), 21, "bf16")
    q[0, 1] *= 40
    q[0, 2] = 0
    q[0, 3] *= 2.0 ** -40
    check_attention(osf, 1, 4, 1, 1, 500, D, "bf16", seed=22, q=q)
    cache, rec = random_cache(1, 1, 600, D, 23)
    pairs = cache[..., D:D + D // 8].clone().view(torch.bfloat16).unflatten(-1, (-1, 2))
    ramp = torch.linspace(0, 3, 600, device="cuda").view(1, 1, 600, 1)
    pairs[..., 1] = (pairs[..., 1].float() + ramp).to(torch.bfloat16)
    cache[..., D:D + D // 8] = pairs.flatten(-2).contiguous().view(torch.uint8)
    q = torch.ones(1, 2, 1, D, device="cuda", dtype=torch.bfloat16)
    q[0, 1] = -1
    check_attention(osf, 1, 2, 1, 1, 600, D, "bf16", seed=24, q=q, cache=cache)
    big = torch.zeros(1, 1, 1, D, device="cuda", dtype=torch.bfloat16)
    big[..., 5] = 2.0 ** 90
    small = cache.clone()
    p2 = small[..., D:D + D // 8].clone().view(torch.bfloat16) * 2.0 ** -90
    small[..., D:D + D // 8] = p2.contiguous().view(torch.uint8)
    check_attention(osf, 1, 1, 1, 1, 600, D, "bf16", seed=25, q=big, cache=small, scale=1.0)


def test_attention_length_out_of_range_is_cut_and_recorded(osf):
    cache, _ = random_cache(2, 1, 50, 64, 31)
    q, _ = rows((2, 2, 1, 64), 32, "bf16")
    got = osf.osf_attn_kv4(q, cache, lens=ints([60, -3]))
    assert osf.osf_device_status() == osf.OSF_ERR_INVALID
    assert torch.equal(got, osf.osf_attn_kv4(q, cache, lens=ints([50, 0])))
    assert osf.osf_device_status() == osf.OSF_OK


def test_attention_over_an_empty_cache(osf):
    q, _ = rows((2, 2, 1, 64), 33, "bf16")
    cache = torch.empty(2, 1, 0, 80, dtype=torch.uint8, device="cuda")
    lse = torch.zeros(2, 2, 1, device="cuda")
    out = osf.osf_attn_kv4(q, cache, lse=lse)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_workspace_too_small_is_refused(osf):
    cache, _ = random_cache(1, 1, 4096, 128, 34)
    q, _ = rows((1, 4, 1, 128), 35, "bf16")
    w = torch.zeros(1, 1, 4096, device="cuda")
    n = osf.osf_attn_kv4_workspace_bytes(osf.OSF_BF16, 1, 4, 1, 1, 4096, 128, True)
    with pytest.raises(osf.OsfError) as err:
        osf.osf_attn_kv4(q, cache, weights=w, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert err.value.status == osf.OSF_ERR_WORKSPACE


def test_workspace_that_is_not_aligned_is_refused(osf):
    cache, _ = random_cache(1, 1, 4096, 128, 36)
    q, _ = rows((1, 4, 1, 128), 37, "bf16")
    n = osf.osf_attn_kv4_workspace_bytes(osf.OSF_BF16, 1, 4, 1, 1, 4096, 128)
    with pytest.raises(osf.OsfError) as err:
        osf.osf_attn_kv4(q, cache, workspace=torch.empty(n + 4, dtype=torch.uint8, device="cuda")[4:])
    assert err.value.status == osf.OSF_ERR_INVALID
