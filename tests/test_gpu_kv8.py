"""The paged 8-bit cache (osf_kv8_append, osf_kv8_read, osf_attn_kv8) against oracle.kv8 and oracle.attention_window.

Codes, scales and the values read back are exact: equal.  Rotated queries, a c - b s in float32: the product b s rounded
(2^-24 of it), the fused difference (2^-24 of that), then the type (2^-8 in bfloat16).
Attention, from what is rounded: bfloat16 O once (2^-8 |O|), P to float16 (2^-11 of size = sum P |V|); the queries
are exact, scores and sums float32 (2^-24 a step, D + log steps deep: below 2^-15 of size with the inputs here).
float32: 2e-5 of size, as the windowed forward.  lse: 2e-5 absolute and relative.
"""
import numpy as np
import pytest

import oracle
import seeded_inputs as si
from conftest import bf16_tensor, f32_tensor
from test_gpu_attention_bwd import f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def new_cache(B, Hkv, per, P, D, seed=0, extra=2, fill=None):
    """Pages full of random bytes (NaN codes among them), scales that mean nothing, a shuffled table; numpy."""
    rng = np.random.default_rng(seed)
    n_pages = B * per + extra
    pages = rng.integers(0, 256, (n_pages, 2, Hkv, P, D)).astype(np.uint8) if fill is None else \
        np.full((n_pages, 2, Hkv, P, D), fill, np.uint8)
    scales = np.ldexp(1.0, rng.integers(-9, 3, (n_pages, 2, Hkv))).astype(np.float32)
    table = rng.permutation(n_pages)[:B * per].reshape(B, per).astype(np.int32)
    return pages, scales, table


def to_gpu(*arrays):
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def tables(positions, R, seed=0):
    if not R:
        return None, None
    ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(R // 2) * 2 / R) + seed
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def rows(rng, shape, dtype):
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-3, 4, shape[:2] + (1, 1))
    x = x.astype(np.float32)
    if dtype == "bf16":
        x = torch.from_numpy(x).bfloat16().float().numpy()
    return x, torch.from_numpy(x).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def check_rotated(got, q, ref, dtype):
    """ref: rotated exactly, but for one rounding to float32 (2^-24 more)."""
    u = 2.0 ** -8 if dtype == "bf16" else 0.0
    pair = np.abs(q).max(-1, keepdims=True)   # |b s| is at most the row's largest
    bound = 2.0 ** -24 * pair + (u + 2.0 ** -23) * np.abs(ref)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= bound * (1 + 1 / 16))


CASES = [
    # B, Hkv, n, D, P, per, lens, counts, rot, interleaved
    (1, 1, 1, 32, 16, 1, [0], None, 32, False),
    (2, 2, 1, 128, 64, 3, [0, 70], None, 128, False),
    (2, 3, 5, 64, 16, 4, [13, 16], None, 64, True),
    (3, 2, 40, 96, 32, 4, [0, 31, 60], [40, 0, 17], 48, False),
    (1, 2, 300, 256, 128, 4, [100], None, 64, True),
    (2, 1, 129, 64, 64, 5, [1, 127], [129, 128], 0, False),
    (1, 4, 33, 160, 16, 4, [7], None, 152, False),
    (5, 1, 1, 64, 128, 2, [0, 1, 127, 128, 255], None, 8, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,n,D,P,per,lens,counts,rot,inter", CASES)
def test_append_and_read(osf, dtype, B, Hkv, n, D, P, per, lens, counts, rot, inter):
    rng = np.random.default_rng(n + D)
    pages, scales, table = new_cache(B, Hkv, per, P, D, seed=n)
    cos, sin = tables(per * P, rot)
    # what is there already, of another size now and then, put there in two steps
    for step in (0, 1):
        old, _ = rows(rng, (2 * B, Hkv, per * P, D), dtype)
        m = np.maximum(np.array(lens) - 3 * (1 - step), 0)
        for b in range(B):
            at = 0 if step == 0 else int(max(lens[b] - 3, 0))
            cnt = int(m[b]) - at
            if cnt > 0:
                oracle.kv8_append(old[b:b + 1, :, :cnt], old[B + b:B + b + 1, :, :cnt], pages, scales, table[b:b + 1], [at])
    k, K = rows(rng, (B, Hkv, n, D), dtype)
    v, V = rows(rng, (B, Hkv, n, D), dtype)
    q, Q = rows(rng, (B, 2 * Hkv, n, D), dtype)
    gp, gs, gt, gl, gc, gcos, gsin = to_gpu(pages, scales, table, np.array(lens, np.int32),
                                            None if counts is None else np.array(counts, np.int32), cos, sin)
    mark = torch.full_like(Q, 77.0)
    qo = osf.osf_kv8_append(K, V, gp, gs, gt, lens=gl, counts=gc, cos=gcos, sin=gsin, interleaved=inter, q=Q, q_out=mark)
    oracle.kv8_append(k, v, pages, scales, table, lens, counts, cos, sin, inter)
    assert np.array_equal(gs.cpu().numpy(), scales)
    assert np.array_equal(gp.cpu().numpy(), pages)
    new = [n] * B if counts is None else counts
    for b in range(B):
        ref = oracle.rotate(q[b], np.arange(lens[b], lens[b] + n) if cos is None else
                            np.minimum(np.arange(lens[b], lens[b] + n), len(cos) - 1), cos, sin, inter)
        check_rotated(qo[b, :, :new[b]], q[b, :, :new[b]], ref[:, :new[b]], dtype)
        assert (qo[b, :, new[b]:] == 77).all()
    # read back from around the new tokens
    starts = np.array([x - 2 for x in lens], np.int32)
    after = np.array([x + y for x, y in zip(lens, new)], np.int32)
    for dt in (torch.float32, torch.bfloat16):
        rk, rv = osf.osf_kv8_read(gp, gs, gt, n + 4, starts=to_gpu(starts)[0], lens=to_gpu(after)[0], dtype=dt)
        for b in range(B):
            kv = oracle.kv8_values(pages, scales, table[b], int(after[b]))
            for got, ref in zip((rk, rv), kv):
                want = np.zeros((Hkv, n + 4, D))
                for t in range(n + 4):
                    if 0 <= starts[b] + t < after[b]:
                        want[:, t] = ref[:, starts[b] + t]
                assert np.array_equal(got[b].double().cpu().numpy(), want, equal_nan=True)
    # a position behind the tables is recorded (the last case of each kind has none)
    assert osf.osf_device_status() == osf.OSF_OK


def test_codes_at_every_tie_and_edge(osf):
    """Values at and around the midpoints of codes, the largest of a binade, subnormals of the scale, signed zeros."""
    v = oracle.e4m3_values()[:127]
    mid = (v[1:] + v[:-1]) / 2
    x = np.r_[v, mid, np.nextafter(mid.astype(np.float32), 0), np.nextafter(mid.astype(np.float32), 500), 0.0, 2.0 ** -11, 2.0 ** -10]
    x = x[x <= 448].astype(np.float32)
    x = np.r_[x, -x][:32 * 16]
    for shift in (0, -6, 40, -100, 110):
        k = np.ldexp(np.resize(x, (1, 1, 32, 32)), shift).astype(np.float32)
        k[0, 0, 0, 0] = k[0, 0, 16, 0] = np.ldexp(448.0, shift)   # both pages: the same scale
        pages, scales, table = new_cache(1, 1, 2, 16, 32, seed=1)
        gp, gs, gt = to_gpu(pages, scales, table)
        osf.osf_kv8_append(f32_tensor(k), f32_tensor(-k), gp, gs, gt)
        oracle.kv8_append(k, -k, pages, scales, table)
        assert np.array_equal(gp.cpu().numpy(), pages) and np.array_equal(gs.cpu().numpy(), scales)


def test_rotation_is_rounded_once(osf):
    """K's products that cancel to their last bits: the code of the float32 nearest to a c - b s."""
    rng = np.random.default_rng(8)
    n, D = 64, 64
    c = rng.uniform(0.5, 1, (n, 32)).astype(np.float32)
    s = rng.uniform(0.5, 1, (n, 32)).astype(np.float32)
    k = rng.standard_normal((1, 1, n, D)).astype(np.float32)
    k[0, 0, :, 32:] = (k[0, 0, :, :32] * (c / s)).astype(np.float32)   # a c = b s to 2^-24
    pages, scales, table = new_cache(1, 1, 1, 64, D)
    gp, gs, gt, gc, gsn = to_gpu(pages, scales, table, c, s)
    osf.osf_kv8_append(f32_tensor(k), f32_tensor(k), gp, gs, gt, cos=gc, sin=gsn)
    oracle.kv8_append(k, k, pages, scales, table, None, None, c, s)
    assert np.array_equal(gp.cpu().numpy(), pages) and np.array_equal(gs.cpu().numpy(), scales)
    ref = oracle.rotate(k[0], np.arange(n), c, s, False)
    assert (np.abs(ref[0, :, :32]) < 1e-5).mean() > 0.9   # the input does what it is for
    # a = b and c = s to a step: both results are differences or twice a product, by turns of the sign
    k3 = np.repeat(k[..., :32], 2, -1).reshape(1, 1, n, 32, 2).transpose(0, 1, 2, 4, 3).reshape(1, 1, n, D).copy()
    s3 = np.nextafter(c, np.float32(2)) * np.where(np.arange(32) % 2, 1, -1).astype(np.float32)
    gp, gs, gt, g3 = to_gpu(pages, scales, table, s3)
    osf.osf_kv8_append(f32_tensor(k3), f32_tensor(k3), gp, gs, gt, cos=gc, sin=g3)
    oracle.kv8_append(k3, k3, pages, scales, table, None, None, c, s3)
    assert np.array_equal(gp.cpu().numpy(), pages) and np.array_equal(gs.cpu().numpy(), scales)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_rotation_to_the_ties_of_codes(osf, dtype, inter):
    """a c - b s (b = 1) a quarter of a unit in the last place after another around the midpoints of codes and around 448, where
    the scale grows: the code of the value rounded once to float32."""
    v = oracle.e4m3_values()[:127]
    mids = np.r_[(v[9:] + v[8:-1]) / 2, v[8:127:7], 448.0, 448.0]
    n, D, R = 64, 64, 64
    for shift in (0, -30):
        rng = np.random.default_rng(11 - shift)
        mid = np.ldexp(rng.choice(mids, (n, R // 2)), shift).astype(np.float64)
        a = rows(rng, (1, 1, n, R // 2), dtype)[0][0, 0]
        a[a == 0] = 1
        c = (mid / a).astype(np.float32)
        step = np.spacing(mid.astype(np.float32)).astype(np.float64)
        s = (a.astype(np.float64) * c - mid - rng.integers(-12, 13, mid.shape) * step / 4).astype(np.float32)
        k = np.ones((1, 1, n, D), np.float32)
        k[0, 0, :, slice(0, None, 2) if inter else slice(0, R // 2)] = a
        near = oracle.rotate(k[0], np.arange(n), c, s, inter)[0][:, slice(0, None, 2) if inter else slice(0, R // 2)]
        assert np.all(np.abs(near - mid) <= 5 * step)   # the input does what it is for
        for P in (16, 64):
            pages, scales, table = new_cache(1, 1, n // P, P, D, seed=2)
            gp, gs, gt, gc, gsn = to_gpu(pages, scales, table, c, s)
            K = torch.from_numpy(k).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
            osf.osf_kv8_append(K, K, gp, gs, gt, cos=gc, sin=gsn, interleaved=inter)
            oracle.kv8_append(k, k, pages, scales, table, None, None, c, s, inter)
            assert np.array_equal(gp.cpu().numpy(), pages) and np.array_equal(gs.cpu().numpy(), scales)


def test_nan_and_infinity_are_stored_as_nan(osf):
    for dt in (torch.float32, torch.bfloat16):
        k = torch.ones(1, 1, 20, 32, device="cuda", dtype=dt)
        k[0, 0, 3, 5], k[0, 0, 17, 1], k[0, 0, 18, 2] = float("nan"), float("inf"), -float("inf")
        pages, scales, table = to_gpu(*new_cache(1, 1, 2, 16, 32, fill=0))
        osf.osf_kv8_append(k, k, pages, scales, table)
        rk, rv = osf.osf_kv8_read(pages, scales, table, 20, dtype=torch.float32)
        want = k.float().clone()
        want[~torch.isfinite(want)] = float("nan")
        assert torch.equal(torch.nan_to_num(rk, 7.0), torch.nan_to_num(want, 7.0)) and torch.equal(
            torch.nan_to_num(rv, 7.0), torch.nan_to_num(want, 7.0))


def test_bad_tables_lengths_and_counts(osf):
    """Bad entries are skipped, bad lengths cut, both recorded; nothing else is written."""
    P, D = 16, 64
    pages, scales, table = new_cache(3, 1, 3, P, D, seed=5)
    table[0, 1], table[1, 0] = -1, len(pages)
    k, K = rows(np.random.default_rng(0), (3, 1, 40, D), "f32")
    for lens, counts in (([0, 0, 0], None), ([20, 30, -1], None), ([10, 0, 0], [41, -1, 40])):
        gp, gs, gt, gl, gc = to_gpu(pages, scales, table, np.array(lens, np.int32), None if counts is None else np.array(counts, np.int32))
        osf.osf_kv8_append(K, K, gp, gs, gt, lens=gl, counts=gc)
        assert osf.osf_device_status() == osf.OSF_ERR_INVALID and osf.osf_device_status() == osf.OSF_OK
        rp, rs = pages.copy(), scales.copy()
        oracle.kv8_append(k, k, rp, rs, table, lens, None if counts is None else [min(max(c, 0), 40) for c in counts])
        assert np.array_equal(gp.cpu().numpy(), rp) and np.array_equal(gs.cpu().numpy(), rs)
    q = torch.randn(3, 2, 1, D, device="cuda")
    gp, gs, gt = to_gpu(np.full_like(pages, 0x38), np.ones_like(scales), table)   # every value 1
    o = osf.osf_attn_kv8(q, gp, gs, gt, lens=torch.tensor([48, 16, 100], dtype=torch.int32, device="cuda"))
    assert osf.osf_device_status() == osf.OSF_ERR_INVALID
    assert torch.allclose(o[0], torch.ones_like(o[0])) and not o[1].any() and torch.allclose(o[2], torch.ones_like(o[2]))
    # entries that nothing sees are not read: no record
    osf.osf_attn_kv8(q[1:], gp, gs, gt[1:], lens=torch.tensor([48, 20], dtype=torch.int32, device="cuda"), window=8)
    assert osf.osf_device_status() == osf.OSF_OK
    # positions behind the tables
    cos = torch.ones(5, 8, device="cuda")
    osf.osf_kv8_append(K[2:], K[2:], gp, gs, gt[2:], cos=cos, sin=torch.zeros_like(cos))
    assert osf.osf_device_status() == osf.OSF_ERR_INVALID


def fill_cache(B, Hkv, P, D, lens, seed, spread=0):
    """A cache of normal rows; each page's size is 2^(0 .. spread) times another's."""
    rng = np.random.default_rng(seed)
    per = max(1, -(-max(list(lens) + [1]) // P))
    pages, scales, table = new_cache(B, Hkv, per, P, D, seed=seed)
    for b in range(B):
        for t in range(0, lens[b], P):
            c = min(P, lens[b] - t)
            kv = rng.standard_normal((2, 1, Hkv, c, D)) + 0.3
            if spread:
                kv[1] *= 2.0 ** rng.integers(-spread, 1, (1, Hkv, 1, 1))
            oracle.kv8_append(kv[0], kv[1], pages, scales, table[b:b + 1], [t])
    return pages, scales, table


def reference(q, pages, scales, table, lens, window, sinks, scale=None):
    outs = []
    for b in range(q.shape[0]):
        K, V = oracle.kv8_values(pages, scales, table[b], int(lens[b]))
        outs.append(oracle.attention_window(q[b:b + 1], K[None], V[None], window, sinks, scale))
    return [np.concatenate([o[i] for o in outs]) for i in range(3)]


def check_attn(o, lse, ref, dtype, what):
    O, L, size = ref
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    bound = (2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2.0 ** -15) * size) * (1 + 1 / 16) if dtype == "bf16" else 2e-5 * size
    bad = np.abs(got - O) > bound + 1e-30
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {(np.abs(got - O) / (bound + 1e-30)).max():.3g} bounds"
    assert np.array_equal(np.isneginf(gl), np.isneginf(L)), what
    live = ~np.isneginf(L)
    assert np.all(np.abs(gl[live] - L[live]) <= 2e-5 * (1 + np.abs(L[live]))), what


ATTN = [
    # B, Hq, Hkv, Sq, P, lens, window, sinks
    (1, 1, 1, 1, 16, [1], 0, 0),
    (1, 4, 1, 1, 64, [500], 0, 0),
    (3, 8, 2, 1, 32, [0, 33, 700], 0, 0),
    (2, 10, 2, 3, 16, [2, 260], 0, 0),
    (2, 6, 2, 4, 128, [129, 1000], 100, 5),
    (1, 16, 1, 1, 64, [3000], 1, 0),
    (1, 16, 1, 1, 64, [3000], 1, 1),
    (2, 4, 4, 5, 16, [300, 77], 64, 17),
    (2, 8, 1, 7, 64, [640, 641], 128, 130),
    (4, 24, 2, 1, 16, [1, 128, 129, 2000], 0, 0),
    (1, 4, 2, 40, 32, [333], 50, 3),
    (1, 4, 2, 40, 32, [33], 0, 0),
    (2, 3, 3, 2, 64, [5000, 4000], 1500, 4),
    # long enough to be cut over CTAs
    (3, 4, 1, 1, 64, [9000, 5, 4100], 0, 0),
    (1, 8, 1, 1, 32, [6001], 0, 0),
    (2, 16, 1, 1, 64, [0, 7000], 0, 0),
    (2, 4, 1, 5, 128, [8000, 6500], 4000, 200),
]


@pytest.mark.parametrize("dtype,D", [("bf16", 32), ("bf16", 64), ("bf16", 96), ("bf16", 128), ("bf16", 160), ("f32", 64), ("f32", 128), ("f32", 256)])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,P,lens,window,sinks", ATTN)
def test_attention(osf, dtype, D, B, Hq, Hkv, Sq, P, lens, window, sinks):
    pages, scales, table = fill_cache(B, Hkv, P, D, lens, seed=D + Sq)
    q = si.qkv((B, Hq, Sq, D), (1, 1, 1, D), seed=D, dtype=dtype)[0]
    Q = (bf16_tensor if dtype == "bf16" else f32_tensor)(q)
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array(lens, np.int32))
    lse = torch.full((B, Hq, Sq), float("nan"), device="cuda")
    o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl, window=window, sinks=sinks, lse=lse)
    ref = reference(f64(q, dtype), pages, scales, table, lens, window, sinks)
    check_attn(o, lse, ref, dtype, f"{dtype} {D} {B},{Hq},{Hkv},{Sq} P={P} {lens} {window} {sinks}")
    assert osf.osf_device_status() == osf.OSF_OK


@pytest.mark.parametrize("D", [64, 128])
def test_pages_of_very_different_sizes(osf, D):
    """V scales 2^40 apart, with queries that put the weight now here, now there."""
    lens = [900, 1500]
    pages, scales, table = fill_cache(2, 2, 32, D, lens, seed=11, spread=40)
    for mul in (0.0, 1.0, 8.0):
        q, Q = rows(np.random.default_rng(5), (2, 8, 1, D), "bf16")
        q, Q = q * mul, Q * mul
        gp, gs, gt, gl = to_gpu(pages, scales, table, np.array(lens, np.int32))
        lse = torch.empty(2, 8, 1, device="cuda")
        o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl, lse=lse)
        check_attn(o, lse, reference(q, pages, scales, table, lens, 0, 0), "bf16", f"x{mul}")


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_one_heavy_key_and_many_light_ones(osf, dtype, D):
    """The light keys' weights are 2^-12 .. 2^-20 of the heavy one's; their values are larger by as much."""
    n, P = 4000, 64
    rng = np.random.default_rng(2)
    for gap in (12, 16, 20):
        k = np.zeros((1, 1, n, D))
        k[0, 0, 1234, 0] = 1.0
        v = np.full((1, 1, n, D), 2.0 ** gap / 64) * rng.choice([1.0, 1.125, 1.5], (1, 1, n, D))
        v[0, 0, 1234] = 1.0
        pages, scales, table = new_cache(1, 1, -(-n // P), P, D)
        oracle.kv8_append(k, v, pages, scales, table)
        q = np.zeros((1, 2, 1, D))
        q[..., 0] = gap * np.log(2) if dtype == "f32" else float(torch.tensor(gap * np.log(2)).bfloat16())
        q = q.astype(np.float32)
        Q = torch.from_numpy(q).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        gp, gs, gt = to_gpu(pages, scales, table)
        lse = torch.empty(1, 2, 1, device="cuda")
        o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0, lse=lse)
        check_attn(o, lse, reference(q.astype(np.float64), pages, scales, table, [n], 0, 0, 1.0), dtype, f"gap {gap}")


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 32), ("f32", 64)])
@pytest.mark.parametrize("Sq,window,sinks", [(1, 0, 0), (4, 0, 0), (1, 70, 3), (5, 70, 3)])
def test_nan_reaches_only_the_rows_that_see_it(osf, dtype, D, Sq, window, sinks):
    """Slots behind the last token, hidden tokens of the tiles that are read, and one token that only some rows see hold
    NaN codes in K, V, or both."""
    n, P, Hq = 400, 16, 4
    for where in ("k", "v"):
        pages, scales, table = fill_cache(1, 1, P, D, [n], seed=3)
        half = 0 if where == "k" else 1
        see = oracle.window_mask(Sq, n, window, sinks)
        clean = reference_rows = None
        q = si.qkv((1, Hq, Sq, D), (1, 1, 1, D), seed=1, dtype=dtype)[0]
        clean = reference(f64(q, dtype), pages, scales, table, [n], window, sinks)
        hidden = [t for t in range(n) if not see[:, t].any()]
        for t in hidden:
            pages[table[0, t // P], half, 0, t % P] = 0x7f
        bad = n - 1 if Sq > 1 else None          # seen by the last row alone
        if bad is not None:
            pages[table[0, bad // P], half, 0, bad % P, 5] = 0xff
        Q = (bf16_tensor if dtype == "bf16" else f32_tensor)(q)
        gp, gs, gt, gl = to_gpu(pages, scales, table, np.array([n], np.int32))
        lse = torch.empty(1, Hq, Sq, device="cuda")
        o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl, window=window, sinks=sinks, lse=lse)
        rows_ok = slice(0, Sq) if bad is None else slice(0, Sq - 1)
        check_attn(o[:, :, rows_ok], lse[:, :, rows_ok], [x[:, :, rows_ok] for x in clean], dtype, f"{where}")
        if bad is not None:
            last = o[0, :, -1].float()
            if where == "k":
                assert torch.isnan(last).all() and torch.isnan(lse[0, :, -1]).all()
            else:   # that channel alone
                assert torch.isnan(last[:, 5]).all() and torch.isnan(last).sum() == Hq
                assert torch.isfinite(lse).all()


def test_queries_that_are_not_finite(osf):
    pages, scales, table = fill_cache(1, 1, 16, 64, [200], seed=3)
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array([200], np.int32))
    for dt in (torch.bfloat16, torch.float32):
        q = torch.randn(1, 4, 1, 64, device="cuda").to(dt)
        q[0, 1, 0, 3], q[0, 2, 0, 7] = float("nan"), float("inf")
        lse = torch.empty(1, 4, 1, device="cuda")
        o = osf.osf_attn_kv8(q, gp, gs, gt, lens=gl, lse=lse)
        assert torch.isnan(o[0, 1:3]).all() and torch.isnan(lse[0, 1:3]).all()
        assert torch.isfinite(o[0, ::3]).all() and torch.isfinite(lse[0, ::3]).all()


def test_large_and_small_queries(osf):
    """Queries of any size keep their 8 bits (down to 2^-14 of a row's largest)."""
    lens = [300]
    for D in (64, 128):
        pages, scales, table = fill_cache(1, 1, 64, D, lens, seed=4)
        gp, gs, gt, gl = to_gpu(pages, scales, table, np.array(lens, np.int32))
        rng = np.random.default_rng(1)
        for size in (2.0 ** -60, 2.0 ** -10, 2.0 ** 40):
            q, Q = rows(rng, (1, 4, 1, D), "bf16")
            q, Q = q * size, Q * size
            lse = torch.empty(1, 4, 1, device="cuda")
            o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl, lse=lse, scale=0.1 / size)
            check_attn(o, lse, reference(q.astype(np.float64), pages, scales, table, lens, 0, 0, 0.1 / size), "bf16", f"{size}")


def test_strided_queries_and_outputs(osf):
    B, Hq, Hkv, Sq, D, lens = 2, 8, 2, 3, 128, [200, 90]
    pages, scales, table = fill_cache(B, Hkv, 32, D, lens, seed=6)
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array(lens, np.int32))
    q, Q = rows(np.random.default_rng(1), (B, Hq, Sq, D), "bf16")
    ref = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl)
    view = Q.transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.zeros(B, Sq, Hq + 1, D, dtype=Q.dtype, device="cuda")[:, :, :Hq].transpose(1, 2)
    assert torch.equal(osf.osf_attn_kv8(view, gp, gs, gt, lens=gl, out=out), ref)
    odd = torch.zeros(B, Hq, Sq, D + 1, dtype=Q.dtype, device="cuda")[..., 1:]   # rows that start on odd addresses
    odd.copy_(Q)
    assert torch.equal(osf.osf_attn_kv8(odd, gp, gs, gt, lens=gl, out=torch.zeros_like(odd)[..., :]), ref)
    k, K = rows(np.random.default_rng(2), (B, Hkv, 4, D), "bf16")
    base = [x.clone() for x in (gp, gs)]
    osf.osf_kv8_append(K, K, *base, gt, lens=gl)
    odd = torch.zeros(B, Hkv, 4, D + 1, dtype=Q.dtype, device="cuda")[..., 1:]
    odd.copy_(K)
    again = [x.clone() for x in (gp, gs)]
    osf.osf_kv8_append(odd, K.transpose(1, 2).contiguous().transpose(1, 2), *again, gt, lens=gl)
    assert all(torch.equal(a, b) for a, b in zip(base, again))


def test_serving_loop(osf):
    """A windowed model's prompt and decode steps: the prompt through the windowed forward and into the cache, then tokens one
    by one (append with rotated queries, attention with the same window), the whole step captured and replayed."""
    B, Hq, Hkv, D, P, per, window, sinks = 2, 8, 2, 64, 16, 12, 40, 3
    rng = np.random.default_rng(9)
    cos, sin = tables(per * P, D)
    pages, scales, table = new_cache(B, Hkv, per, P, D, seed=1)
    gp, gs, gt, gc, gsn = to_gpu(pages, scales, table, cos, sin)
    n = 90
    k, K = rows(rng, (B, Hkv, n, D), "bf16")
    v, V = rows(rng, (B, Hkv, n, D), "bf16")
    q, Q = rows(rng, (B, Hq, n, D), "bf16")
    rq = osf.osf_kv8_append(K, V, gp, gs, gt, cos=gc, sin=gsn, q=Q)
    oracle.kv8_append(k, v, pages, scales, table, None, None, cos, sin)
    rk, rv = osf.osf_kv8_read(gp, gs, gt, n)
    lens = [n, n]
    lse = torch.empty(B, Hq, n, device="cuda")
    o = osf.osf_attn_fwd_gqa_window(rq, rk, rv, window, sinks, lse=lse)
    ref = reference(rq.double().cpu().numpy(), pages, scales, table, lens, window, sinks)
    assert np.all(np.abs(o.double().cpu().numpy() - ref[0]) <= 2.0 ** -8 * 17 / 16 * (np.abs(ref[0]) + ref[2]))
    kb, vb, qb = (torch.zeros(B, h, 1, D, dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hq))
    qr, ob, gl = torch.empty_like(qb), torch.empty_like(qb), torch.tensor(lens, dtype=torch.int32, device="cuda")
    l1 = torch.empty(B, Hq, 1, device="cuda")
    ws = torch.empty(max(1, osf.osf_attn_kv8_workspace_bytes(osf.OSF_BF16, B, Hq, Hkv, 1, D, P, per, window, sinks)),
                     dtype=torch.uint8, device="cuda")

    def step():
        osf.osf_kv8_append(kb, vb, gp, gs, gt, lens=gl, cos=gc, sin=gsn, q=qb, q_out=qr)
        gl.add_(1)
        osf.osf_attn_kv8(qr, gp, gs, gt, lens=gl, out=ob, window=window, sinks=sinks, lse=l1, workspace=ws)
    graph, snapshot = torch.cuda.CUDAGraph(), [x.clone() for x in (gp, gs, gl)]
    step()
    torch.cuda.synchronize()
    for x, y in zip((gp, gs, gl), snapshot):
        x.copy_(y)
    with torch.cuda.graph(graph):
        step()
    for t in range(30):
        k, K = rows(rng, (B, Hkv, 1, D), "bf16")
        v, V = rows(rng, (B, Hkv, 1, D), "bf16")
        q, Q = rows(rng, (B, Hq, 1, D), "bf16")
        for x, y in zip((kb, vb, qb), (K, V, Q)):
            x.copy_(y)
        graph.replay()
        oracle.kv8_append(k, v, pages, scales, table, lens, None, cos, sin)
        lens = [x + 1 for x in lens]
        assert np.array_equal(gp.cpu().numpy(), pages) and np.array_equal(gs.cpu().numpy(), scales)
        check_attn(ob, l1, reference(qr.double().cpu().numpy(), pages, scales, table, lens, window, sinks), "bf16", f"step {t}")
    assert osf.osf_device_status() == osf.OSF_OK


def test_two_streams_at_once(osf):
    """Calls on two streams, each with its workspace, give what they give alone."""
    lens = [3000]
    pages, scales, table = fill_cache(1, 2, 64, 128, lens, seed=8)
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array(lens, np.int32))
    qs = [torch.randn(1, 8, 1, 128, device="cuda").bfloat16() for _ in range(2)]
    alone = [osf.osf_attn_kv8(q, gp, gs, gt, lens=gl) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(osf.osf_attn_kv8(qs[i], gp, gs, gt, lens=gl))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


def test_mostly_empty_batch(osf):
    """Hundreds of sequences of which few hold tokens: every CTA goes through several empty ones in a row before and after the
    pieces that it has to work on."""
    B, Hq, Hkv, D, P, per = 600, 4, 2, 64, 32, 1000
    rng = np.random.default_rng(2)
    lens = np.zeros(B, np.int32)
    for b in (0, 7, 8, 40, 41, 43, 200, 299, 300, 450, 598):
        lens[b] = rng.integers(1, 700)
    lens[301] = 3000
    used = int(sum(-(-n // P) for n in lens))
    pages, scales, _ = new_cache(1, Hkv, used, P, D, seed=5)
    table, at = np.full((B, per), -1, np.int32), 0   # (entries behind a sequence's last page are not read)
    for b in np.flatnonzero(lens):
        n = -(-int(lens[b]) // P)
        table[b, :n] = np.arange(at, at + n)
        at += n
        kv = rng.standard_normal((2, 1, Hkv, int(lens[b]), D))
        oracle.kv8_append(kv[0], kv[1], pages, scales, table[b:b + 1])
    q, Q = rows(rng, (B, Hq, 1, D), "bf16")
    gp, gs, gt, gl = to_gpu(pages, scales, table, lens)
    lse = torch.empty(B, Hq, 1, device="cuda")
    some = np.flatnonzero(lens)
    ref = reference(q[some].astype(np.float64), pages, scales, table[some], lens[some], 0, 0)
    for _ in range(20):
        o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl, lse=lse)
        check_attn(o[some], lse[some], ref, "bf16", "mostly empty")
        rest = torch.from_numpy(lens == 0).cuda()
        assert (o[rest] == 0).all() and torch.isneginf(lse[rest]).all()
    assert osf.osf_device_status() == osf.OSF_OK


def test_a_cache_past_2_31_bytes(osf):
    """More tokens than 2^22 of D = 256 in one call, into more than 2^31 bytes of pages: what is stored, rotated and read there."""
    D, P, R, n = 256, 128, 8, (1 << 22) + 37
    per = -(-n // P)
    rng = np.random.default_rng(3)
    k, K = rows(rng, (1, 1, 1, D), "bf16")
    v, V = rows(rng, (1, 1, 1, D), "bf16")
    q, Q = rows(rng, (1, 1, 1, D), "bf16")
    wide = [x.expand(1, 1, n, D) for x in (K, V, Q)]   # every token the same row
    ang = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * torch.tensor([1.0, 0.1, 0.01, 0.001], device="cuda", dtype=torch.float64)
    cos, sin = ang.cos().float(), ang.sin().float()
    gp = torch.zeros(per, 2, 1, P, D, dtype=torch.uint8, device="cuda")
    gs = torch.ones(per, 2, 1, device="cuda")
    table = torch.randperm(per, device="cuda", dtype=torch.int32)[None]
    qo = osf.osf_kv8_append(wide[0], wide[1], gp, gs, table, cos=cos, sin=sin, q=wide[2])
    some = np.r_[0, 1, 4097, n // 2, (1 << 22) - 2:(1 << 22) + 2, n - 40:n]
    c, s = cos.cpu().numpy(), sin.cpu().numpy()
    ref = oracle.rotate(np.repeat(q[0], len(some), 1), some, c, s, False)
    check_rotated(qo[0][:, some], np.repeat(q[0], len(some), 1), ref, "bf16")
    # the pages of those tokens, filled again by the oracle
    pages = np.unique(some // P)
    for pg in pages:
        t = np.arange(pg * P, min(n, (pg + 1) * P))
        op, os_ = np.zeros((1, 2, 1, P, D), np.uint8), np.ones((1, 2, 1), np.float32)
        oracle.kv8_append(np.repeat(k, len(t), 2), np.repeat(v, len(t), 2), op, os_, np.zeros((1, 1), np.int32), None, None, c[t], s[t])
        at = int(table[0, pg])
        assert np.array_equal(gp[at].cpu().numpy(), op[0]) and np.array_equal(gs[at].cpu().numpy(), os_[0])
        rk, rv = osf.osf_kv8_read(gp, gs, table, len(t), starts=torch.tensor([t[0]], dtype=torch.int32, device="cuda"),
                                  dtype=torch.float32)
        kv = oracle.kv8_values(op, os_, np.zeros(1, np.int32), len(t))
        assert np.array_equal(rk[0].cpu().numpy(), kv[0]) and np.array_equal(rv[0].cpu().numpy(), kv[1])
    assert osf.osf_device_status() == osf.OSF_OK


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 128), ("bf16", 256)])
def test_attention_over_pages_past_2_31_bytes(osf, dtype, D):
    """A short sequence whose pages lie at the end of a large cache gives what it gives with the same pages in a small one."""
    Hkv, P, n = 8, 128, 1000
    pages, scales, table = fill_cache(1, Hkv, P, D, [n], seed=12)
    n_pages = (1 << 31) // (2 * Hkv * P * D) + 20
    big = torch.zeros(n_pages, 2, Hkv, P, D, dtype=torch.uint8, device="cuda")
    bs = torch.ones(n_pages, 2, Hkv, device="cuda")
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array([n], np.int32))
    big[-len(pages):], bs[-len(pages):] = gp, gs
    q = torch.randn(1, 32, 1, D, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    o = osf.osf_attn_kv8(q, gp, gs, gt, lens=gl)
    assert torch.equal(osf.osf_attn_kv8(q, big, bs, gt + (n_pages - len(pages)), lens=gl), o)
    assert osf.osf_device_status() == osf.OSF_OK


@pytest.mark.parametrize("dtype,B,Hq,Hkv,Sq,D,P,per,lens,window", [
    ("bf16", 1, 8, 2, 1, 128, 64, 100, [6000], 0), ("bf16", 2, 16, 2, 2, 64, 16, 400, [10, 6000], 4000),
    ("bf16", 3, 12, 1, 3, 96, 32, 300, [9000, 1, 0], 0), ("f32", 2, 4, 2, 1, 64, 64, 40, [2000, 30], 0),
    ("bf16", 1, 4, 4, 3, 160, 64, 40, [2500], 1500)])
def test_attention_stays_in_its_workspace(osf, dtype, B, Hq, Hkv, Sq, D, P, per, lens, window):
    code = osf.OSF_BF16 if dtype == "bf16" else osf.OSF_F32
    pages, scales, table = fill_cache(B, Hkv, P, D, [per * P] * B, seed=2)
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array(lens, np.int32))
    _, Q = rows(np.random.default_rng(1), (B, Hq, Sq, D), dtype)
    n = osf.osf_attn_kv8_workspace_bytes(code, B, Hq, Hkv, Sq, D, P, per, window, 4)
    assert n > 0
    whole = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    ref = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl, window=window, sinks=4)
    assert torch.equal(osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl, window=window, sinks=4, workspace=whole[:n]), ref)
    assert (whole[n:] == 0xA5).all()
    for part, status in ((whole[:n - 1], osf.OSF_ERR_WORKSPACE), (whole[8:n + 8], osf.OSF_ERR_INVALID)):
        with pytest.raises(osf.OsfError) as e:
            osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl, window=window, sinks=4, workspace=part)
        assert e.value.status == status


def test_a_prefix_shared_by_two_sequences(osf):
    """Two sequences whose tables name the same full pages, then pages of their own."""
    Hkv, D, P = 2, 64, 16
    rng = np.random.default_rng(4)
    pages, scales, _ = new_cache(1, Hkv, 12, P, D, seed=9)
    table = np.array([[0, 1, 2, 3, -1, -1], [0, 1, 2, 5, 6, 7]], np.int32)
    kv = rng.standard_normal((2, 1, Hkv, 48, D))
    oracle.kv8_append(kv[0], kv[1], pages, scales, table[:1])
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array([48, 48], np.int32))
    k, K = rows(rng, (2, Hkv, 20, D), "bf16")
    counts = [9, 20]
    osf.osf_kv8_append(K, K, gp, gs, gt, lens=gl, counts=to_gpu(np.array(counts, np.int32))[0])
    oracle.kv8_append(k, k, pages, scales, table, [48, 48], counts)
    assert np.array_equal(gp.cpu().numpy(), pages) and np.array_equal(gs.cpu().numpy(), scales)
    lens = [57, 68]
    q, Q = rows(rng, (2, 4, 3, D), "bf16")
    lse = torch.empty(2, 4, 3, device="cuda")
    o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=to_gpu(np.array(lens, np.int32))[0], lse=lse)
    check_attn(o, lse, reference(q.astype(np.float64), pages, scales, table, lens, 0, 0), "bf16", "shared prefix")
    assert osf.osf_device_status() == osf.OSF_OK


def test_two_graphs_with_one_workspace(osf):
    """Two captured calls of different sizes that use one workspace, replayed in turn on one stream."""
    lens = [5000]
    pages, scales, table = fill_cache(1, 2, 64, 64, lens, seed=8)
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array(lens, np.int32))
    qs = [torch.randn(1, 8, s, 64, device="cuda").bfloat16() for s in (1, 4)]
    need = [osf.osf_attn_kv8_workspace_bytes(osf.OSF_BF16, 1, 8, 2, s, 64, 64, gt.shape[1], 0, 0) for s in (1, 4)]
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    alone = [osf.osf_attn_kv8(q, gp, gs, gt, lens=gl) for q in qs]
    outs, graphs = [torch.empty_like(q) for q in qs], []
    for q, o in zip(qs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            osf.osf_attn_kv8(q, gp, gs, gt, lens=gl, out=o, workspace=ws)
    for _ in range(5):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, alone))
