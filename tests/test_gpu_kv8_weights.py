"""osf_attn_kv8 where a channel's output is due to weights far below the largest one: every weight counts with float16's 11 bits.

Bound (as in test_gpu_kv8): bfloat16 O once (2^-8 |O|), P to float16 (2^-11 of size = sum P |V|), sums and weights float32
(2^-15 of size); where scores are large, float32 scores as well: of |s| nats each of two roundings and the accumulation
(2^-24, 2^-24, 2^-22 of it) moves the weight by as much, for the key and for the largest one: 2^-20 |s| of size with 1 / 16 to spare.
"""
import numpy as np
import pytest

import oracle
from test_gpu_kv8 import new_cache, reference, rows, to_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def check(o, ref, what, nats=0.0):
    """Every channel by its own sum P |V|; 2^-133 is half of bfloat16's smallest step."""
    O, _, size = ref
    got = o.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    bound = (2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2.0 ** -15 + 2.0 ** -20 * nats) * size) * (1 + 1 / 16) + 2.0 ** -133
    bad = np.abs(got - O) > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {(np.abs(got - O) / bound).max():.3g} bounds"


def scores(q, K, scale):
    """Scores in nats of rows q [Hq, D] against K [Hkv, n, D]."""
    G = q.shape[0] // K.shape[0]
    return np.einsum("hgd,hnd->hgn", q.reshape(K.shape[0], G, -1), K) * scale


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("n", [8192, 32768])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [4, 8, 16])
def test_a_heavy_key_without_a_value(osf, G, D, n, whole):
    """One key has nearly all of the weight and V = 0, so the output is due to the others alone.  whole: as many items as SMs,
    which are not cut."""
    P = 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hkv = 8 if whole and sms % 8 == 0 else 1
    B = sms // Hkv if whole else 1
    rng = np.random.default_rng(G + D)
    k = rng.standard_normal((1, 1, n, D))
    v = rng.standard_normal((1, 1, n, D))
    k[..., 0] = 0.0
    at = n // 3 + 1
    v[0, 0, at] = 0.0
    q = rng.standard_normal((1, G, 1, D))
    q[..., 0] = 4.0
    q = torch.from_numpy(q).bfloat16().double().numpy()
    light = scores(q[0, :, 0], k[0], D ** -0.5)
    tail = np.log(np.exp(np.delete(light, at, 2)).sum(2)).max()
    for bits in (np.log2(100.0), np.log2(1000.0), 20, 45, 70):   # the others' share of the sum: 2^-bits
        k[0, 0, at] = 0.0
        k[0, 0, at, 0] = (tail + bits * np.log(2)) * D ** 0.5 / 4.0
        pages, scales, table = new_cache(1, 1, -(-n // P), P, D, seed=n)
        oracle.kv8_append(k, v, pages, scales, table)
        # the same for every kv head and sequence
        pages, scales = np.repeat(pages, Hkv, 2), np.repeat(scales, Hkv, 2)
        gp, gs, gt, gl = to_gpu(pages, scales, np.repeat(table, B, 0), np.full(B, n, np.int32))
        Q = torch.from_numpy(np.tile(q, (B, Hkv, 1, 1))).cuda().bfloat16()
        ref = reference(q, pages[:, :, :1], scales[:, :, :1], table, [n], 0, 0)
        o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl)
        nats = 0.0 if bits < 10 else tail + bits
        check(o[:1, :G], ref, f"bits {bits:.3g}", nats)
        check(o[-1:, -G:], ref, f"bits {bits:.3g}, last head", nats)
    assert osf.osf_device_status() == osf.OSF_OK


@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (128, 8), (128, 16), (64, 16), (96, 2), (32, 8)])
def test_pages_with_one_large_channel(osf, D, G):
    """Pages whose V is zero but for one channel, of 2^gap, among ordinary ones: in the other channels the ordinary pages
    are all there is."""
    n, P = 3000, 32
    rng = np.random.default_rng(D + G)
    k = rng.standard_normal((1, 1, n, D))
    q, Q = rows(rng, (1, G, 1, D), "bf16")
    q, Q = q / 4, Q / 4
    for gap in (10, 14, 16, 20, 24, 40, 60, 90):
        v = rng.standard_normal((1, 1, n, D))
        for page in (0, 7, 50, 51, (n - 1) // P):
            v[0, 0, page * P:(page + 1) * P] = 0.0
            v[0, 0, page * P:(page + 1) * P, 5] = 2.0 ** gap * 1.3
        pages, scales, table = new_cache(1, 1, -(-n // P), P, D, seed=gap)
        oracle.kv8_append(k, v, pages, scales, table)
        gp, gs, gt, gl = to_gpu(pages, scales, table, np.array([n], np.int32))
        o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl)
        check(o, reference(q.astype(np.float64), pages, scales, table, [n], 0, 0), f"gap {gap}")


@pytest.mark.parametrize("order", ["mixed", "rising", "falling"])
@pytest.mark.parametrize("D,G,Sq", [(64, 4, 1), (128, 4, 1), (128, 8, 1), (64, 8, 1), (128, 16, 1), (64, 16, 1), (96, 4, 1), (32, 4, 1),
                                    (128, 10, 3)])
def test_a_channel_for_each_depth_of_weight(osf, D, G, Sq, order):
    """Scores spread over 2^0 .. 2^-100 of the largest weight, and V nonzero in one channel for each narrow band of them: each
    channel's output is due to weights of one size.  rising: the largest comes last, so the references move all the way."""
    n, P, deep = 6000, 64, 100.0
    rng = np.random.default_rng(D + G + Sq)
    k = torch.from_numpy(rng.standard_normal((1, 1, n, D))).bfloat16().double().numpy()
    q = rng.standard_normal((1, G, Sq, D)) * 12.0
    q = torch.from_numpy(q).bfloat16().double().numpy()
    pages, scales, table = new_cache(1, 1, -(-n // P), P, D, seed=D)
    oracle.kv8_append(k, k, pages, scales, table)
    k = oracle.kv8_values(pages, scales, table[0], n)[0]
    s = scores(q[0, 0], k, D ** -0.5)[0, Sq - 1]   # the last row of the first head sees all keys
    by = np.argsort(s, kind="stable")
    if order != "mixed":
        by = by if order == "rising" else by[::-1]
        k, s = k[:, by], s[by]
    depth = (s.max() - s) / np.log(2)
    assert (depth < deep).mean() > 0.5 and depth.max() > 60   # the input does what it is for
    band = np.minimum((depth * (D - 1) / deep).astype(int), D - 1)
    v = np.zeros((1, 1, n, D))
    live = depth < deep
    v[0, 0, np.flatnonzero(live), band[live]] = rng.choice([-1.5, 1.0, 1.25, 1.875], live.sum())
    pages, scales, table = new_cache(1, 1, -(-n // P), P, D, seed=D)
    oracle.kv8_append(k[None], v, pages, scales, table)
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array([n], np.int32))
    o = osf.osf_attn_kv8(torch.from_numpy(q).cuda().bfloat16(), gp, gs, gt, lens=gl)
    ref = reference(q, pages, scales, table, [n], 0, 0)
    nats = np.abs(scores(q[0].reshape(G * Sq, D), oracle.kv8_values(pages, scales, table[0], n)[0], D ** -0.5)).max()
    row = [x[:, :1, Sq - 1:] for x in ref]
    check(o[:, :1, Sq - 1:], row, "the row that the bands are made for", nats)
    # the other rows: weights below 2^-100 of the row's largest may count with fewer bits
    O, _, size = ref
    got = o.double().cpu().numpy()
    slack = 2.0 ** -100 * np.abs(v).sum((0, 1, 2))
    bound = (2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2.0 ** -15 + 2.0 ** -20 * nats) * size + slack) * (1 + 1 / 16) + 2.0 ** -133
    assert np.all(np.abs(got - O) <= bound)
    assert osf.osf_device_status() == osf.OSF_OK


@pytest.mark.parametrize("D,G", [(64, 4), (128, 8), (128, 16)])
def test_queries_of_any_size(osf, D, G):
    """Rows up to the largest bfloat16 keep their bits, with a scale that makes up for it."""
    n = 300
    rng = np.random.default_rng(D)
    pages, scales, table = new_cache(1, 1, 5, 64, D, seed=4)
    kv = rng.standard_normal((2, 1, 1, n, D))
    oracle.kv8_append(kv[0], kv[1], pages, scales, table)
    gp, gs, gt, gl = to_gpu(pages, scales, table, np.array([n], np.int32))
    for size in (-110, -100, 100, 105, 110, 120):
        q, Q = rows(rng, (1, G, 1, D), "bf16")
        q, Q = q * 2.0 ** size, Q * 2.0 ** size
        assert torch.isfinite(Q).all()
        scale = 0.1 * 2.0 ** -size
        o = osf.osf_attn_kv8(Q, gp, gs, gt, lens=gl, scale=scale)
        check(o, reference(q.astype(np.float64), pages, scales, table, [n], 0, 0, scale), f"2^{size}")
