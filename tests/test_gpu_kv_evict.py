"""osf_kv_evict against the sorted definition: every index, row, weight and length exactly."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def check(osf, w, budget, sinks=0, recent=0, lens=None, row=(torch.bfloat16, 64), two=True, in_place=False, S_out=None):
    """w: numpy float32 [B, Hkv, S]."""
    B, Hkv, S = w.shape
    dt, D = row
    make = lambda: (torch.randint(0, 120, (B, Hkv, S, D), device="cuda").to(dt))  # noqa: E731
    k, v = make(), (make() if two else None)
    wt = torch.from_numpy(w).cuda()
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    k0, v0, w0 = k.clone(), None if v is None else v.clone(), w.copy()
    kw = {}
    if in_place:
        kw = dict(k_out=k, v_out=v, weights_out=wt, lens_out=lt)
        S_out = S
    elif S_out is not None:
        fill = lambda t: torch.full((B, Hkv, S_out, D), 77, device="cuda").to(t.dtype)  # noqa: E731
        kw = dict(k_out=fill(k), v_out=None if v is None else fill(v))
    else:
        S_out = budget
    old = {n: kw[n].clone() for n in ("k_out", "v_out") if kw.get(n) is not None}
    ko, vo, wo, lo, idx = osf.osf_kv_evict(k, v, wt, budget, lens=lt, sinks=sinks, recent=recent, **kw)
    gi, gw = idx.cpu().numpy(), wo.cpu().numpy()
    for b in range(B):
        n = S if lens is None else min(max(lens[b], 0), S)
        new = min(n, budget)
        assert int(lo[b]) == new
        for h in range(Hkv):
            keep = oracle.evict(w0[b, h], n, budget, sinks, recent)
            assert np.array_equal(gi[b, h, :new], keep) and np.all(gi[b, h, new:] == -1)
            at = torch.from_numpy(keep).cuda()
            assert torch.equal(ko[b, h, :new], k0[b, h][at])
            if two:
                assert torch.equal(vo[b, h, :new], v0[b, h][at])
            assert np.array_equal(gw[b, h, :new], w0[b, h][keep], equal_nan=True) and np.all(gw[b, h, new:] == 0)
            for name, t in (("k_out", ko), ("v_out", vo)):
                if name in old:   # rows behind the kept ones stay as they were
                    assert torch.equal(t[b, h, new:], old[name][b, h, new:])
    assert osf.osf_device_status() == osf.OSF_OK


def weights(B, H, S, seed, kind="skewed"):
    rng = np.random.default_rng(seed)
    if kind == "skewed":
        w = rng.random((B, H, S)) ** 6 * 8
        w[rng.random((B, H, S)) < 0.2] = 0
    elif kind == "ties":
        w = rng.integers(0, 4, (B, H, S)).astype(float)
    elif kind == "equal":
        w = np.full((B, H, S), 0.25)
    else:   # close together: the last bits decide
        w = 1.0 + rng.integers(0, 5000, (B, H, S)) * 2.0 ** -23
    return w.astype(np.float32)


@pytest.mark.parametrize("kind", ["skewed", "ties", "equal", "close"])
@pytest.mark.parametrize("S,budget,sinks,recent", [(1, 1, 0, 0), (2, 1, 0, 0), (2, 1, 1, 0), (2, 1, 0, 1), (33, 32, 0, 0), (100, 100, 3, 5),
                                                   (100, 99, 3, 5), (1000, 10, 4, 6), (1000, 1, 0, 0), (1000, 700, 0, 100),
                                                   (5000, 2500, 4, 500), (9001, 4000, 1, 7)])
def test_selection(osf, kind, S, budget, sinks, recent):
    check(osf, weights(2, 2, S, S + budget, kind), budget, sinks, recent)


@pytest.mark.parametrize("kind", ["skewed", "ties", "equal", "close"])
@pytest.mark.parametrize("S", [8192, 8193, 20000, 70001, 200000])
def test_selection_over_several_slices(osf, kind, S):
    check(osf, weights(1, 2, S, S, kind), S // 3, 4, 1000, row=(torch.uint8, 16), two=False)


def test_selection_longer_than_the_slices_hold(osf):
    """More keys than eight CTAs keep in shared memory: they are read again in every pass."""
    for kind in ("skewed", "ties"):
        check(osf, weights(1, 1, 500003, 12, kind), 200001, 3, 777, row=(torch.uint8, 4), two=False)


def test_ragged_lengths(osf):
    lens = [0, 1, 63, 64, 65, 500, 1000]
    for in_place in (False, True):
        check(osf, weights(len(lens), 3, 1000, 1), 64, 2, 10, lens=lens, in_place=in_place)
        check(osf, weights(len(lens), 3, 1000, 2), 600, 2, 100, lens=lens, in_place=in_place)


@pytest.mark.parametrize("row", [(torch.bfloat16, 128), (torch.float32, 64), (torch.uint8, 160), (torch.uint8, 80), (torch.uint8, 40),
                                 (torch.uint8, 7), (torch.bfloat16, 33), (torch.bfloat16, 1), (torch.float32, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_row_sizes(osf, row, in_place):
    check(osf, weights(2, 2, 777, 3), 300, 4, 20, row=row, in_place=in_place)
    check(osf, weights(1, 1, 3000, 4), 2900, 0, 0, row=row, in_place=in_place, two=False)


def test_in_place_long(osf):
    check(osf, weights(2, 2, 20000, 5), 9000, 4, 500, row=(torch.bfloat16, 128), in_place=True, lens=[20000, 9500])


def test_roomier_output(osf):
    check(osf, weights(2, 2, 400, 6), 100, 4, 20, lens=[400, 50], S_out=256)


def test_nan_infinite_and_negative_weights(osf):
    w = weights(1, 2, 300, 7)
    w[0, 0, ::7] = np.nan
    w[0, 0, 5] = np.inf
    w[0, 0, 11] = -np.inf
    w[0, 1] -= 2
    w[0, 1, ::3] = -0.0
    for budget in (10, 250, 280):
        check(osf, w, budget, 2, 3)


def test_length_out_of_range_is_cut_and_recorded(osf):
    w = torch.from_numpy(weights(2, 1, 50, 8)).cuda()
    k = torch.zeros(2, 1, 50, 16, dtype=torch.uint8, device="cuda")
    _, _, _, lo, idx = osf.osf_kv_evict(k, None, w, 20, lens=torch.tensor([70, -4], dtype=torch.int32, device="cuda"))
    assert osf.osf_device_status() == osf.OSF_ERR_INVALID
    assert lo.tolist() == [20, 0] and bool((idx[1] == -1).all())
    assert osf.osf_device_status() == osf.OSF_OK


def test_empty_cache(osf):
    k = torch.empty(2, 3, 0, 64, device="cuda")
    ko, vo, wo, lo, idx = osf.osf_kv_evict(k, k.clone(), torch.empty(2, 3, 0, device="cuda"), 4, sinks=1)
    assert bool((ko == 0).all()) and bool((vo == 0).all()) and bool((wo == 0).all())
    assert lo.tolist() == [0, 0] and bool((idx == -1).all())
    assert osf.osf_device_status() == osf.OSF_OK


def test_weights_alone(osf):
    """Without cache arrays the call only selects (the caller gathers by idx)."""
    w = weights(1, 2, 90, 9)
    wt = torch.from_numpy(w).cuda()
    out, idx = torch.empty(1, 2, 30, device="cuda"), torch.empty(1, 2, 30, dtype=torch.int32, device="cuda")
    st = osf.lib().osf_kv_evict(None, None, 0, None, None, 0, wt.data_ptr(), out.data_ptr(), None, None, idx.data_ptr(), 1, 2, 90, 30, 30, 1,
                                2, torch.cuda.current_stream().cuda_stream)
    assert st == osf.OSF_OK
    torch.cuda.synchronize()
    for h in range(2):
        assert np.array_equal(idx[0, h].cpu().numpy(), oracle.evict(w[0, h], 90, 30, 1, 2))
