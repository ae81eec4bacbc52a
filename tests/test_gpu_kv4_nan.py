"""NaN scores and NaN records in attention over 4-bit records: what they reach, the same on every path."""
import pytest

from test_gpu_kv4 import random_cache, rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

KINDS = [("bf16", 64), ("bf16", 128), ("bf16", 96), ("f32", 64), ("f32", 128)]


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("S", [9, 300, 3000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_row_with_a_nan_score(osf, dtype, D, S, bad):
    """Its output and lse are NaN, so are the weights of the records that it sees; other rows, and records that it does
    not see, are as without it."""
    Sq = 4
    q, _ = rows((1, 4, Sq, D), 61, dtype)
    cache, _ = random_cache(1, 2, S, D, 62)

    def run(q, accumulate):
        lse = torch.zeros(1, 4, Sq, device="cuda")
        w = torch.full((1, 2, S), 0.5, device="cuda")
        out = osf.osf_attn_kv4(q, cache, mask="bottom_right", lse=lse, weights=w, accumulate=accumulate)
        return out, lse, w

    for accumulate in (False, True):
        want = run(q, accumulate)
        nan_q = q.clone()
        nan_q[0, 1, 1] = bad          # head 1 (kv head 0), row 1: sees all but the last two records
        out, lse, w = run(nan_q, accumulate)
        hit = torch.zeros(1, 4, Sq, dtype=torch.bool, device="cuda")
        hit[0, 1, 1] = True
        assert bool(torch.isnan(out[hit]).all()) and torch.equal(out[~hit], want[0][~hit])
        assert bool(torch.isnan(lse[hit]).all()) and torch.equal(lse[~hit], want[1][~hit])
        assert bool(torch.isnan(w[0, 0, :S - 2]).all())
        # one addend fewer: a row that does not see a record adds nothing to it
        assert torch.equal(w[0, 0, S - 2:], want[2][0, 0, S - 2:]) and torch.equal(w[0, 1], want[2][0, 1])
    assert osf.osf_device_status() == osf.OSF_OK


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("S", [9, 300, 3000])
def test_a_nan_key_reaches_the_rows_that_see_it(osf, dtype, D, S):
    Sq = 3
    q, _ = rows((1, 2, Sq, D), 63, dtype)
    cache, _ = random_cache(1, 1, S, D, 64)
    clean_lse, lse = torch.zeros(1, 2, Sq, device="cuda"), torch.zeros(1, 2, Sq, device="cuda")
    want = osf.osf_attn_kv4(q, cache, mask="bottom_right", lse=clean_lse)
    bad = cache.clone()
    bad[0, 0, S - 1, D:D + D // 8] = 0xFF          # K of the last record, which the last row alone sees
    w = torch.zeros(1, 1, S, device="cuda")
    out = osf.osf_attn_kv4(q, bad, mask="bottom_right", lse=lse, weights=w)
    assert torch.equal(out[:, :, :2], want[:, :, :2]) and torch.equal(lse[:, :, :2], clean_lse[:, :, :2])
    assert bool(torch.isnan(out[:, :, 2]).all()) and bool(torch.isnan(lse[:, :, 2]).all()) and bool(torch.isnan(w).all())


@pytest.mark.parametrize("dtype,D", KINDS)
@pytest.mark.parametrize("S", [40, 300])
def test_a_nan_value_reaches_the_rows_that_see_it_whatever_its_weight(osf, dtype, D, S):
    """A record whose weight underflows to 0 still gives NaN to the rows that see it (0 * NaN), inside and outside of the
    tiles that the mask cuts."""
    Sq = 4
    q = torch.ones(1, 2, Sq, D, device="cuda", dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    for at in (2, S - 3):                                            # row 0 does not see record S - 3, rows 1 .. 3 do
        cache, _ = random_cache(1, 1, S, D, 65)
        far = torch.tensor([0.0, -512.0] * (D // 32), dtype=torch.bfloat16, device="cuda").view(torch.uint8)
        cache[0, 0, at, D:D + D // 8] = far                          # K = -512 in every channel: a score of -512 sqrt(D)
        want = osf.osf_attn_kv4(q, cache, mask="bottom_right")
        cache[0, 0, at, D + D // 8:] = 0xFF                          # V: NaN
        out = osf.osf_attn_kv4(q, cache, mask="bottom_right")
        first = 0 if at == 2 else 1
        assert bool(torch.isnan(out[:, :, first:]).all()) and torch.equal(out[:, :, :first], want[:, :, :first])
