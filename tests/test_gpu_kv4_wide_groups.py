"""4-bit records of groups whose range comes near the end of float32's, or passes it: byte for byte the oracle's."""
import numpy as np
import pytest

import oracle
import seeded_inputs as si
from conftest import bf16_tensor, f32_tensor

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FAR = float(np.finfo(np.float32).max)
TOP = float(np.array(0x7F7F0000, np.uint32).view(np.float32))   # the largest bfloat16


def groups():
    """Float64 values [n, 32] that float32 holds."""
    rng = np.random.default_rng(70)
    g = []
    for lo, hi in ((-2e38, 2e38), (-TOP, TOP), (-TOP, FAR), (0.0, FAR), (-1e30, 3.1e38), (-1.5e38, 1.55e38), (-3e38, 1e37), (-TOP, 1e-45),
                   (-TOP, 0.0), (-TOP, -TOP), (FAR, FAR), (3e38, 3.4e38), (0.0, 3.0e38), (0.0, 3.01e38), (-2.0 ** 126, 2.0 ** 126)):
        x = rng.uniform(0, 1, 32) * (hi / 4 - lo / 4) * 4 + lo
        x[:2] = lo, hi
        g.append(x)
        x = np.array([lo, hi] + [1e-45, -1e-45, 0.0, 1.0] * 7 + [lo, hi]) if lo < 0 < hi else np.full(32, lo)
        g.append(x)
    for s, m in ((2.0 ** 124, -TOP), (1.5 * 2.0 ** 124, -2.0 ** 127), (2.0 ** 123, 0.0), (2.0 ** 122, -2.0 ** 126), (1.9921875 * 2.0 ** 122, 0.0)):
        # on the ties of a code, and one step to each side
        ties = (m + s * (np.arange(15) + 0.5)).astype(np.float32)
        x = np.concatenate([[m, m + 15 * s], ties, np.nextafter(ties, np.float32(np.inf))])
        y = np.concatenate([[m, m + 15 * s], ties, np.nextafter(ties, np.float32(-np.inf))])
        g += [x[:32], y[:32]]
    g = np.clip(np.array(g, np.float64), -TOP, FAR).astype(np.float32)
    return np.concatenate([g, np.ones((-len(g) % 4, 32), np.float32)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_groups_of_any_finite_range_are_stored_exactly(osf, dtype):
    x = groups().reshape(1, 1, -1, 128)
    if dtype == "bf16":
        bits = (x.view(np.uint32) >> 16).astype(np.uint16)           # towards zero: none becomes infinite
        t, x = bf16_tensor(bits), si.bf16_bits_to_f32(bits)
    else:
        t = f32_tensor(x)
    n = x.shape[2]
    cache = torch.zeros(1, 1, n, 160, dtype=torch.uint8, device="cuda")
    osf.osf_kv4_append(t, t.flip(2), cache)
    want = oracle.records(x, x[:, :, ::-1])
    diff = np.argwhere(cache.cpu().numpy() != want)
    assert len(diff) == 0, diff[:20].tolist()
    (K, V), _ = oracle.record_values(want)
    for got, ref in zip(osf.osf_kv4_read(cache, 128, n, dtype=torch.float32), (K, V)):
        got = got.double().cpu().numpy()
        with np.errstate(over="ignore"):
            assert np.array_equal(got, ref.astype(np.float32).astype(np.float64))   # one rounding


def test_a_value_below_the_least_finite_bfloat16_reads_nan(osf):
    x = torch.zeros(1, 1, 1, 64, device="cuda")
    x[..., 5] = -FAR
    cache = torch.zeros(1, 1, 1, 80, dtype=torch.uint8, device="cuda")
    osf.osf_kv4_append(x, x, cache)
    k, v = osf.osf_kv4_read(cache, 64, 1, dtype=torch.float32)
    assert bool(torch.isnan(k[..., :32]).all()) and bool((k[..., 32:] == 0).all()) and torch.equal(torch.isnan(k), torch.isnan(v))
