"""A serving loop whose every step is worked out on the host: append, attention with accumulated weights, and eviction in
place with the lengths written over the old ones.  The choice follows the device's own weights (so near ties cannot
differ); records, weights, lengths and indices are then exact.

Tolerances, u = 2^-24, h = 2^-8, A = sum p (|minimum| + scale * code), T = the largest scale sum |q| |k|, |k| taken as
|minimum| + scale * code: a score is within 2 (D + 8) u T (products of exact operands, truncated sums), so p within
e = 2 (D + 8) u T + 4 u (T + 12) + 2^-21 of itself, as is its denominator; p * scale has 11 bits and the result is a
bfloat16: O is within (2 e + 2^-11 + 2 (n + 8) u) A + h |O|.  A step's weights are sums of G rows of p: 2 e + 8 u of
them, and an addition's u."""
import numpy as np
import pytest

import oracle
from test_gpu_cache_run import normal
from test_gpu_kv4 import H, U

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("D", [64, 128, 96])
def test_every_step_of_a_serving_loop(osf, D):
    B, Hq, Hkv, P, S, budget = 2, 8, 2, 260, 290, 180
    sinks, recent = 4, 32
    R = osf.osf_kv4_record_bytes(D)
    k, v = normal((B, Hkv, P, D), 1), normal((B, Hkv, P, D), 2)
    cache = torch.zeros(B, Hkv, S, R, dtype=torch.uint8, device="cuda")
    counts = [P, 150]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    osf.osf_kv4_append(k, v, cache, lens=lens, counts=torch.tensor(counts, dtype=torch.int32, device="cuda"))
    lens += torch.tensor(counts, dtype=torch.int32, device="cuda")
    n = list(counts)
    w = torch.zeros(B, Hkv, S, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    for b in range(B):
        w[b, :, :n[b]] = torch.rand(Hkv, n[b], generator=g, device="cuda")
    w[0, 0, 20:60] = 0.25                                   # ties, of which the lower indices stay
    for step in range(9):
        if step % 4 == 0:
            before, w0, n0 = cache.cpu().numpy(), w.cpu().numpy(), list(n)
            _, _, _, _, idx = osf.osf_kv_evict(cache, None, w, budget, lens=lens, sinks=sinks, recent=recent, k_out=cache,
                                               weights_out=w, lens_out=lens)
            after, w1, idx = cache.cpu().numpy(), w.cpu().numpy(), idx.cpu().numpy()
            for b in range(B):
                n[b] = min(n0[b], budget)
                for h in range(Hkv):
                    keep = oracle.evict(w0[b, h], n0[b], budget, sinks, recent)
                    assert np.array_equal(idx[b, h, :n[b]], keep) and np.all(idx[b, h, n[b]:] == -1)
                    assert np.array_equal(after[b, h, :n[b]], before[b, h, keep])
                    assert np.array_equal(after[b, h, n[b]:], before[b, h, n[b]:])   # rows behind are left as they were
                    assert np.array_equal(w1[b, h, :n[b]], w0[b, h, keep]) and np.all(w1[b, h, n[b]:] == 0)
            assert lens.tolist() == n
        qn, kn, vn = (normal((B, h, 1, D), 100 + 3 * step + i) for i, h in enumerate((Hq, Hkv, Hkv)))
        before = cache.cpu().numpy()
        osf.osf_kv4_append(kn, vn, cache, lens=lens)
        lens += 1
        for b in range(B):
            before[b, :, n[b]] = oracle.records(kn[b, :, 0].double().cpu().numpy(), vn[b, :, 0].double().cpu().numpy())
            n[b] += 1
        assert np.array_equal(cache.cpu().numpy(), before)
        w0 = w.double().cpu().numpy()
        out = osf.osf_attn_kv4(qn, cache, lens=lens, mask="bottom_right", weights=w, accumulate=True)
        O, _, W, A = oracle.attention_records(qn.double().cpu().numpy(), before, n, "bottom_right")
        _, (Km, _) = oracle.record_values(before)
        qa = np.abs(qn.double().cpu().numpy())
        T = max((qa[b, h] @ Km[b, h * Hkv // Hq, :n[b]].T).max() for b in range(B) for h in range(Hq)) * D ** -0.5
        e = 2 * (D + 8) * U * T + 4 * U * (T + 12) + 2.0 ** -21
        tol = (2 * e + 2.0 ** -11 + 2 * (max(n) + 8) * U) * A + H * np.abs(O)
        assert np.all(np.abs(out.double().cpu().numpy() - O) <= tol)
        assert np.all(np.abs(w.double().cpu().numpy() - w0 - W) <= (2 * e + 8 * U) * W + U * (w0 + W))
    assert osf.osf_device_status() == osf.OSF_OK
