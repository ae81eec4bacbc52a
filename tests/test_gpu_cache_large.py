"""The cache operators on arrays of more than 2^32 bytes: the last head's last keys against the same
operation on a small array.

Tolerances, h = 2^-8 (bfloat16's half step), u = 2^-24: an output is rounded twice (the small call's, its own) and its
weights once, 3 h of the sum of |terms|, here at most 3 h (|O| + h); a log-sum-exp within 64 u of its size.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

H, U = 2.0 ** -8, 2.0 ** -24


def test_records_past_32_bits(osf):
    Hkv, S, n, D = 40, 1_000_000, 1000, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(1, Hkv, n, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = (2 * torch.randn(1, Hkv, 1, D, generator=g, device="cuda")).to(torch.bfloat16)
    small = torch.zeros(1, Hkv, n, 160, dtype=torch.uint8, device="cuda")
    osf.osf_kv4_append(k, v, small)
    big = torch.zeros(1, Hkv, S, 160, dtype=torch.uint8, device="cuda")
    assert big.numel() > 2 ** 32
    at = torch.tensor([S - n], dtype=torch.int32, device="cuda")
    osf.osf_kv4_append(k, v, big, lens=at)
    assert torch.equal(big[:, :, S - n:], small) and not bool(big[:, :, :S - n].any())
    for a, b in zip(osf.osf_kv4_read(big, D, n, starts=at), osf.osf_kv4_read(small, D, n)):
        assert torch.equal(a, b)
    # the records before them are zeros: S - n keys of score 0 and value 0
    lse, lse_small = torch.empty(1, Hkv, 1, device="cuda"), torch.empty(1, Hkv, 1, device="cuda")
    w = torch.empty(1, Hkv, S, device="cuda")
    o = osf.osf_attn_kv4(q, big, lse=lse, weights=w).double()
    o_small = osf.osf_attn_kv4(q, small, lse=lse_small).double()
    part = lse_small.double().exp()
    want = torch.log(part + (S - n))
    assert bool(((lse.double() - want).abs() <= 64 * U * (want + 1) + 2.0 ** -18).all())
    ref = o_small * (part / (part + (S - n))).unsqueeze(-1)
    assert bool(((o - ref).abs() <= 3 * H * (ref.abs() + H)).all())
    assert bool(((w.double().sum(-1) - 1).abs() <= 1e-4).all())
    # the heaviest keys: the stored ones
    w.zero_()
    w[:, :, S - n:] = torch.rand(1, Hkv, n, generator=g, device="cuda") + 1
    kept, _, wo, lens, idx = osf.osf_kv_evict(big, None, w, n)
    assert torch.equal(kept, small) and torch.equal(wo, w[:, :, S - n:]) and lens.tolist() == [n]
    assert bool((idx == torch.arange(S - n, S, device="cuda", dtype=torch.int32)).all())
    assert osf.osf_device_status() == osf.OSF_OK


@pytest.mark.parametrize("Sq", [1, 130])
def test_key_weights_past_32_bits(osf, Sq):
    Hkv, S, n, D = 40, 500_000, 1024, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.zeros(1, Hkv, S, D, dtype=torch.bfloat16, device="cuda")
    assert k.numel() * 2 > 2 ** 32
    k[:, :, S - n:] = torch.randn(1, Hkv, n, D, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, Hkv, Sq, D, generator=g, device="cuda").to(torch.bfloat16)
    lse = torch.full((1, Hkv, Sq), 3.0, device="cuda")
    w = osf.osf_attn_key_weights(q, k, lse)
    small = osf.osf_attn_key_weights(q, k[:, :, S - n:].contiguous(), lse)
    assert torch.allclose(w[:, :, S - n:], small, rtol=512 * U, atol=0)   # the same terms, sums of 130 in another order
    assert bool(((w[:, :, :S - n] / (Sq * math.exp(-3)) - 1).abs() <= 1e-4).all())
    assert osf.osf_device_status() == osf.OSF_OK
