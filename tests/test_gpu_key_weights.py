"""osf_attn_key_weights against the fp64 column sums of the softmax matrix.

Tolerance, u = 2^-24: a score is a float32 sum of D exact (bfloat16) or once-rounded (float32)
products, off by at most ds = 2 (D + 8) u scale max sum |q| |k| (the factor 2 allows the tensor core to
truncate); a term is off by a factor 1 + ds + 4 u (|lse| + |score| + 8) + 2^-20 (exponent and 2^x), and
float32 sums of non-negative terms by (terms in the longest chain) u, at most rows u.
"""
import numpy as np
import pytest

import oracle
import seeded_inputs as si
from conftest import bf16_tensor, f32_tensor

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


def qk(B, Hq, Hkv, Sq, Sk, D, dtype, seed):
    q, k, _ = si.qkv((B, Hq, Sq, D), (B, Hkv, Sk, D), seed=seed, dtype="bf16" if dtype == "bf16" else "f32")
    if dtype == "bf16":
        return bf16_tensor(q), bf16_tensor(k)
    return f32_tensor(q), f32_tensor(k)


def check(osf, q, k, mask, scale=None, lse=None):
    qv, kv = q.double().cpu().numpy(), k.double().cpu().numpy()
    B, Hq, Sq, D = qv.shape
    Hkv, Sk = kv.shape[1], kv.shape[2]
    if lse is None:
        _, lse64 = oracle.attention_gqa(qv, kv, kv, mask=mask, scale=scale)
        lse = f32_tensor(lse64)
    lv = lse.double().cpu().numpy()
    want = oracle.key_weights(qv, kv, lv, mask, scale)
    got = osf.osf_attn_key_weights(q, k, lse, mask=mask, scale=scale)
    sc = D ** -0.5 if scale is None else scale
    G = Hq // Hkv
    top = max((np.abs(qv[b, h]) @ np.abs(kv[b, h // G]).T).max() for b in range(B) for h in range(Hq)) * sc
    big = np.abs(lv[np.isfinite(lv)]).max() if np.isfinite(lv).any() else 0.0
    rel = 2 * (D + 8) * U * top + 4 * U * (big + top + 8) + 2.0 ** -20 + min(G * Sq, 4096) * U
    g = got.double().cpu().numpy()
    assert np.all(np.isfinite(g))
    excess = np.max(np.abs(g - want) - want * rel - 1e-30)
    assert excess <= 0, f"off by {excess:.3e} past the tolerance ({rel:.2e} relative)"
    base = torch.rand(B, Hkv, Sk, device="cuda")
    acc = osf.osf_attn_key_weights(q, k, lse, weights=base.clone(), mask=mask, scale=scale, accumulate=True)
    assert torch.equal(acc, base + got)
    assert osf.osf_device_status() == osf.OSF_OK
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mask", ["none", "top_left", "bottom_right"])
@pytest.mark.parametrize("Sq,Sk", [(1, 1), (1, 300), (7, 7), (128, 128), (129, 257), (300, 77), (33, 500), (500, 500)])
def test_masks_and_lengths(osf, dtype, mask, Sq, Sk):
    for D in (64, 128):
        q, k = qk(2, 4, 2, Sq, Sk, D, dtype, Sq + Sk + D)
        check(osf, q, k, mask)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 8, 31, 32, 80, 96, 160, 256])
def test_head_dims(osf, dtype, D):
    q, k = qk(1, 6, 3, 45, 70, D, dtype, D)
    check(osf, q, k, "bottom_right")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(1, 1, 1), (8, 1, 1), (9, 1, 1), (16, 1, 1), (4, 1, 4), (5, 1, 3), (17, 1, 1), (12, 4, 5), (32, 2, 2)])
def test_few_rows(osf, D, Hq, Hkv, Sq):
    for Sk in (Sq, 16, 100, 1111):
        if Sk >= Sq:
            q, k = qk(2, Hq, Hkv, Sq, Sk, D, "bf16", Hq + Sq + Sk)
            check(osf, q, k, "bottom_right")


@pytest.mark.parametrize("D", [32, 96])
@pytest.mark.parametrize("Hq,Hkv,Sq", [(1, 1, 1), (8, 1, 1), (6, 3, 4), (16, 2, 2), (10, 2, 2)])
def test_few_rows_of_other_head_dims(osf, D, Hq, Hkv, Sq):
    for Sk in (Sq, 17, 1111):
        q, k = qk(2, Hq, Hkv, Sq, Sk, D, "bf16", Hq + Sq + Sk)
        check(osf, q, k, "bottom_right")
        check(osf, q, k, "none")


@pytest.mark.parametrize("D", [64, 128])
def test_longer_prompts(osf, D):
    q, k = qk(1, 4, 2, 1100, 1100, D, "bf16", 3)
    check(osf, q, k, "top_left")
    q, k = qk(1, 2, 2, 600, 1700, D, "bf16", 4)
    check(osf, q, k, "bottom_right", scale=0.3)
    q, k = qk(1, 2, 1, 900, 200, D, "bf16", 5)     # most rows see nothing
    check(osf, q, k, "bottom_right")


def test_with_the_forward_calls_own_lse(osf):
    """The weights of each kv head sum to its rows."""
    B, Hq, Hkv, S, D = 2, 8, 2, 700, 128
    q, k = qk(B, Hq, Hkv, S, S, D, "bf16", 6)
    lse = torch.empty(B, Hq, S, device="cuda")
    osf.osf_attn_fwd_gqa_ex(q, k, k, mask="top_left", lse=lse)
    w = osf.osf_attn_key_weights(q, k, lse, mask="top_left")
    rows = Hq // Hkv * S
    assert torch.allclose(w.double().sum(-1), torch.full((B, Hkv), float(rows), dtype=torch.float64, device="cuda"), rtol=1e-4)
    check(osf, q, k, "top_left", lse=lse)


def test_rows_that_see_nothing_or_have_no_lse(osf):
    q, k = qk(1, 4, 2, 40, 64, 64, "bf16", 7)
    lse = torch.randn(1, 4, 40, device="cuda") + 5
    lse[0, :, 3:9] = float("-inf")
    check(osf, q, k, "none", lse=lse)
    lse.fill_(float("-inf"))
    assert bool((osf.osf_attn_key_weights(q, k, lse) == 0).all())


@pytest.mark.parametrize("dtype,Sq", [("bf16", 1), ("bf16", 4), ("bf16", 300), ("f32", 4), ("f32", 300)])
def test_rows_without_an_lse_may_hold_anything(osf, dtype, Sq):
    """Padding rows: lse = -inf, and NaN or infinite queries."""
    for mask in ("none", "bottom_right"):
        q, k = qk(1, 4, 2, Sq, 500, 64, dtype, 17)
        lse = torch.full((1, 4, Sq), 7.0, device="cuda")
        lse[0, 1] = float("-inf")
        lse[0, 2:, Sq // 2 + 1:] = float("-inf")
        clean = osf.osf_attn_key_weights(q, k, lse, mask=mask)
        check(osf, q, k, mask, lse=lse)
        q[0, 1, 0] = float("nan")
        q[0, 2:, Sq // 2 + 1:] = float("inf")
        assert torch.equal(osf.osf_attn_key_weights(q, k, lse, mask=mask), clean)


def test_strides(osf):
    B, Hq, Hkv, Sq, Sk, D = 2, 4, 2, 150, 260, 128
    x = bf16_tensor(si.qkv((B, Sq, Hq, D + 8), (B, Sk, Hkv, D + 8), seed=8, dtype="bf16")[0])
    y = bf16_tensor(si.qkv((B, Sq, Hq, D + 8), (B, Sk, Hkv, D + 8), seed=8, dtype="bf16")[1])
    lse = torch.full((B, Hq, Sq), 6.0, device="cuda")
    for a in (0, 1, 8):   # aligned, at an odd element, a shifted start
        q, k = x[..., a:a + D].transpose(1, 2), y[..., a:a + D].transpose(1, 2)
        got = osf.osf_attn_key_weights(q, k, lse, mask="bottom_right")
        check(osf, q, k, "bottom_right", lse=lse)
        ref = osf.osf_attn_key_weights(q.contiguous(), k.contiguous(), lse, mask="bottom_right")
        assert torch.allclose(got, ref, rtol=1e-4, atol=1e-7)
    few = x[:, :2, :, :D].transpose(1, 2)   # two rows: the path of a decode step
    for a in (0, 1, 8):
        check(osf, few, y[..., a:a + D].transpose(1, 2), "bottom_right", lse=lse[:, :, :2].contiguous())
    one = y[:1, ..., :D].transpose(1, 2).expand(B, -1, -1, -1)   # a broadcast batch
    check(osf, x[..., :D].transpose(1, 2), one, "none", lse=lse)


def test_large_and_infinite_values(osf):
    q, k = qk(1, 2, 1, 64, 128, 64, "bf16", 9)
    q[0, 0] *= 30
    check(osf, q, k, "none")
    k[0, 0, 100] = float("nan")            # a key that the mask hides from the rows before it
    lse = torch.full((1, 2, 64), 5.0, device="cuda")
    w = osf.osf_attn_key_weights(q, k, lse, mask="top_left")
    # the scores of the enlarged head pass 5 + ln(float32's largest) = 93.7: those weights are infinite
    want = oracle.key_weights(*(x.double().cpu().numpy() for x in (q, k[:, :, :64], lse)), mask="top_left")[0, 0]
    got = w[0, 0, :64].double().cpu().numpy()
    far = np.finfo(np.float32).max
    assert bool((w[0, 0, 64:] == 0).all()) and not np.any(np.isnan(got))
    assert np.all(got[want > 1.01 * far] == np.inf) and np.all(got[want < 0.99 * far] < np.inf)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 40), ("bf16", 96)])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk", [(1, 3, 1, 700, 700), (1, 2, 2, 65, 3000), (2, 4, 1, 900, 130), (1, 1, 1, 2500, 64), (1, 5, 1, 3, 2000)])
def test_cuda_core_path_row_parts(osf, dtype, D, B, Hq, Hkv, Sq, Sk):
    """Rows in several parts, key blocks that few or no rows see, tiles that cross heads."""
    for mask in ("none", "top_left", "bottom_right"):
        q, k = qk(B, Hq, Hkv, Sq, Sk, D, dtype, Sq + Sk)
        n = osf.osf_attn_key_weights_workspace_bytes(osf.OSF_F32 if dtype == "f32" else osf.OSF_BF16, B, Hq, Hkv, Sq, Sk, D)
        assert n == osf.osf_attn_key_weights_workspace_bytes(osf.OSF_F32 if dtype == "f32" else osf.OSF_BF16, B, Hq, Hkv, Sq, Sk, D)
        check(osf, q, k, mask)


def test_no_rows(osf):
    q, k = torch.empty(1, 2, 0, 64, device="cuda"), torch.randn(1, 2, 9, 64, device="cuda")
    w = torch.ones(1, 2, 9, device="cuda")
    osf.osf_attn_key_weights(q, k, torch.empty(1, 2, 0, device="cuda"), weights=w, accumulate=True)
    assert bool((w == 1).all())
    osf.osf_attn_key_weights(q, k, torch.empty(1, 2, 0, device="cuda"), weights=w)
    assert bool((w == 0).all())


def test_workspace_too_small_is_refused(osf):
    q, k = qk(1, 4, 1, 2048, 128, 64, "f32", 10)
    n = osf.osf_attn_key_weights_workspace_bytes(osf.OSF_F32, 1, 4, 1, 2048, 128, 64)
    assert n > 0
    with pytest.raises(osf.OsfError) as err:
        osf.osf_attn_key_weights(q, k, torch.zeros(1, 4, 2048, device="cuda"), workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert err.value.status == osf.OSF_ERR_WORKSPACE
