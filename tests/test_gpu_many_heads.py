"""Calls with more (batch, head) pairs than a grid's second dimension holds (65535): large batches of single tokens.

Bounds: test_gpu_window's (float32 2e-5 of sum P |V|; bfloat16 2^-8 of that and of |O|).
"""
import pytest

import oracle
from test_gpu_window import check_grads, check_out

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HEADS = [(2200, 32, 8), (70000, 1, 1), (1, 72000, 9000), (1, 70001, 1)]   # B, Hq, Hkv


def tensors(shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16 if dtype == "bf16" else torch.float32)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 64), ("bf16", 72), ("bf16", 64)])
@pytest.mark.parametrize("B,Hq,Hkv", HEADS)
def test_windowed_forward(osf, dtype, D, B, Hq, Hkv):
    for Sq in (1, 3):
        q, k, v = (tensors((B, h, s, D), dtype, i) for i, (h, s) in enumerate(((Hq, Sq), (Hkv, 20), (Hkv, 20))))
        lse = torch.empty(B, Hq, Sq, device="cuda")
        o = osf.osf_attn_fwd_gqa_window(q, k, v, 5, 2, lse=lse)
        some = torch.tensor(sorted({0, B // 2, B - 1}), device="cuda")
        ref = oracle.attention_window(*(x[some].double().cpu().numpy() for x in (q, k, v)), 5, 2)
        check_out(o[some], lse[some], ref, dtype, f"{B} x {Hq}, {Sq} rows")


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("bf16", 72)])
@pytest.mark.parametrize("B,Hq,Hkv", HEADS)
def test_plain_forward(osf, dtype, D, B, Hq, Hkv):
    q, k, v = (tensors((B, h, s, D), dtype, i) for i, (h, s) in enumerate(((Hq, 2), (Hkv, 20), (Hkv, 20))))
    lse = torch.empty(B, Hq, 2, device="cuda")
    o = osf.osf_attn_fwd_gqa_ex(q, k, v, mask="bottom_right", lse=lse)
    some = torch.tensor(sorted({0, B // 2, B - 1}), device="cuda")
    ref = oracle.attention_window(*(x[some].double().cpu().numpy() for x in (q, k, v)), 20, 0)
    check_out(o[some], lse[some], ref, dtype, f"{B} x {Hq}")


def test_an_explicit_split_count(osf):
    """osf_attn_decode_gqa on the CUDA cores: a count of key splits there is no room for is not taken."""
    B, Hq, Hkv = HEADS[0]
    q, k, v = (tensors((B, h, s, 32), "f32", i) for i, (h, s) in enumerate(((Hq, 1), (Hkv, 200), (Hkv, 200))))
    ref = osf.osf_attn_fwd_gqa(q, k, v)
    assert torch.equal(osf.osf_attn_decode_gqa(q, k, v, num_splits=3), ref)


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 160), ("bf16", 64), ("bf16", 40)])
def test_windowed_gradients(osf, dtype, D):
    B, H, S, window, sinks = 70000, 1, 6, 3, 1
    q, k, v, g = (tensors((B, H, S, D), dtype, i) for i in range(4))
    lse = torch.empty(B, H, S, device="cuda")
    o = osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks, lse=lse)
    grads = osf.osf_attn_bwd_gqa_window(q, k, v, o, g, lse, window, sinks)
    some = torch.tensor([0, B // 2, B - 1], device="cuda")
    q, k, v, g = (x[some].double().cpu().numpy() for x in (q, k, v, g))
    check_grads([x[some] for x in grads], oracle.attention_window(q, k, v, window, sinks, dO=g), dtype, "gradients")
    assert osf.osf_device_status() == osf.OSF_OK
