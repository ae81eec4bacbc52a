"""float32 rows of 64 channels under a window on the tensor cores: what some row sees of K and V is split into bfloat16 parts, and
nothing else of a long cache is read, kept or paid for.  Bounds: test_gpu_window's (2e-5 of size = sum P |V|; lse 2e-5).
"""
import numpy as np
import pytest

import oracle
import seeded_inputs as si
from conftest import f32_tensor
from test_gpu_window import check_out, guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# B, Hq, Hkv, Sq, Sk, window, sinks: many rows, few in key splits, sinks in one tile, in several, up to the window and into it, rows before
# the first key, hidden tiles in the middle, one or none
SHAPES = [
    (2, 20, 4, 520, 5000, 300, 0), (2, 20, 4, 520, 5000, 300, 5), (1, 16, 4, 600, 3333, 129, 260), (1, 16, 16, 600, 1500, 700, 190),
    (1, 16, 2, 700, 1600, 500, 399), (1, 16, 2, 700, 1600, 500, 450), (1, 24, 8, 900, 1000, 50, 1), (3, 8, 2, 700, 650, 100, 3),
    (1, 2, 1, 300, 9000, 4000, 7), (1, 2, 1, 1000, 9000, 1000, 130), (1, 1, 1, 40, 20000, 5000, 1), (1, 4, 2, 2, 9000, 4000, 0),
    (1, 24, 8, 513, 513 + 128, 1, 127), (1, 24, 8, 513, 513 + 256, 1, 129), (1, 40, 8, 256, 1024, 128, 128),
]


def bytes_of(osf, B, Hq, Hkv, Sq, Sk, window, sinks):
    return osf.osf_attn_window_workspace_bytes(osf.OSF_F32, B, Hq, Hkv, Sq, Sk, 64, window, sinks)


@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk,window,sinks", SHAPES)
def test_forward(osf, B, Hq, Hkv, Sq, Sk, window, sinks):
    """Against the oracle; the same bits, whatever stands where no row sees it; within the workspace."""
    q, k, v = si.qkv((B, Hq, Sq, 64), (B, Hkv, Sk, 64), seed=Sq, dtype="f32")
    Q, K, V = f32_tensor(q), f32_tensor(k), f32_tensor(v)
    lse = torch.empty(B, Hq, Sq, device="cuda")
    n = bytes_of(osf, B, Hq, Hkv, Sq, Sk, window, sinks)
    assert n >= 4 * (3 * Q.numel()) // 2   # Q's parts: the tensor-core path
    ws, behind = guarded(n)
    o = osf.osf_attn_fwd_gqa_window(Q, K, V, window, sinks, lse=lse, workspace=ws)
    assert (behind == 0xA5).all()
    check_out(o, lse, oracle.attention_window(q, k, v, window, sinks), "f32", f"{Sq},{Sk} {window},{sinks}")
    lo = max(0, Sk - Sq - window + 1)   # the first key of a window
    inside, outside = -(-sinks // 128) * 128, lo // 128 * 128
    K[:, :, sinks:lo] = float("nan")
    if inside < outside:   # whole tiles that nothing reads
        K[:, :, inside:outside], V[:, :, inside:outside] = float("inf"), float("nan")
    again, lse2 = torch.empty_like(o), torch.empty_like(lse)
    osf.osf_attn_fwd_gqa_window(Q, K, V, window, sinks, out=again, lse=lse2)
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    assert osf.osf_device_status() == osf.OSF_OK


def test_workspace_grows_with_the_window_alone(osf):
    for B, Hq, Hkv, Sq, Sk, window, sinks in SHAPES:
        if Sk > Sq + window + sinks + 256:   # the middle is hidden: 1000 more tiles of it
            a, b = (bytes_of(osf, B, Hq, Hkv, Sq, Sk + 128 * x, window, sinks) for x in (0, 1000))
            assert a == b, (Sq, Sk, window, sinks)


def test_strided_views(osf):
    """[B, S, H, D] tensors of Q, V and O, K shared by the batch (stride 0), a long cache's last keys as a view."""
    B, Hq, Hkv, Sq, Sk, window, sinks = 2, 20, 4, 520, 3000, 300, 140
    q, k, v = si.qkv((B, Hq, Sq, 64), (B, Hkv, Sk, 64), seed=3, dtype="f32")
    k[1] = k[0]
    Q = f32_tensor(q).transpose(1, 2).contiguous().transpose(1, 2)
    K = f32_tensor(k[:1]).expand(B, -1, -1, -1)
    V = torch.zeros(B, Sk + 100, Hkv, 64, device="cuda")[:, :Sk].transpose(1, 2)
    V.copy_(f32_tensor(v))
    out = torch.zeros(B, Sq, Hq, 64, device="cuda").transpose(1, 2)
    lse = torch.empty(B, Hq, Sq, device="cuda")
    osf.osf_attn_fwd_gqa_window(Q, K, V, window, sinks, out=out, lse=lse)
    check_out(out, lse, oracle.attention_window(q, k, v, window, sinks), "f32", "strided")
    plain = osf.osf_attn_fwd_gqa_window(Q.contiguous(), K.contiguous(), V.contiguous(), window, sinks)
    assert torch.equal(out, plain)


def test_captured_in_a_graph(osf):
    B, Hq, Hkv, Sq, Sk, window, sinks = 1, 16, 4, 600, 3000, 129, 260
    q, k, v = (torch.randn(B, h, s, 64, device="cuda") for h, s in ((Hq, Sq), (Hkv, Sk), (Hkv, Sk)))
    ws = torch.empty(bytes_of(osf, B, Hq, Hkv, Sq, Sk, window, sinks), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(q)
    osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks, out=o, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks, out=o, workspace=ws)
    for x in (q, k, v):
        x.copy_(torch.randn_like(x))
    graph.replay()
    assert torch.equal(o, osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks))
