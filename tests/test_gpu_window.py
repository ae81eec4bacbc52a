"""Sliding-window attention with sinks (osf_attn_fwd_gqa_window, osf_attn_bwd_gqa_window) against
oracle.attention_window, in 64 bits.

Tolerances, from what is rounded.  bf16 forward: P to bfloat16 before the product with V (2^-8 of each term, so 2^-8
of size = sum P |V|) and O once (2^-8 |O|); scores, sums and exponentials are float32 (2^-24 a step, far below): a
sixteenth of slack covers those.  float32 forward on the CUDA cores: a score is a sum of D products, |err| <= D 2^-24
sum |q k| scale, and moves P by that much, relatively; with the inputs here that is below 2e-5 of size.  With D = 64 on the
tensor cores P and V have 17 bits: 2^-17 each, within the same 2e-5.  lse: float32 scores, 2e-5 absolute and relative.
Gradients: P, dS and O (in the row sums D) are rounded once each to the inputs' type, 2^-8 in bfloat16, and the result
once more; the float32 sums dP and D, the scores and the log-sum-exp add 2^-16 of the terms (a score's error, D 2^-24 sum |q k|
scale, moves P by that much).  oracle.attention_window gives what those are relative to.  float32: 2e-5 of both.
"""
import numpy as np
import pytest

import oracle
import seeded_inputs as si
from conftest import bf16_tensor, f32_tensor
from test_gpu_attention_bwd import f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def check_out(o, lse, ref, dtype, what):
    O, L, size = ref[:3]
    got = o.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    if dtype == "bf16":
        bound = (1 + 1 / 16) * 2.0 ** -8 * (size + np.abs(O)) + 1e-30
    else:
        bound = 2e-5 * size + 1e-30
    bad = np.abs(got - O) > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - O).max():.3g}"
    gl = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(gl), np.isneginf(L)), what
    live = ~np.isneginf(L)
    assert np.all(np.abs(gl[live] - L[live]) <= 2e-5 * (1 + np.abs(L[live]))), what


def check_grads(grads, ref, dtype, what):
    for name, got, r, (near, far) in zip(("dq", "dk", "dv"), grads, ref[3:6], ref[6]):
        u, w = (2.0 ** -8, 2.0 ** -16) if dtype == "bf16" else (2e-5, 2e-5)
        bound = (1 + 1 / 16) * (u * (near + np.abs(r)) + w * far) + 1e-30
        err = np.abs(got.double().cpu().numpy() - r)
        assert np.isfinite(err).all() and not (err > bound).any(), \
            f"{what} {name}: {(err > bound).sum()} of {err.size} off, worst {err.max():.3g}, {(err / bound).max():.3g} of the bound"


def run(osf, dtype, B, Hq, Hkv, Sq, Sk, D, window, sinks, grad=False, store_ds=True, seed=0):
    what = f"{dtype} {B},{Hq},{Hkv},{Sq},{Sk},{D} window={window} sinks={sinks}"
    q, k, v = si.qkv((B, Hq, Sq, D), (B, Hkv, Sk, D), seed=seed, dtype=dtype)
    g = si.qkv((B, Hq, Sq, D), (1, 1, 1, D), seed=seed + 1000, dtype=dtype)[0] if grad else None
    dev = bf16_tensor if dtype == "bf16" else f32_tensor
    Q, K, V = dev(q), dev(k), dev(v)
    lse = torch.full((B, Hq, Sq), float("nan"), device="cuda")
    o = osf.osf_attn_fwd_gqa_window(Q, K, V, window, sinks, lse=lse)
    ref = oracle.attention_window(f64(q, dtype), f64(k, dtype), f64(v, dtype), window, sinks,
                                  dO=f64(g, dtype) if grad else None)
    check_out(o, lse, ref, dtype, what)
    if grad:
        G, ws = dev(g), None
        if not store_ds:   # all but the dS^T tiles
            code = osf.OSF_F32 if dtype == "f32" else osf.OSF_BF16
            n = osf.osf_attn_bwd_window_workspace_bytes(code, B, Hq, Hkv, Sq, Sk, D, window, sinks)
            tiles = -(-Sq // 128) * min(-(-Sk // 128), -(-sinks // 128) + (window + 253) // 128 + 1)
            assert n > 32768 * B * Hq * tiles, "a problem that stores dS"
            ws = torch.empty(n - 32768 * B * Hq * tiles, dtype=torch.uint8, device="cuda")
        grads = osf.osf_attn_bwd_gqa_window(Q, K, V, o, G, lse, window, sinks, workspace=ws)
        check_grads(grads, ref, dtype, f"{what} store_ds={store_ds}")
    assert osf.osf_device_status() == osf.OSF_OK


# windows around the tile sizes (64, 128), sinks inside a tile, over several, and into the window; rows that see nothing
SHAPES = [
    (1, 1, 1, 1, 1, 1, 0), (1, 2, 1, 1, 300, 1, 0), (1, 2, 1, 1, 300, 1, 1), (2, 4, 2, 1, 1000, 64, 4), (1, 4, 1, 3, 700, 100, 5),
    (1, 2, 1, 2, 130, 63, 66), (1, 2, 1, 5, 3, 2, 1), (1, 2, 1, 40, 17, 3, 0),
    (1, 2, 1, 200, 200, 1, 0), (1, 2, 1, 200, 200, 127, 0), (1, 2, 1, 257, 257, 128, 1), (1, 2, 1, 300, 300, 129, 130),
    (1, 2, 2, 384, 512, 65, 0), (2, 3, 1, 333, 999, 200, 17), (1, 2, 1, 520, 520, 255, 250), (1, 1, 1, 700, 650, 100, 3),
    (1, 2, 1, 129, 1290, 300, 129), (1, 8, 2, 256, 640, 384, 0),
]


@pytest.mark.parametrize("dtype,D", [("bf16", 32), ("bf16", 64), ("bf16", 96), ("bf16", 128), ("bf16", 72), ("f32", 64), ("f32", 40), ("f32", 256)])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk,window,sinks", SHAPES)
def test_forward(osf, dtype, D, B, Hq, Hkv, Sq, Sk, window, sinks):
    run(osf, dtype, B, Hq, Hkv, Sq, Sk, D, window, sinks)


@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk,window,sinks", [
    (2, 20, 4, 520, 700, 129, 130), (1, 32, 8, 700, 700, 64, 300), (3, 16, 16, 500, 1300, 200, 17), (1, 24, 8, 1000, 1000, 127, 0),
    (2, 16, 2, 640, 640, 255, 1)])
def test_forward_of_many_float32_rows(osf, B, Hq, Hkv, Sq, Sk, window, sinks):
    """Enough rows for the tensor cores (D = 64, bfloat16 parts)."""
    run(osf, "f32", B, Hq, Hkv, Sq, Sk, 64, window, sinks)


@pytest.mark.parametrize("dtype,D", [("bf16", 32), ("bf16", 64), ("bf16", 96), ("bf16", 128), ("bf16", 72), ("f32", 64), ("f32", 100), ("f32", 250)])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk,window,sinks", SHAPES)
def test_gradients(osf, dtype, D, B, Hq, Hkv, Sq, Sk, window, sinks):
    run(osf, dtype, B, Hq, Hkv, Sq, Sk, D, window, sinks, grad=True)


# heads enough for dS to be stored, with sink tiles that are shared out and not
WIDE = [(3, 80, 20, 520, 520, 130, 3), (2, 96, 96, 300, 700, 1, 130), (1, 160, 80, 390, 390, 200, 0), (5, 64, 32, 140, 260, 64, 17)]


@pytest.mark.parametrize("store_ds", [True, False])
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk,window,sinks", WIDE)
def test_gradients_of_many_heads(osf, D, B, Hq, Hkv, Sq, Sk, window, sinks, store_ds):
    run(osf, "bf16", B, Hq, Hkv, Sq, Sk, D, window, sinks, grad=True, store_ds=store_ds)


@pytest.mark.parametrize("D", [64, 96, 128])
def test_many_items(osf, D):
    """More query blocks than SMs, so that a CTA goes from one to the next."""
    run(osf, "bf16", 5, 8, 4, 1100, 1100, D, 190, 3, grad=True)


def test_a_window_that_hides_nothing_is_the_causal_call(osf):
    q, k, v = (bf16_tensor(x) for x in si.qkv((1, 4, 200, 64), (1, 2, 300, 64), seed=3, dtype="bf16"))
    lse, ref_lse = torch.empty(1, 4, 200, device="cuda"), torch.empty(1, 4, 200, device="cuda")
    ref = osf.osf_attn_fwd_gqa_ex(q, k, v, mask="bottom_right", lse=ref_lse)
    exact = oracle.attention_window(*(x.double().cpu().numpy() for x in (q, k, v)), 300, dO=q.double().cpu().numpy())
    for window, sinks in ((300, 0), (2 ** 31 - 1, 0), (100, 200), (1, 2 ** 31 - 1)):
        o = osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks, lse=lse)
        assert torch.equal(o, ref) and torch.equal(lse, ref_lse)
        grads = osf.osf_attn_bwd_gqa_window(q, k, v, o, q, lse, window, sinks)
        check_grads(grads, exact, "bf16", f"{window} {sinks}")


def test_strided_views(osf):
    """[B, S, H, D] tensors, and K, V shared by the batch (stride 0)."""
    B, Hq, Hkv, Sq, Sk, D, window, sinks = 2, 4, 2, 150, 400, 64, 77, 6
    for dtype, dev in (("bf16", bf16_tensor), ("f32", f32_tensor)):
        q, k, v = si.qkv((B, Hq, Sq, D), (1, Hkv, Sk, D), seed=7, dtype=dtype)
        Q = dev(q).transpose(1, 2).contiguous().transpose(1, 2)
        K, V = dev(k).expand(B, -1, -1, -1), dev(v).transpose(1, 2).contiguous().transpose(1, 2).expand(B, -1, -1, -1)
        out = torch.zeros(B, Sq, Hq, D, dtype=Q.dtype, device="cuda").transpose(1, 2)
        lse = torch.empty(B, Hq, Sq, device="cuda")
        for rows in (Sq, 2):
            o = out[:, :, :rows]
            osf.osf_attn_fwd_gqa_window(Q[:, :, :rows], K, V, window, sinks, out=o, lse=lse[:, :, :rows].contiguous())
            l2 = torch.empty(B, Hq, rows, device="cuda")
            osf.osf_attn_fwd_gqa_window(Q[:, :, :rows], K, V, window, sinks, out=o, lse=l2)
            ref = oracle.attention_window(f64(q, dtype)[:, :, :rows], np.repeat(f64(k, dtype), B, 0),
                                          np.repeat(f64(v, dtype), B, 0), window, sinks)
            check_out(o, l2, ref, dtype, f"strided {dtype} {rows}")


def test_hidden_keys_do_not_matter(osf):
    """NaN and infinities in keys and values that no row sees, inside and outside the tiles that are read."""
    Sk, window, sinks = 900, 200, 5
    for dtype, dev, D in (("bf16", bf16_tensor, 64), ("bf16", bf16_tensor, 128), ("f32", f32_tensor, 64), ("f32", f32_tensor, 32)):
        for Sq in (1, 3, 150):
            q, k, v = (dev(x) for x in si.qkv((1, 2, Sq, D), (1, 1, Sk, D), seed=9, dtype=dtype))
            lo = Sk - Sq - window + 1
            ref = osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks)
            # outside every tile that is read: whatever is there
            k[:, :, 128:lo // 128 * 128] = float("nan")
            v[:, :, 128:lo // 128 * 128] = float("inf")
            # inside one: hidden keys may be anything
            k[:, :, sinks:128] = float("nan")
            k[:, :, lo // 128 * 128:lo] = float("inf")
            assert torch.equal(osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks), ref), (dtype, D, Sq)


def test_no_keys(osf):
    q = torch.randn(2, 4, 3, 64, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        k = torch.empty(2, 2, 0, 64, dtype=dt, device="cuda")
        lse = torch.zeros(2, 4, 3, device="cuda")
        o = osf.osf_attn_fwd_gqa_window(q.to(dt), k, k, 5, 1, out=torch.ones_like(q, dtype=dt), lse=lse)
        assert not o.any() and torch.isneginf(lse).all()
        dq, dk, dv = osf.osf_attn_bwd_gqa_window(q.to(dt), k, k, o, o, lse, 5, 1, dq=torch.ones_like(o))
        assert not dq.any() and dk.numel() == dv.numel() == 0
        e = torch.empty(2, 4, 0, 64, dtype=dt, device="cuda")
        kk = torch.ones(2, 2, 7, 64, dtype=dt, device="cuda")
        _, dk, dv = osf.osf_attn_bwd_gqa_window(e, kk, kk, e, e, lse[:, :, :0].contiguous(), 5, 1, dk=kk + 1, dv=kk + 1)
        assert not dk.any() and not dv.any()


def test_against_differences(osf):
    """float32 gradients against central differences of the forward pass in 64 bits."""
    rng = np.random.default_rng(5)
    B, Hq, Hkv, Sq, Sk, D, window, sinks = 1, 2, 1, 9, 13, 8, 4, 2
    q, k, v, g = (rng.standard_normal(s) for s in ((B, Hq, Sq, D), (B, Hkv, Sk, D), (B, Hkv, Sk, D), (B, Hq, Sq, D)))
    Q, K, V, G = (f32_tensor(x) for x in (q, k, v, g))
    lse = torch.empty(B, Hq, Sq, device="cuda")
    o = osf.osf_attn_fwd_gqa_window(Q, K, V, window, sinks, lse=lse)
    grads = osf.osf_attn_bwd_gqa_window(Q, K, V, o, G, lse, window, sinks)
    loss = lambda: (oracle.attention_window(q, k, v, window, sinks)[0] * g).sum()  # noqa: E731
    for x, d in zip((q, k, v), grads):
        for i in rng.choice(x.size, 12, replace=False):
            at = np.unravel_index(i, x.shape)
            old, h = x[at], 1e-5
            x[at] = old + h
            up = loss()
            x[at] = old - h
            down = loss()
            x[at] = old
            # differences: h^2 and 1e-15 / h; the float32 pass 1e-5
            assert abs((up - down) / (2 * h) - d[at].item()) <= 1e-4, at


def test_same_bits_every_time(osf):
    q, k, v, g = (torch.randn(1, h, 2000, 64, device="cuda").bfloat16() for h in (8, 2, 2, 8))
    lse = torch.empty(1, 8, 2000, device="cuda")
    o = osf.osf_attn_fwd_gqa_window(q, k, v, 300, 9, lse=lse)
    first = osf.osf_attn_bwd_gqa_window(q, k, v, o, g, lse, 300, 9)
    for _ in range(3):
        again = osf.osf_attn_bwd_gqa_window(q, k, v, osf.osf_attn_fwd_gqa_window(q, k, v, 300, 9), g, lse, 300, 9)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_captured_training_step(osf):
    """Forward and backward in one graph, on a stream of its own, replayed with other inputs."""
    S, D, window, sinks = 500, 64, 130, 4
    q, k, v, g = (torch.randn(1, h, S, D, device="cuda").bfloat16() for h in (4, 2, 2, 4))
    lse, o = torch.empty(1, 4, S, device="cuda"), torch.empty_like(q)
    grads = [torch.empty_like(x) for x in (q, k, v)]
    ws = torch.empty(osf.osf_attn_window_workspace_bytes(osf.OSF_BF16, 1, 4, 2, S, S, D, window, sinks) + 1, dtype=torch.uint8,
                     device="cuda")
    wb = torch.empty(osf.osf_attn_bwd_window_workspace_bytes(osf.OSF_BF16, 1, 4, 2, S, S, D, window, sinks),
                     dtype=torch.uint8, device="cuda")

    def step():
        osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks, out=o, lse=lse, workspace=ws)
        osf.osf_attn_bwd_gqa_window(q, k, v, o, g, lse, window, sinks, *grads, workspace=wb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (q, k, v, g):
        x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (o, lse, *grads)]
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, (o, lse, *grads)))


def guarded(n):
    """A workspace of exactly n bytes, and the bytes behind it."""
    whole = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    return whole[:n], whole[n:]


@pytest.mark.parametrize("dtype,B,Hq,Hkv,Sq,Sk,D,window,sinks", [
    ("bf16", 1, 8, 2, 1, 9000, 128, 4096, 4), ("bf16", 1, 8, 2, 2, 5000, 96, 3000, 0), ("f32", 1, 4, 2, 3, 4000, 64, 3000, 9),
    ("f32", 1, 2, 1, 40, 4000, 100, 3000, 9), ("bf16", 1, 4, 2, 100, 8000, 64, 5000, 4), ("bf16", 1, 2, 1, 17, 8000, 72, 5000, 4)])
def test_forward_stays_in_its_workspace(osf, dtype, B, Hq, Hkv, Sq, Sk, D, window, sinks):
    dev, code = (bf16_tensor, osf.OSF_BF16) if dtype == "bf16" else (f32_tensor, osf.OSF_F32)
    q, k, v = (dev(x) for x in si.qkv((B, Hq, Sq, D), (B, Hkv, Sk, D), seed=1, dtype=dtype))
    n = osf.osf_attn_window_workspace_bytes(code, B, Hq, Hkv, Sq, Sk, D, window, sinks)
    assert n > 0
    ws, behind = guarded(n)
    ref = osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks)
    assert torch.equal(osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks, workspace=ws), ref)
    assert (behind == 0xA5).all()
    for part, status in ((ws[:16], osf.OSF_ERR_WORKSPACE), (guarded(n + 8)[0][8:], osf.OSF_ERR_INVALID)):
        with pytest.raises(osf.OsfError) as e:
            osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks, workspace=part)
        assert e.value.status == status


@pytest.mark.parametrize("dtype,B,Hq,Hkv,Sq,Sk,D,window,sinks", [
    ("bf16", 1, 4, 2, 1000, 1000, 64, 300, 4), ("bf16", 1, 8, 2, 700, 900, 96, 200, 0), ("bf16", 4, 32, 8, 1024, 1024, 128, 200, 5),
    ("bf16", 2, 32, 8, 1500, 1500, 64, 100, 0), ("f32", 1, 4, 2, 301, 301, 64, 65, 3), ("bf16", 2, 32, 8, 1000, 1000, 64, 2000, 0)])
def test_backward_stays_in_its_workspace(osf, dtype, B, Hq, Hkv, Sq, Sk, D, window, sinks):
    dev, code = (bf16_tensor, osf.OSF_BF16) if dtype == "bf16" else (f32_tensor, osf.OSF_F32)
    q, k, v = (dev(x) for x in si.qkv((B, Hq, Sq, D), (B, Hkv, Sk, D), seed=1, dtype=dtype))
    g = dev(si.qkv((B, Hq, Sq, D), (1, 1, 1, D), seed=2, dtype=dtype)[0])
    lse = torch.empty(B, Hq, Sq, device="cuda")
    o = osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks, lse=lse)
    n = osf.osf_attn_bwd_window_workspace_bytes(code, B, Hq, Hkv, Sq, Sk, D, window, sinks)
    ws, behind = guarded(n)
    ref = osf.osf_attn_bwd_gqa_window(q, k, v, o, g, lse, window, sinks)
    got = osf.osf_attn_bwd_gqa_window(q, k, v, o, g, lse, window, sinks, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and (behind == 0xA5).all()
    with pytest.raises(osf.OsfError) as e:
        osf.osf_attn_bwd_gqa_window(q, k, v, o, g, lse, window, sinks, workspace=ws[:64])
    assert e.value.status == osf.OSF_ERR_WORKSPACE
    if dtype == "bf16" and window < Sk:
        with pytest.raises(osf.OsfError) as e:
            osf.osf_attn_bwd_gqa_window(q, k, v, o, g, lse, window, sinks, workspace=guarded(n + 64)[0][64:])
        assert e.value.status == osf.OSF_ERR_INVALID


def test_two_streams_train_at_once(osf):
    """Forward and backward on two streams, each with its own workspaces, give what they give alone."""
    S, D, window, sinks = 1200, 128, 200, 4
    sets = [[torch.randn(1, h, S, D, device="cuda").bfloat16() for h in (8, 2, 2, 8)] for _ in range(2)]

    def step(q, k, v, g):
        lse = torch.empty(1, 8, S, device="cuda")
        o = osf.osf_attn_fwd_gqa_window(q, k, v, window, sinks, lse=lse)
        return (o, lse, *osf.osf_attn_bwd_gqa_window(q, k, v, o, g, lse, window, sinks))
    alone = [step(*x) for x in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for got in outs[i]:
            assert all(torch.equal(a, b) for a, b in zip(got, alone[i]))
    assert osf.osf_device_status() == osf.OSF_OK


def test_shared_keys_across_the_batch(osf):
    """K and V expanded over heads and batch (strides of 0, another kernel than their copies') give what their copies do, each
    within the bounds."""
    q, k, v = si.qkv((3, 4, 50, 64), (1, 1, 400, 64), seed=3, dtype="bf16")
    Q, K, V = (bf16_tensor(x) for x in (q, k, v))
    wide = [x.expand(3, 2, 400, 64) for x in (K, V)]
    for n in (50, 1):
        ref = oracle.attention_window(f64(q, "bf16")[:, :, :n], *(np.tile(f64(x, "bf16"), (3, 2, 1, 1)) for x in (k, v)), 100, 3)
        for kv in (wide, [x.contiguous() for x in wide]):
            lse = torch.empty(3, 4, n, device="cuda")
            o = osf.osf_attn_fwd_gqa_window(Q[:, :, :n], *kv, 100, 3, lse=lse)
            check_out(o, lse, ref, "bf16", f"{n} rows")


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv,S,window,sinks", [
    ("f32", 64, 3, 20, 10, 390, 70, 3), ("f32", 40, 3, 20, 10, 390, 390, 0), ("bf16", 72, 3, 20, 10, 250, 30, 45),
    ("bf16", 48, 4, 20, 10, 300, 500, 7), ("f32", 250, 2, 20, 10, 200, 33, 9), ("f32", 256, 1, 6, 3, 300, 64, 40),
    ("f32", 64, 1, 4, 2, 1500, 65, 20), ("bf16", 80, 1, 3, 1, 1300, 40, 8), ("f32", 128, 1, 2, 2, 1000, 32, 1)])
def test_gradients_on_the_cuda_cores(osf, dtype, D, B, Hq, Hkv, S, window, sinks):
    """Many vectors (32 to a block) and few (8), sinks whose rows are shared out over blocks."""
    run(osf, dtype, B, Hq, Hkv, S, S, D, window, sinks, grad=True)


@pytest.mark.parametrize("D", [64, 96])
def test_gradients_of_tensors_off_16_bytes(osf, D):
    """bfloat16 tensors that the tensor-core path cannot address: the CUDA cores', with its workspace."""
    B, Hq, Hkv, S, window, sinks = 1, 4, 2, 500, 100, 9
    q, k, v = si.qkv((B, Hq, S, D), (B, Hkv, S, D), seed=4, dtype="bf16")
    g = si.qkv((B, Hq, S, D), (1, 1, 1, D), seed=5, dtype="bf16")[0]
    off = [torch.empty(x.size + 1, dtype=torch.bfloat16, device="cuda")[1:].view(x.shape).copy_(bf16_tensor(x)) for x in (q, k, v, g)]
    ref = oracle.attention_window(f64(q, "bf16"), f64(k, "bf16"), f64(v, "bf16"), window, sinks, dO=f64(g, "bf16"))
    lse = torch.empty(B, Hq, S, device="cuda")
    o = osf.osf_attn_fwd_gqa_window(*off[:3], window, sinks, lse=lse)
    check_out(o, lse, ref, "bf16", "off 16 bytes")
    check_grads(osf.osf_attn_bwd_gqa_window(*off[:3], o, off[3], lse, window, sinks), ref, "bf16", "off 16 bytes")
