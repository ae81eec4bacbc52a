"""The cache operators together, as a serving loop uses them: a prompt through the forward kernel, the
weights its rows leave on the keys, the prompt stored in 4 bits and cut to a budget, then decode steps
that append, attend, accumulate weights and evict.  Also the calls inside a captured graph, on another
stream, and two at once."""
import numpy as np
import pytest

import oracle
from conftest import bf16_tensor
import seeded_inputs as si

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def normal(shape, seed):
    return bf16_tensor(si.f32_to_bf16_bits(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)))


@pytest.mark.parametrize("D", [64, 128])
def test_serving_loop(osf, D):
    B, Hq, Hkv, P, S, budget, steps = 2, 8, 2, 300, 340, 200, 12
    R = osf.osf_kv4_record_bytes(D)
    q, k, v = (normal((B, h, P, D), i) for i, h in enumerate((Hq, Hkv, Hkv)))
    lse = torch.empty(B, Hq, P, device="cuda")
    osf.osf_attn_fwd_gqa_ex(q, k, v, mask="top_left", lse=lse)
    w = torch.zeros(B, Hkv, S, device="cuda")
    w[:, :, :P] = osf.osf_attn_key_weights(q, k, lse, mask="top_left")
    want_w = oracle.key_weights(*(x.double().cpu().numpy() for x in (q, k, lse)), mask="top_left")
    assert np.allclose(w[:, :, :P].cpu().numpy(), want_w, rtol=1e-4)
    cache = torch.zeros(B, Hkv, S, R, dtype=torch.uint8, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    counts = torch.tensor([P, 170], dtype=torch.int32, device="cuda")   # the second prompt is shorter
    w[1, :, 170:] = 0
    osf.osf_kv4_append(k, v, cache, lens=lens, counts=counts)
    lens += counts
    rec, host_w, host_n = cache.cpu().numpy(), w.cpu().numpy().astype(np.float64), [P, 170]
    for step in range(steps):
        if step % 5 == 0:
            osf.osf_kv_evict(cache, None, w, budget, lens=lens, sinks=4, recent=32, k_out=cache, weights_out=w, lens_out=lens)
            # the host follows the device's own weights, so that near ties cannot differ
            keep_w = w.cpu().numpy()
            for b in range(B):
                for h in range(Hkv):
                    got = cache[b, h].cpu().numpy()
                    new = min(host_n[b], budget)
                    live = {r.tobytes() for r in rec[b, h, :host_n[b]]}
                    assert all(r.tobytes() in live for r in got[:new])
                host_n[b] = min(host_n[b], budget)
            rec, host_w = cache.cpu().numpy(), keep_w.astype(np.float64)
            assert lens.tolist() == host_n
        qn, kn, vn = (normal((B, h, 1, D), 100 + 3 * step + i) for i, h in enumerate((Hq, Hkv, Hkv)))
        osf.osf_kv4_append(kn, vn, cache, lens=lens)
        lens += 1
        out = osf.osf_attn_kv4(qn, cache, lens=lens, mask="bottom_right", weights=w, accumulate=True)
        for b in range(B):
            rec[b, :, host_n[b]] = oracle.records(kn[b, :, 0].double().cpu().numpy(), vn[b, :, 0].double().cpu().numpy())
            host_n[b] += 1
        assert np.array_equal(cache.cpu().numpy()[0, :, :host_n[0]], rec[0, :, :host_n[0]])
        O, _, W, A = oracle.attention_records(qn.double().cpu().numpy(), rec, host_n, "bottom_right")
        host_w += W
        assert np.all(np.abs(out.double().cpu().numpy() - O) <= 3 * 2.0 ** -8 * A + 1e-3 * A)
        assert np.allclose(w.cpu().numpy(), host_w, rtol=1e-4, atol=1e-6)
    # the stored prefix through the prompt kernel: the same keys and values as the decode kernel saw
    kk, vv = osf.osf_kv4_read(cache, D, int(lens.min()), lens=lens)
    n = int(lens.min())
    qn = normal((B, Hq, 40, D), 999)
    o = osf.osf_attn_fwd_gqa_ex(qn, kk, vv, mask="bottom_right")
    ref, _ = oracle.attention_gqa(*(x.double().cpu().numpy() for x in (qn, kk, vv)), mask="bottom_right")
    assert np.all(np.abs(o.double().cpu().numpy() - ref) <= 2e-2 + 1e-2 * np.abs(ref)) and n == kk.shape[2]
    assert osf.osf_device_status() == osf.OSF_OK


def step_state(osf, seed=0, B=2, Hq=8, Hkv=2, S=5000, D=128, n=4000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    st = dict(q=r(B, Hq, 1, D), kn=r(B, Hkv, 1, D), vn=r(B, Hkv, 1, D), cache=torch.zeros(B, Hkv, S, 160, dtype=torch.uint8, device="cuda"),
              lens=torch.full((B,), n, dtype=torch.int32, device="cuda"), one=torch.ones(B, dtype=torch.int32, device="cuda"),
              w=torch.rand(B, Hkv, S, generator=g, device="cuda"), out=torch.zeros(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda"),
              lse=torch.zeros(B, Hq, 1, device="cuda"), kq=r(B, Hkv, 700, D), qq=r(B, Hq, 700, D), w2=torch.zeros(B, Hkv, 700, device="cuda"),
              lse2=torch.full((B, Hq, 700), 8.0, device="cuda"))
    osf.osf_kv4_append(r(B, Hkv, n, D), r(B, Hkv, n, D), st["cache"])
    st["ws"] = torch.empty(osf.osf_attn_kv4_workspace_bytes(osf.OSF_BF16, B, Hq, Hkv, 1, S, D, True), dtype=torch.uint8, device="cuda")
    st["ws2"] = torch.empty(max(1, osf.osf_attn_key_weights_workspace_bytes(osf.OSF_BF16, B, Hq, Hkv, 700, 700, D)), dtype=torch.uint8,
                            device="cuda")
    st["idx"] = torch.zeros(B, Hkv, 3000, dtype=torch.int32, device="cuda")
    return st


def step(osf, st):
    osf.osf_kv4_append(st["kn"], st["vn"], st["cache"], lens=st["lens"])
    st["lens"].add_(st["one"])
    osf.osf_attn_kv4(st["q"], st["cache"], lens=st["lens"], out=st["out"], lse=st["lse"], weights=st["w"], accumulate=True,
                     workspace=st["ws"])
    osf.osf_kv_evict(st["cache"], None, st["w"], 3000, lens=st["lens"], sinks=4, recent=100, k_out=st["cache"], weights_out=st["w"],
                     lens_out=st["lens"], idx=st["idx"])
    osf.osf_attn_key_weights(st["qq"], st["kq"], st["lse2"], weights=st["w2"], mask="top_left", workspace=st["ws2"])


RESULTS = ("cache", "lens", "w", "out", "lse", "idx", "w2")


def test_captured_steps_equal_eager_ones(osf):
    eager, graphed = step_state(osf), step_state(osf)
    warm = step_state(osf, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(osf, warm)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(osf, graphed)
    for _ in range(3):
        step(osf, eager)
        g.replay()
    torch.cuda.synchronize()
    for name in RESULTS:
        assert torch.equal(eager[name], graphed[name]), name
    assert eager["lens"].tolist() == [3000, 3000]
    assert osf.osf_device_status() == osf.OSF_OK


def test_two_streams_at_once(osf):
    states = [step_state(osf, seed=s) for s in (2, 3)]
    alone = [step_state(osf, seed=s) for s in (2, 3)]
    for st in alone:
        step(osf, st)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for s, st in zip(streams, states):
        with torch.cuda.stream(s):
            step(osf, st)
    torch.cuda.synchronize()
    for a, b in zip(alone, states):
        for name in RESULTS:
            assert torch.equal(a[name], b[name]), name
