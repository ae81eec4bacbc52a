"""Workspaces of the cache operators: what the query says is enough, for every mask, and nothing behind it is written."""
import pytest

from test_gpu_key_weights import qk
from test_gpu_kv4 import random_cache, rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CANARY = 0x5A


def guarded(n):
    """(workspace of exactly n bytes, the bytes behind it)."""
    buf = torch.full((n + 4096,), CANARY, dtype=torch.uint8, device="cuda")
    return buf[:n], buf[n:]


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv,Sq,Sk,split", [
    ("f32", 64, 1, 3, 1, 700, 700, True), ("f32", 40, 1, 2, 2, 65, 5000, True), ("bf16", 96, 2, 4, 1, 900, 130, True),
    ("f32", 64, 1, 1, 1, 2500, 64, True), ("bf16", 96, 1, 1, 1, 2500, 64, True), ("bf16", 64, 1, 4, 2, 300, 1500, True),
    ("bf16", 128, 3, 5, 1, 257, 511, True), ("bf16", 128, 2, 8, 2, 1, 3000, False)])
def test_key_weights(osf, dtype, D, B, Hq, Hkv, Sq, Sk, split):
    q, k = qk(B, Hq, Hkv, Sq, Sk, D, dtype, Sq + Sk)
    lse = torch.full((B, Hq, Sq), 7.0, device="cuda")
    n = osf.osf_attn_key_weights_workspace_bytes(osf.OSF_F32 if dtype == "f32" else osf.OSF_BF16, B, Hq, Hkv, Sq, Sk, D)
    if split:
        assert n > 0
    used = False
    for mask in ("none", "top_left", "bottom_right"):
        ws, behind = guarded(n)
        got = osf.osf_attn_key_weights(q, k, lse, mask=mask, workspace=ws)
        want = osf.osf_attn_key_weights(q, k, lse, mask=mask)
        assert torch.equal(got, want) and bool((behind == CANARY).all())
        used |= bool((ws != CANARY).any())
    assert used == split   # parts were kept there (under some mask: one that hides most rows may leave a single part)
    assert osf.osf_device_status() == osf.OSF_OK


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv,Sq,S,split", [
    ("bf16", 64, 2, 8, 2, 1, 5000, True), ("bf16", 128, 1, 4, 1, 5, 3000, True), ("bf16", 128, 40, 8, 1, 3, 4000, True),
    ("f32", 128, 2, 4, 2, 3, 3000, True), ("bf16", 96, 1, 6, 3, 1, 2000, True), ("bf16", 64, 2, 4, 2, 1, 300, False)])
def test_attention(osf, dtype, D, B, Hq, Hkv, Sq, S, split):
    q, _ = rows((B, Hq, Sq, D), S, dtype)
    cache, _ = random_cache(1, Hkv, S, D, D)
    cache = cache.expand(B, -1, -1, -1).contiguous()
    lens = torch.randint(0, S + 1, (B,), dtype=torch.int32, device="cuda")
    lens[0] = S
    for weights in (False, True):
        n = osf.osf_attn_kv4_workspace_bytes(osf.OSF_F32 if dtype == "f32" else osf.OSF_BF16, B, Hq, Hkv, Sq, S, D, weights)
        if split or weights:
            assert n > 0
        for mask in ("none", "bottom_right"):
            w = [torch.zeros(B, Hkv, S, device="cuda") if weights else None for _ in range(2)]
            ws, behind = guarded(n)
            got = osf.osf_attn_kv4(q, cache, lens=lens, mask=mask, weights=w[0], workspace=ws)
            want = osf.osf_attn_kv4(q, cache, lens=lens, mask=mask, weights=w[1])
            assert torch.equal(got, want) and bool((behind == CANARY).all())
            assert not weights or torch.equal(w[0], w[1])
    assert osf.osf_device_status() == osf.OSF_OK
