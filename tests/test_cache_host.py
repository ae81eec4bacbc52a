"""The cache entry points without a GPU: the oracle's own pins, and every refusal that the host makes
before it touches a device."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import oracle

P = [ctypes.c_void_p(x << 40) for x in range(1, 12)]


# ------------------------------------------------------------------------------------------ oracle
def test_quantised_group_covers_its_values():
    rng = np.random.default_rng(0)
    for _ in range(200):
        x = (rng.standard_normal(32) * 10.0 ** rng.integers(-6, 6) + rng.standard_normal()).astype(np.float32)
        codes, s, m = oracle.quantise_group(x)
        assert min(codes) >= 0 and max(codes) <= 15
        for v, c in zip(x, codes):
            assert abs(Fraction(m) + Fraction(s) * c - Fraction(float(v))) <= Fraction(s) / 2
        for b in (s, m):   # both are bfloat16
            assert int(np.float32(b).view(np.uint32)) & 0xFFFF == 0


def test_quantised_group_closed_forms():
    # 0 .. 15 twice: scale 1, minimum 0; a constant group: scale 0
    assert oracle.quantise_group(list(range(16)) * 2) == (list(range(16)) * 2, 1.0, 0.0)
    assert oracle.quantise_group([-3.5] * 32) == ([0] * 32, 0.0, -3.5)
    # ties go to the even code: 0.5, 1.5, 2.5 of scale 1
    codes, s, m = oracle.quantise_group([0.0, 0.5, 1.5, 2.5, 15.0] + [0.0] * 27)
    assert (codes[:5], s, m) == ([0, 0, 2, 2, 15], 1.0, 0.0)


def test_record_round_trip():
    rng = np.random.default_rng(1)
    for D in (32, 64, 96, 128, 256):
        k, v = rng.standard_normal((2, 3, D)).astype(np.float32)
        rec = oracle.records(k, v)
        assert rec.shape == (3, D + D // 4)
        (K, V), _ = oracle.record_values(rec)
        for x, y in ((k, K), (v, V)):
            for r in range(3):
                for g in range(D // 32):
                    codes, s, m = oracle.quantise_group(x[r, 32 * g:32 * g + 32])
                    assert np.array_equal(y[r, 32 * g:32 * g + 32], m + s * np.array(codes, float))


def test_key_weights_sum_to_the_rows():
    """Every row's weights sum to one, so a kv head's weights sum to its G * Sq rows."""
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((1, 4, 5, 8)), rng.standard_normal((1, 2, 7, 8)), rng.standard_normal((1, 2, 7, 8))
    _, lse = oracle.attention_gqa(q, k, v, mask="bottom_right")
    w = oracle.key_weights(q, k, lse, mask="bottom_right")
    assert np.allclose(w.sum(-1), 2 * 5, atol=1e-12)
    assert w[0, 0, -1] < w[0, 0].sum() / 5   # the last key is seen by the last row alone


def test_evict_oracle_closed_forms():
    w = np.array([9, 1, 5, 5, 0, 7, 2, 3], float)
    assert list(oracle.evict(w, 8, 8, 0, 0)) == list(range(8))
    assert list(oracle.evict(w, 8, 4, 1, 1)) == [0, 2, 5, 7]        # tie of 5s: the lower index
    assert list(oracle.evict(w, 6, 3, 0, 3)) == [3, 4, 5]
    assert list(oracle.evict(np.array([np.nan, 0.0, -0.0, -1.0]), 4, 3, 0, 0)) == [1, 2, 3]


# ------------------------------------------------------------------------------------------ refusals
def test_record_bytes(osf):
    n = ctypes.c_size_t(7)
    lib = osf.lib()
    for D in range(32, 257, 32):
        assert lib.osf_kv4_record_bytes(D, ctypes.byref(n)) == osf.OSF_OK and n.value == D * 5 // 4
    assert lib.osf_kv4_record_bytes(0, ctypes.byref(n)) == osf.OSF_ERR_INVALID
    assert lib.osf_kv4_record_bytes(48, ctypes.byref(n)) == osf.OSF_ERR_UNSUPPORTED
    assert lib.osf_kv4_record_bytes(288, ctypes.byref(n)) == osf.OSF_ERR_UNSUPPORTED
    assert lib.osf_kv4_record_bytes(64, None) == osf.OSF_ERR_INVALID


def test_append_refusals(osf):
    f = osf.lib().osf_kv4_append
    good = dict(K=P[0], V=P[1], dt=1, B=2, H=2, n=3, D=64, st=None, cache=P[2], S=8, lens=None, counts=None)

    def call(**kw):
        a = {**good, **kw}
        st = a["st"] and ctypes.cast((ctypes.c_longlong * 6)(*a["st"]), ctypes.c_void_p)
        return f(a["K"], a["V"], a["dt"], a["B"], a["H"], a["n"], a["D"], st, a["cache"], a["S"], a["lens"], a["counts"], None)

    bad, off = osf.OSF_ERR_INVALID, osf.OSF_ERR_UNSUPPORTED
    assert call(dt=5) == bad and call(B=-1) == bad and call(H=0) == bad and call(n=-1) == bad and call(S=-1) == bad
    assert call(D=48) == off and call(D=288) == off and call(B=70000) == off and call(S=1 << 30) == off
    assert call(K=None) == bad and call(V=None) == bad and call(cache=None) == bad
    assert call(cache=ctypes.c_void_p((3 << 40) + 8)) == bad             # 16-byte alignment
    assert call(cache=P[0]) == bad and call(V=P[2]) == bad               # overlap
    assert call(n=9) == bad                                              # more rows than records, without counts
    assert call(st=[-1, 64, 64, 1, 1, 1]) == bad and call(st=[1 << 41, 64, 64, 1, 1, 1]) == off
    assert call(lens=P[2]) == bad and call(counts=P[2]) == bad
    assert call(B=0) == osf.OSF_OK and call(n=0, K=None) == osf.OSF_OK


def test_read_refusals(osf):
    f = osf.lib().osf_kv4_read
    bad = osf.OSF_ERR_INVALID

    def call(cache=P[0], K=P[1], V=P[2], dt=1, B=2, H=2, n=3, D=64, S=8, starts=None, lens=None):
        return f(cache, K, V, dt, B, H, n, D, S, starts, lens, None)

    assert call(K=P[2]) == bad and call(K=P[0]) == bad and call(V=None) == bad and call(cache=None) == bad
    assert call(lens=P[1]) == bad and call(starts=P[2]) == bad and call(dt=3) == bad
    assert call(D=100) == osf.OSF_ERR_UNSUPPORTED
    assert call(n=0) == osf.OSF_OK


def test_attention_refusals(osf):
    f = osf.lib().osf_attn_kv4
    bad, off = osf.OSF_ERR_INVALID, osf.OSF_ERR_UNSUPPORTED

    def call(Q=P[0], cache=P[1], O=P[2], dt=1, B=2, Hq=4, Hkv=2, Sq=1, S=8, D=64, st=None, lens=None, mask=0, scale=0.0,
             lse=None, w=None, acc=0, ws=None, n=0):
        st = st and ctypes.cast((ctypes.c_longlong * 6)(*st), ctypes.c_void_p)
        return f(Q, cache, O, dt, B, Hq, Hkv, Sq, S, D, st, lens, mask, scale, lse, w, acc, ws, n, None)

    assert call(Hq=3) == bad and call(Hq=0) == bad and call(Sq=-1) == bad and call(mask=1) == bad and call(mask=9) == bad
    assert call(scale=float("nan")) == bad and call(Q=None) == bad and call(O=None) == bad and call(cache=None) == bad
    assert call(O=P[0]) == bad and call(O=P[1]) == bad and call(w=P[2]) == bad and call(lse=P[1]) == bad and call(w=P[0]) == bad
    assert call(lse=P[3], w=P[3]) == bad and call(lens=P[2]) == bad
    assert call(st=[64] * 6) == bad                                      # rows of O collide
    assert call(st=[-1, 1, 1, 256, 128, 64]) == bad
    assert call(D=80) == off and call(Sq=1 << 15) == off
    assert call(Sq=0) == osf.OSF_OK and call(B=0) == osf.OSF_OK
    n = ctypes.c_size_t(3)
    g = osf.lib().osf_attn_kv4_workspace_bytes
    assert g(1, 2, 3, 2, 1, 8, 64, 0, ctypes.byref(n)) == bad and n.value == 0
    assert g(1, 2, 4, 2, 1, 8, 64, 0, None) == bad


def test_key_weights_refusals(osf):
    f = osf.lib().osf_attn_key_weights
    bad, off = osf.OSF_ERR_INVALID, osf.OSF_ERR_UNSUPPORTED

    def call(Q=P[0], K=P[1], lse=P[2], w=P[3], dt=1, B=2, Hq=4, Hkv=2, Sq=3, Sk=8, D=64, st=None, mask=0, scale=0.0):
        st = st and ctypes.cast((ctypes.c_longlong * 6)(*st), ctypes.c_void_p)
        return f(Q, K, lse, w, dt, B, Hq, Hkv, Sq, Sk, D, st, mask, scale, 0, None, 0, None)

    assert call(dt=2) == bad and call(Hq=5) == bad and call(D=0) == bad and call(Sq=-1) == bad and call(mask=3) == bad
    assert call(Q=None) == bad and call(K=None) == bad and call(lse=None) == bad and call(w=None) == bad
    assert call(w=P[0]) == bad and call(w=P[1]) == bad and call(w=P[2]) == bad and call(scale=float("nan")) == bad
    assert call(D=300) == off and call(B=40000) == off
    assert call(st=[1, -1, 1, 1, 1, 1]) == bad
    assert call(Sk=0) == osf.OSF_OK and call(B=0) == osf.OSF_OK
    n = ctypes.c_size_t(3)
    assert osf.lib().osf_attn_key_weights_workspace_bytes(1, 2, 3, 2, 1, 8, 64, ctypes.byref(n)) == bad
    assert osf.lib().osf_attn_key_weights_workspace_bytes(1, 2, 4, 2, 1, 8, 64, None) == bad


def test_evict_refusals(osf):
    f = osf.lib().osf_kv_evict
    bad, off = osf.OSF_ERR_INVALID, osf.OSF_ERR_UNSUPPORTED

    def call(s0=P[0], d0=P[1], r0=128, s1=P[2], d1=P[3], r1=128, w=P[4], wo=P[5], lens=None, lo=None, idx=P[6], B=2, H=2, S=16,
             So=8, budget=8, sinks=1, recent=2):
        return f(s0, d0, r0, s1, d1, r1, w, wo, lens, lo, idx, B, H, S, So, budget, sinks, recent, None)

    assert call(budget=0) == bad and call(sinks=-1) == bad and call(recent=-1) == bad and call(sinks=7) == bad
    assert call(So=7) == bad and call(H=0) == bad and call(S=-1) == bad and call(r0=0) == bad and call(r1=-4) == bad
    assert call(d0=None) == bad and call(s1=None) == bad and call(w=None) == bad and call(wo=None) == bad and call(idx=None) == bad
    assert call(d0=P[0]) == bad                                          # in place needs S_out == S
    assert call(d1=P[0], So=16) == bad and call(wo=P[0]) == bad and call(idx=P[4]) == bad and call(lo=P[6]) == bad
    assert call(d0=ctypes.c_void_p((1 << 40) + 128), So=16) == bad       # shifted within the source
    assert call(B=40000) == off and call(S=1 << 30, So=1 << 29) == off and call(r0=1 << 29) == off
    assert call(B=0) == osf.OSF_OK


def test_binding_refuses_wrong_tensors(osf):
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 4, 64)
    c = torch.zeros(1, 2, 8, 80, dtype=torch.uint8)
    w = torch.zeros(1, 2, 8)
    for call in (lambda: osf.osf_kv4_append(x, x, c), lambda: osf.osf_kv4_read(c, 64, 4), lambda: osf.osf_attn_kv4(x, c),
                 lambda: osf.osf_attn_key_weights(x, x, w), lambda: osf.osf_kv_evict(c, None, w, 4)):
        with pytest.raises(ValueError):
            call()
