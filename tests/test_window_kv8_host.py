"""The windowed and paged entry points without a GPU: pins of the oracle, and every refusal that the host makes before it
touches a device."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import oracle

P = [ctypes.c_void_p(x << 40) for x in range(1, 20)]
torch = pytest.importorskip("torch")


# ------------------------------------------------------------------------------------------ oracle
def test_window_mask_closed_forms():
    m = oracle.window_mask(4, 6, 2, 1).astype(int).tolist()
    assert m == [[1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert oracle.window_mask(3, 1, 5, 2).astype(int).tolist() == [[0], [0], [1]]
    assert (oracle.window_mask(5, 9, 9, 0) == oracle.window_mask(5, 9, 0, 3)).all()


def test_windowed_attention_is_the_masked_one():
    rng = np.random.default_rng(0)
    q, k, v, g = (rng.standard_normal((1, h, s, 8)) for h, s in ((4, 6), (2, 9), (2, 9), (4, 6)))
    O, lse, size, dq, dk, dv, _ = oracle.attention_window(q, k, v, 9, 0, dO=g)
    ref, ref_lse = oracle.attention_gqa(q, k, v, mask="bottom_right")
    assert np.allclose(O, ref, atol=1e-12) and np.allclose(lse, ref_lse, atol=1e-12) and (size >= np.abs(O) - 1e-12).all()
    for a, b in zip((dq, dk, dv), oracle.attention_gqa_bwd(q, k, v, g, mask="bottom_right")):
        assert np.allclose(a, b, atol=1e-12)
    # a window of one token: every row is its own value
    O = oracle.attention_window(q, k, v, 1, 0)[0]
    assert np.allclose(O[0, 3], v[0, 1, 3:])
    # one row by brute force
    O, lse, _ = oracle.attention_window(q, k, v, 2, 1)
    keys = [0, 5, 6]   # row 3 stands at 6
    s = [float(q[0, 1, 3] @ k[0, 0, j]) * 8 ** -0.5 for j in keys]
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(O[0, 1, 3], sum(x * v[0, 0, j] for x, j in zip(w, keys)))
    assert np.isclose(lse[0, 1, 3], np.log(np.exp(s).sum()))


def test_windowed_gradients_by_differences():
    rng = np.random.default_rng(1)
    q, k, v, g = (rng.standard_normal((1, h, s, 4)) for h, s in ((2, 5), (1, 7), (1, 7), (2, 5)))
    grads = oracle.attention_window(q, k, v, 3, 1, dO=g)[3:6]
    for x, d in zip((q, k, v), grads):
        for i in range(0, x.size, 3):
            at = np.unravel_index(i, x.shape)
            old, f = x[at], []
            for step in (1e-6, -1e-6):
                x[at] = old + step
                f.append((oracle.attention_window(q, k, v, 3, 1)[0] * g).sum())
            x[at] = old
            assert abs((f[0] - f[1]) / 2e-6 - d[at]) < 1e-7


def test_e4m3_values_and_codes():
    v = oracle.e4m3_values()
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and np.isnan(v[0x7f]) and v[0x38] == 1.0
    assert np.array_equal(v[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    codes = np.r_[0:127, 128:255].astype(np.uint8)
    assert np.array_equal(oracle.e4m3_codes(v[codes]), codes)
    rng = np.random.default_rng(2)
    x = rng.standard_normal(2000) * 2.0 ** rng.uniform(-14, 6, 2000)
    x = np.r_[x, (v[1:127] + v[:126]) / 2]   # and every tie
    assert np.abs(x).max() <= 448
    ref = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.e4m3_codes(x.astype(np.float32)), ref)
    assert list(oracle.e4m3_codes([np.nan, np.inf, -np.inf])) == [127] * 3


def test_scale_exponents():
    assert oracle.scale_exponent(448.0) == 0 and oracle.scale_exponent(np.nextafter(448.0, 500)) == 1
    assert oracle.scale_exponent(224.0) == -1 and oracle.scale_exponent(0.0) == -110
    assert oracle.scale_exponent(float(np.finfo(np.float32).max)) == 120


def test_rotation_by_fractions():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 8)).astype(np.float32)
    ang = rng.uniform(0, 6, (2, 4))
    c, s = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    for inter in (False, True):
        y = oracle.rotate(x, np.arange(2), c, s, inter)
        for t in range(2):
            for i in range(4):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + 4)
                exact = Fraction(float(x[t, a])) * Fraction(float(c[t, i])) - Fraction(float(x[t, b])) * Fraction(float(s[t, i]))
                assert abs(Fraction(float(y[t, a])) - exact) <= abs(exact) * Fraction(1, 2 ** 24)


def test_appending_piece_by_piece():
    """A page's values do not depend on how its tokens came while its scale does not grow; where it grows, codes shift."""
    rng = np.random.default_rng(4)
    k, v = rng.standard_normal((2, 1, 1, 20, 8))
    table = np.array([[1, 0]])
    k[0, 0, 0, 0] = v[0, 0, 0, 0] = 4.0   # the largest comes first
    k, v = np.clip(k, -4, 4), np.clip(v, -4, 4)
    whole, parts = [(np.zeros((2, 2, 1, 16, 8), np.uint8), np.ones((2, 2, 1), np.float32)) for _ in range(2)]
    oracle.kv8_append(k, v, *whole, table)
    for t in range(16):
        oracle.kv8_append(k[:, :, t:t + 1], v[:, :, t:t + 1], *parts, table, lens=[t])
    oracle.kv8_append(k[:, :, 16:], v[:, :, 16:], *parts, table, lens=[16])
    assert np.array_equal(whole[0], parts[0]) and np.array_equal(whole[1], parts[1])
    K, _ = oracle.kv8_values(*whole, table[0], 20)
    assert np.all(np.abs(K - k[0]) <= np.abs(k[0]) / 16 + 2.0 ** -17)


# ------------------------------------------------------------------------------------------ refusals
def _window(lib, fwd=True, B=1, Hq=4, Hkv=2, Sq=5, Sk=9, D=64, dtype=1, window=3, sinks=1, scale=0.0, ptrs=None, lse=None,
            strides=None, ws=None):
    if fwd:
        q, k, v, o = ptrs or P[:4]
        return lib.osf_attn_fwd_gqa_window(q, k, v, o, dtype, B, Hq, Hkv, Sq, Sk, D, strides, window, sinks, scale, lse, ws, 0, None)
    p = ptrs or P[:9]
    return lib.osf_attn_bwd_gqa_window(*p, dtype, B, Hq, Hkv, Sq, Sk, D, window, sinks, scale, ws, 0, None)


@pytest.mark.parametrize("fwd", [True, False])
def test_window_refusals(osf, fwd):
    lib = osf.lib()
    for bad in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(Hq=3), dict(Hkv=0), dict(dtype=2), dict(D=0), dict(Sq=-1),
                dict(scale=float("nan")), dict(Sk=-2)):
        assert _window(lib, fwd, **bad) == osf.OSF_ERR_INVALID, bad
    for bad in (dict(D=257), dict(Sq=1 << 29, D=1, Sk=1 << 29), dict(Sk=1 << 29, D=2)):
        assert _window(lib, fwd, **bad) == osf.OSF_ERR_UNSUPPORTED, bad
    assert _window(lib, fwd, B=0) == osf.OSF_OK
    n = 4 if fwd else 9
    for i in range(n):
        ptrs = list(P[:n])
        ptrs[i] = None
        assert _window(lib, fwd, ptrs=ptrs) == osf.OSF_ERR_INVALID, i
    if fwd:
        assert _window(lib, ptrs=[P[0], P[1], P[2], P[0]]) == osf.OSF_ERR_INVALID   # O over Q
        assert _window(lib, lse=P[3]) == osf.OSF_ERR_INVALID
        st = (ctypes.c_longlong * 12)(*[-1] + [64] * 11)
        assert _window(lib, strides=ctypes.cast(st, ctypes.c_void_p)) == osf.OSF_ERR_INVALID
    else:
        for i, j in ((6, 0), (7, 1), (8, 2), (6, 7), (7, 8), (6, 3), (7, 5)):
            ptrs = list(P[:9])
            ptrs[i] = ptrs[j]
            assert _window(lib, False, ptrs=ptrs) == osf.OSF_ERR_INVALID, (i, j)


def test_window_workspace_refusals(osf):
    lib, n = osf.lib(), ctypes.c_size_t(7)
    for f in (lib.osf_attn_window_workspace_bytes, lib.osf_attn_bwd_window_workspace_bytes):
        assert f(1, 1, 4, 2, 5, 9, 64, 0, 0, ctypes.byref(n)) == osf.OSF_ERR_INVALID and n.value == 0
        assert f(1, 1, 4, 2, 5, 9, 64, 1, -1, ctypes.byref(n)) == osf.OSF_ERR_INVALID
        assert f(1, 1, 4, 3, 5, 9, 64, 1, 1, ctypes.byref(n)) == osf.OSF_ERR_INVALID
        assert f(1, 1, 4, 2, 5, 9, 300, 1, 1, ctypes.byref(n)) == osf.OSF_ERR_UNSUPPORTED
        assert f(1, 1, 4, 2, 5, 9, 64, 1, 1, None) == osf.OSF_ERR_INVALID
        assert f(1, 0, 4, 2, 5, 9, 64, 1, 1, ctypes.byref(n)) == osf.OSF_OK and n.value == 0


def _append(lib, B=1, Hkv=2, n=3, D=64, dtype=1, strides=None, pages=P[2], scales=P[3], n_pages=4, pt=16, table=P[4], per=2,
            lens=None, counts=None, cos=P[5], sin=P[6], maxp=64, rot=32, inter=0, Q=None, Qo=None, Hq=0, k=P[0], v=P[1]):
    return lib.osf_kv8_append(k, v, dtype, B, Hkv, n, D, strides, pages, scales, n_pages, pt, table, per, lens, counts, cos,
                              sin, maxp, rot, inter, Q, Qo, Hq, None)


def test_kv8_append_refusals(osf):
    lib = osf.lib()
    I, U = osf.OSF_ERR_INVALID, osf.OSF_ERR_UNSUPPORTED
    odd = ctypes.c_void_p((3 << 40) + 8)
    for want, bad in ((I, dict(dtype=3)), (I, dict(B=-1)), (I, dict(Hkv=0)), (I, dict(n=-1)), (I, dict(pt=0)), (U, dict(pt=24)),
                      (U, dict(pt=256)), (U, dict(D=48)), (U, dict(D=288)), (I, dict(rot=72)), (I, dict(rot=-8)), (U, dict(rot=12)),
                      (I, dict(k=None)), (I, dict(v=None)), (I, dict(pages=None)), (I, dict(scales=None)), (I, dict(table=None)),
                      (I, dict(cos=None)), (I, dict(sin=None)), (I, dict(maxp=0)), (I, dict(maxp=-1)), (I, dict(pages=odd)),
                      (I, dict(n=40)), (I, dict(n_pages=0)), (I, dict(per=0, counts=P[7])), (I, dict(Q=P[8])),
                      (I, dict(Q=P[8], Qo=P[9], Hq=3)), (I, dict(Q=P[8], Qo=P[9])), (I, dict(Q=P[0], Qo=P[0] and P[1], Hq=2)),
                      (I, dict(pages=P[0])), (I, dict(scales=P[1])), (I, dict(table=P[2])), (I, dict(lens=P[3])),
                      (U, dict(B=40000)), (U, dict(n_pages=1 << 30)), (U, dict(per=1 << 28, counts=P[7]))):
        assert _append(lib, **bad) == want, bad
    assert _append(lib, B=0) == osf.OSF_OK and _append(lib, n=0) == osf.OSF_OK
    st = (ctypes.c_longlong * 6)(*[-1] + [64] * 5)
    assert _append(lib, strides=ctypes.cast(st, ctypes.c_void_p)) == I


def test_kv8_read_refusals(osf):
    lib, I, U = osf.lib(), osf.OSF_ERR_INVALID, osf.OSF_ERR_UNSUPPORTED

    def read(pages=P[0], scales=P[1], n_pages=4, pt=16, table=P[2], per=2, K=P[3], V=P[4], dtype=1, B=1, Hkv=2, n=3, D=64,
             starts=None, lens=None):
        return lib.osf_kv8_read(pages, scales, n_pages, pt, table, per, K, V, dtype, B, Hkv, n, D, starts, lens, None)
    for want, bad in ((I, dict(K=None)), (I, dict(V=None)), (I, dict(K=P[4])), (I, dict(K=P[0])), (I, dict(V=P[1])), (I, dict(V=P[2])),
                      (I, dict(lens=P[3])), (I, dict(starts=P[4])), (U, dict(pt=8)), (U, dict(D=16)), (I, dict(pages=None)),
                      (I, dict(table=None)), (I, dict(dtype=2))):
        assert read(**bad) == want, bad
    assert read(n=0) == osf.OSF_OK


def test_attn_kv8_refusals(osf):
    lib, I, U = osf.lib(), osf.OSF_ERR_INVALID, osf.OSF_ERR_UNSUPPORTED

    def attn(Q=P[0], pages=P[1], scales=P[2], O=P[3], dtype=1, B=1, Hq=4, Hkv=2, Sq=1, n_pages=4, pt=16, D=64, strides=None,
             table=P[4], per=2, lens=None, window=0, sinks=0, scale=0.0, lse=None):
        return lib.osf_attn_kv8(Q, pages, scales, O, dtype, B, Hq, Hkv, Sq, n_pages, pt, D, strides, table, per, lens, window,
                                sinks, scale, lse, None, 0, None)
    for want, bad in ((I, dict(Hq=3)), (I, dict(Hq=0)), (I, dict(window=-1)), (I, dict(sinks=-1)), (I, dict(scale=float("nan"))),
                      (I, dict(Q=None)), (I, dict(O=None)), (I, dict(O=P[0])), (I, dict(O=P[1])), (I, dict(lse=P[3])),
                      (I, dict(lse=P[4])), (I, dict(pages=None)), (I, dict(table=None)), (U, dict(D=80)), (U, dict(pt=512)),
                      (U, dict(Sq=1 << 15)), (I, dict(Sq=-1)), (U, dict(B=1 << 16))):
        assert attn(**bad) == want, bad
    assert attn(Sq=0) == osf.OSF_OK and attn(B=0) == osf.OSF_OK
    n = ctypes.c_size_t(7)
    f = lib.osf_attn_kv8_workspace_bytes
    assert f(1, 1, 4, 2, 1, 64, 16, 2, 0, 0, None) == I
    assert f(1, 1, 4, 2, 1, 64, 17, 2, 0, 0, ctypes.byref(n)) == U and n.value == 0
    assert f(1, 1, 4, 2, 1, 64, 16, 2, -1, 0, ctypes.byref(n)) == I
    assert f(1, 1, 4, 2, 0, 64, 16, 2, 0, 0, ctypes.byref(n)) == osf.OSF_OK and n.value == 0


def test_misaligned_buffers_are_refused(osf):
    """A buffer that does not start on a boundary of its elements would fault in a kernel."""
    lib, I = osf.lib(), osf.OSF_ERR_INVALID

    def off(p, by):
        return ctypes.c_void_p(p.value + by)
    for dtype, by in ((1, 1), (0, 2)):
        for i in range(4):
            ptrs = list(P[:4])
            ptrs[i] = off(ptrs[i], by)
            assert _window(lib, dtype=dtype, ptrs=ptrs) == I, i
        for i in range(9):
            ptrs = list(P[:9])
            ptrs[i] = off(ptrs[i], by)
            assert _window(lib, False, dtype=dtype, ptrs=ptrs) == I, i
        for name, p in (("k", P[0]), ("v", P[1]), ("Q", P[8]), ("Qo", P[9])):
            assert _append(lib, dtype=dtype, **{**dict(Q=P[8], Qo=P[9], Hq=2), name: off(p, by)}) == I, name
        for i in range(2):
            kv = [P[3], P[4]]
            kv[i] = off(kv[i], by)
            assert lib.osf_kv8_read(P[0], P[1], 4, 16, P[2], 2, *kv, dtype, 1, 2, 3, 64, None, None, None) == I
            qo = [P[3], P[4]]
            qo[i] = off(qo[i], by)
            assert lib.osf_attn_kv8(qo[0], P[0], P[1], qo[1], dtype, 1, 4, 2, 1, 4, 16, 64, None, P[2], 2, None, 0, 0, 0.0, None,
                                    None, 0, None) == I
    assert _window(lib, lse=off(P[4], 2)) == I
    for name, p in (("scales", P[3]), ("table", P[4]), ("cos", P[5]), ("sin", P[6]), ("lens", P[10]), ("counts", P[11])):
        assert _append(lib, **{name: off(p, 2)}) == I, name
    for args in ((off(P[1], 2), P[2], None, None), (P[1], off(P[2], 1), None, None), (P[1], P[2], off(P[5], 2), None),
                 (P[1], P[2], None, off(P[6], 2))):
        scales, table, lens, lse = args
        assert lib.osf_attn_kv8(P[3], P[0], scales, P[4], 1, 1, 4, 2, 1, 4, 16, 64, None, table, 2, lens, 0, 0, 0.0, lse, None, 0,
                                None) == I
        if lse is None:
            assert lib.osf_kv8_read(P[0], scales, 4, 16, table, 2, P[3], P[4], 1, 1, 2, 3, 64, lens, None, None) == I
