"""Sizes of the cache operators at the end of 32-bit integers, refused on the host."""
import ctypes


def test_key_weights_of_too_many_keys(osf):
    n = ctypes.c_size_t(3)
    query = osf.lib().osf_attn_key_weights_workspace_bytes
    for Sk in (2 ** 31 - 63, 2 ** 31 - 1):
        for Sq in (0, 1, 100):
            assert query(osf.OSF_F32, 1, 1, 1, Sq, Sk, 1, ctypes.byref(n)) == osf.OSF_ERR_UNSUPPORTED and n.value == 0
    # the largest that is taken (without a GPU the query then fails for want of one)
    assert query(osf.OSF_F32, 1, 1, 1, 100, 2 ** 31 - 64, 1, ctypes.byref(n)) in (osf.OSF_OK, osf.OSF_ERR_CUDA)
    P = [ctypes.c_void_p(x << 40) for x in range(1, 5)]
    call = osf.lib().osf_attn_key_weights
    assert call(P[0], P[1], P[2], P[3], osf.OSF_F32, 1, 1, 1, 4, 2 ** 31 - 1, 1, None, 0, 0.0, 0, None, 0, None) == osf.OSF_ERR_UNSUPPORTED
