"""Attention over 4-bit records around the lengths at which items begin to be shared among CTAs, and past them."""
import numpy as np
import pytest

from test_gpu_kv4 import check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,tile", [(64, 64), (128, 32)])
@pytest.mark.parametrize("B,Hkv,tiles", [(1, 2, 27), (1, 2, 28), (1, 2, 29), (5, 8, 48), (5, 8, 49), (10, 8, 64), (10, 8, 65)])
def test_lengths_at_which_items_begin_to_be_cut(osf, D, tile, B, Hkv, tiles):
    """Items that fill less than a quarter, a quarter and half of the SMs."""
    S = tiles * tile - 3
    lens = [max(S - 6 * b * tile, 1) for b in range(B)]
    check_attention(osf, B, 2 * Hkv, Hkv, 1, S, D, "bf16", lens=lens, seed=tiles, weights=B == 1)


def cut(osf, B, Hq, Hkv, Sq, S, D):
    """Do CTAs share items?  Only then are partial states kept."""
    return osf.osf_attn_kv4_workspace_bytes(osf.OSF_BF16, B, Hq, Hkv, Sq, S, D) > 0


CUT = [(64, 70 * 64 - 5), (128, 70 * 32 - 5)]   # (D, records): 70 tiles, shared whatever the number of items


@pytest.mark.parametrize("D,S", CUT)
def test_a_large_ragged_batch_is_shared(osf, D, S):
    """More than 32 sequences, many of them empty, the long ones first, last and mixed."""
    B = 75
    lens = [int(x) for x in np.random.default_rng(D).integers(0, S + 1, B)]
    lens[:40] = [0] * 40
    for order in (lens, lens[::-1], lens[20:] + lens[:20]):
        assert cut(osf, B, 2, 1, 1, S, D)
        check_attention(osf, B, 2, 1, 1, S, D, "bf16", lens=order, seed=53, weights=False)
    check_attention(osf, B, 4, 2, 2, S, D, "bf16", lens=lens, mask="bottom_right", seed=54, weights=False)
    check_attention(osf, B, 2, 1, 1, S, D, "bf16", lens=[0] * (B - 1) + [S], seed=55)


@pytest.mark.parametrize("D,S", CUT)
@pytest.mark.parametrize("Hq,Hkv,Sq", [(24, 1, 1), (8, 2, 5), (4, 1, 11), (17, 1, 3)])
def test_several_blocks_of_query_rows_are_shared(osf, D, S, Hq, Hkv, Sq):
    """More than 16 rows of a kv head, over sequences of different lengths, some shorter than the rows, some empty."""
    lens = [S, 0, 1, S // 3, Sq, 33]
    assert cut(osf, len(lens), Hq, Hkv, Sq, S, D)
    check_attention(osf, len(lens), Hq, Hkv, Sq, S, D, "bf16", lens=lens, mask="bottom_right", seed=Hq + Sq)


@pytest.mark.parametrize("D,S", CUT)
def test_a_mask_over_a_ragged_batch_is_shared(osf, D, S):
    lens = [0, 1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 1000, S]
    for Hq, Hkv, Sq in ((4, 2, 3), (2, 2, 1), (2, 1, 2), (8, 2, 4)):
        assert cut(osf, len(lens), Hq, Hkv, Sq, S, D)
        check_attention(osf, len(lens), Hq, Hkv, Sq, S, D, "bf16", lens=lens, mask="bottom_right", seed=D + Sq)
    check_attention(osf, len(lens), 2, 1, 2, S, D, "bf16", lens=lens, seed=D)
