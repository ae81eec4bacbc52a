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
