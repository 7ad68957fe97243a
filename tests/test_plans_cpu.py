"""Plans of the paged attention, as the size of their workspace tells them."""
import pytest

from diffusion_draft_tree_gb300 import ops


def _size(B, N, G, Hkv, D, tokens):
    return ops.workspace_size(ops.OP_TREE_ATTN_PAGED, B=B, N=N, Hq=G * Hkv, Hkv=Hkv, D=D, cache_cap=tokens)


@pytest.mark.parametrize("B,tokens,alone", [
    (10, 8192, True),      # 80 units of one pair, lists of 65 tiles: half of the SMs idle
    (12, 8192, True),
    (10, 10000, True),     # 80 tiles
    (10, 12000, False),    # lists long enough to be cut for the idle SMs
    (15, 8192, False),     # units enough
    (40, 8192, False),
])
def test_rows_left_over_are_not_taken_along_by_too_few_units(B, tokens, alone):
    """65 nodes of G = 4 are two query tiles and one node; three pieces a list or more.
    Its rows in a tile of their own need parts of a third tile."""
    part = B * 8 * 128 * 128 * 4
    pieces = -(-(-(-tokens // 128) + 1) // 32)
    n = _size(B, 64, 4, 8, 128, tokens)
    assert (n >= 3 * min(pieces, 4) * part) == alone
    assert n >= 2 * 3 * part
