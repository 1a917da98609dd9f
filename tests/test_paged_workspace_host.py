"""Workspace sizes of the block selection (no GPU needed)."""
import pytest

from mixture_value_projection_amd import binding


@pytest.mark.parametrize("B,H", [(1, 1), (1, 8), (3, 2), (2048, 1)])
@pytest.mark.parametrize("max_blocks", [1, 16, 17, 65, 81, 97, 113, 145, 1000, 60003])
def test_selection_scratch_holds_whole_tiles(B, H, max_blocks):
    """The choice reads a row's blocks in tiles of 16, eight bytes each, up to
    the end of its last tile, and eight bytes a tile."""
    tiles = -(-max_blocks // 16)
    need = 8 * B * H * (16 * tiles + tiles)
    assert binding.load_library().mova_block_select_workspace_bytes(B, 4 * H, H, 128, max_blocks,
                                                                    16, 4) >= need
