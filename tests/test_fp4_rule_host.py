"""The rule that chooses moe_grouped_ffn_fp4's kernels, seen through its size
query (no GPU needed): the few-row form takes 4 I bytes a row, the tile form
2 I bytes for every row of ceil(capacity / 128) + G tiles of 128."""

import pytest

from combine_top_route_moe_amd import ops

# where an expert's weights cost about as much as a tile's walk, and far from it
SIZES = [(26, 4096, 1536), (42, 2048, 1024), (18, 7168, 2048), (52, 2048, 768), (25, 4096, 1536), (27, 4096, 1536),
         (17, 7168, 2048), (19, 7168, 2048), (41, 2048, 1024), (43, 2048, 1024), (110, 1024, 512), (1, 128, 128),
         (3, 512, 19200)]


def _few(n, I):
    return (n * I * 4 + 255) // 256 * 256


def _tile(n, G, I):
    return ((n + 127) // 128 + G) * 128 * I * 2


@pytest.mark.parametrize("G,H,I", SIZES)
def test_a_buffer_for_the_largest_batch_does_for_every_smaller_one(G, H, I):
    sizes = [ops.moe_grouped_ffn_fp4_workspace_bytes(n, G, H, I) for n in range(30 * G + 600)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("G,H,I", SIZES)
def test_sizes_hold_tiles_from_the_first_capacity_that_takes_them(G, H, I):
    """From the first size that is not the few-row form's on, all are at least
    the tile form's."""
    n, top = 1, 30 * G + 600
    while n < top and ops.moe_grouped_ffn_fp4_workspace_bytes(n, G, H, I) == _few(n, I):
        n += 1
    assert n >= min(8 * G, top)
    for m in range(n, top):
        assert ops.moe_grouped_ffn_fp4_workspace_bytes(m, G, H, I) >= _tile(m, G, I)


def test_the_numerics_cases_reach_both_forms():
    """Which kernels the cases of test_gpu_fp4_ffn.py run, so that neither form
    can drop out of them unnoticed."""
    from tests.test_gpu_fp4_ffn import FEW, MANY, TILE

    for form, cases in (("few", FEW + MANY), ("tile", TILE)):
        for counts, H, I in cases:
            n, G = sum(counts), len(counts)
            size = ops.moe_grouped_ffn_fp4_workspace_bytes(n, G, H, I)
            assert (size == _few(n, I)) == (form == "few"), (counts[:8], H, I)
            assert form == "few" or size >= _tile(n, G, I)
