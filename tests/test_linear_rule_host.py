"""Which form of moe_linear_fp8 runs (no GPU needed)."""

import pytest

from combine_top_route_moe_amd import ops
from tests.linear_forms import FORMS


@pytest.mark.parametrize("M,N,K,tile", [
    # 256 x 256 tiles on some of the 256 CUs, us of them and of 128 x 128 tiles
    (1024, 8192, 2048, 128),       # 128 tiles: 29.0, 22.0
    (1536, 6000, 4096, 256),       # 144: 48.0, 53.3
    (2048, 4096, 7168, 128),       # 128: 82.0, 61.8
    (2304, 4096, 7168, 256),       # 144: 82.6, 91.3
    (2816, 4096, 7168, 256),       # 176: 90.3, 95.6
    (2048, 6000, 4096, 256),       # 192: 52.6, 58.3
    # on all of them, and on some of them once more
    (4096, 4096, 7168, 256),       # 256: 98.8, 123
    (2304, 8192, 2048, 128),       # 288: 56.2, 48.1
    (5120, 4096, 7168, 128),       # 320: 166, 159
    (3328, 8192, 2048, 256),       # 416: 60.6, 64.7
    (6144, 4096, 7168, 256),       # 384: 172, 183
    (8192, 4096, 7168, 256),       # 512: 186, 236
])
def test_large_tiles_by_how_many_of_them_run(M, N, K, tile):
    assert ops.moe_linear_fp8_parts(M, N, K) == (1, (tile, tile))


@pytest.mark.parametrize("M,N,K,tile,parts", FORMS)
def test_the_products_that_are_tested_reach_every_form(M, N, K, tile, parts):
    assert ops.moe_linear_fp8_parts(M, N, K) == (parts, tile)


def test_no_form_is_left_out():
    kinds = {(tile, parts) for *_, tile, parts in FORMS}
    assert kinds >= {((64, 64), 2), ((64, 64), 4), ((64, 64), 8), ((64, 128), 2), ((64, 128), 4), ((64, 128), 8),
                     ((128, 128), 2), ((128, 128), 4), ((128, 128), 8)} | {((m, n), 1) for m, n in ((64, 64), (64, 128), (128, 128), (256, 256))}
    for parts in (2, 4, 8):
        assert {min(M * N % 4, 1) for M, N, _, _, p in FORMS if p == parts} == {0, 1}
