"""moe_grouped_ffn_fp4 on segments that overlap: more row tiles, or more runs of
few rows, than disjoint ones could have are reported, whether or not the launch
has workgroups for them."""

import numpy as np
import pytest
import torch

from combine_top_route_moe_amd import ops
from tests import few_util as fu
from tests.gpu_util import need_gpu, dev, dev_bf16

pytestmark = pytest.mark.gpu


def setup_module(module):
    need_gpu()
    assert ops.moe_device_check(0) == 0, "not a gfx950 device"


# rows, counts, H, I; every segment starts at row 0
CASES = [
    (16000, [16000, 600, 600], 256, 128),       # 128 row tiles and workgroups, 135 tiles
    (16000, [600, 16000, 600], 256, 128),
    (9000, [9000, 9000, 9000], 128, 768),       # a launch with workgroups to spare
    (3000, [3000, 3000, 3000], 128, 768),       # few-row kernels
    (20, [20, 20, 20], 128, 128),
]


@pytest.mark.parametrize("flags", [ops.MOE_FFN_ALL, ops.MOE_FFN_DOWN], ids=["all", "down"])
@pytest.mark.parametrize("rows,counts,H,I", CASES)
def test_more_tiles_than_disjoint_segments_have_are_reported(rows, counts, H, I, flags):
    rng = np.random.default_rng(rows)
    G = len(counts)
    w13, w2 = fu.make_weights(rng, G, H, I)
    handle = ops.ffn_weights(dev_bf16(w13), dev_bf16(w2), "mxfp4")
    x = dev_bf16(fu.bf16(rng.standard_normal((rows, H))))
    ws = torch.zeros(ops.moe_grouped_ffn_fp4_workspace_bytes(rows, G, H, I), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = dev(np.zeros(G + 1, np.int32))
    ops.moe_grouped_ffn_fp4(x, at, dev(np.array(counts, np.int32)), handle, flags=flags, workspace=ws, dev_error=err)
    assert int(err.item()) == ops.MOE_DEVERR_ROW_RANGE
    # the same rows in segments that do not overlap: nothing to report
    err.zero_()
    counts = np.diff([0, rows // 2, rows // 2, rows]).astype(np.int32)
    at = dev(np.array([0, rows // 2, rows // 2, rows], np.int32))
    ops.moe_grouped_ffn_fp4(x, at, dev(counts), handle, flags=flags, workspace=ws, dev_error=err)
    assert int(err.item()) == 0
