"""moe_grouped_ffn_fp4: what each of its two forms keeps of the intermediate.
(tests/test_fp4_rule_host.py pins which cases run which.)"""

import numpy as np
import pytest
import torch

from combine_top_route_moe_amd import ops
from tests import few_util as fu
from tests.gpu_util import need_gpu, dev, dev_bf16, host_bits
from tests.test_gpu_fp4_ffn import MANY, _check, _segments, _weights

pytestmark = pytest.mark.gpu


def setup_module(module):
    need_gpu()
    assert ops.moe_device_check(0) == 0, "not a gfx950 device"


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_the_few_row_form_keeps_16_bits(fmt, case):
    """Many groups and long segments, too, within the bound of two bf16 numbers
    per element of the intermediate."""
    counts, H, I = MANY[case]
    rng = np.random.default_rng(200 + case)
    handle, v13, v2 = _weights(rng, fmt, len(counts), H, I)
    cu, cap = _segments(counts)
    x = fu.bf16(rng.standard_normal((cap, H)))
    y = ops.moe_grouped_ffn_fp4(dev_bf16(x), dev(cu), dev(np.array(counts, np.int32)), handle)
    _check(host_bits(y), x, cu, counts, v13, v2, None, fu.PAIR)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("few", [True, False])
def test_the_low_half_of_the_intermediate(fmt, few):
    """An intermediate whose bf16 rounding is all that the output shows: a[0] =
    silu(64) (1 + 2^-8), halfway between two bf16 numbers, minus a[1] = 64.  The
    few-row form gives 64 2^-8 (its silu's float32 steps, a few 2^-24 of 64, are
    within 2^-15 of that), the tile form 0 or 128 2^-8."""
    H, I = 128, 128
    counts = [3] if few else [20000]
    G, rows = len(counts), sum(counts)
    assert (ops.moe_grouped_ffn_fp4_workspace_bytes(rows, G, H, I) == (rows * I * 4 + 255) // 256 * 256) == few
    w13, w2 = np.zeros((G, 2 * I, H), np.float32), np.zeros((G, H, I), np.float32)
    w13[:, 0, 0] = w13[:, 1, 0] = 1.0                     # g = x[0]
    w13[:, I, 1] = w13[:, I, 2] = w13[:, I + 1, 1] = 1.0   # u[0] = x[1] + x[2], u[1] = x[1]
    w2[:, :, 0], w2[:, :, 1] = 1.0, -1.0
    handle = ops.ffn_weights(dev_bf16(fu.bf16(w13)), dev_bf16(fu.bf16(w2)), fmt)
    x = np.zeros((rows, H), np.float32)
    x[:, :3] = 64.0, 1.0, 2.0 ** -8
    cu, _ = _segments(counts)
    y = ops.moe_grouped_ffn_fp4(dev_bf16(fu.bf16(x)), dev(cu), dev(np.array(counts, np.int32)), handle).float()
    if few:
        assert ((y - 0.25).abs() <= 0.25 * 2.0 ** -8).all()
    else:
        assert torch.isin(y, torch.tensor([0.0, 0.5], device="cuda")).all()
