"""moe_rmsnorm_backward on more rows than one launch takes: every width of a row, with and
without the stream's own gradient (whose rows are loaded ahead or not) and for both types
of gain; in place, captured and again."""

import pytest
import torch

from combine_top_route_moe_amd import ops
from tests.around_util import U, gen, within
from tests.test_gpu_norm import EPS, _gradient64, _inputs

pytestmark = pytest.mark.gpu

# one wave a row to 2048 channels (one, two, four vectors a thread), four to 8192 (two, four), sixteen beyond
SHAPES = [(1500, 384), (1030, 640), (2000, 1024), (1300, 1536), (1100, 2048), (1500, 2176), (1600, 4096), (1027, 4224),
          (1300, 7168), (1025, 8192), (1026, 8320), (1100, 20480)]


def _case(T, H, residual, f32):
    x, dh, w = _inputs(T, H, f32=f32)
    dy = torch.randn(T, H, generator=gen(9)).bfloat16()
    r = (1 / torch.sqrt(x.double().square().mean(1) + EPS)).float()
    return dy, x, r, w, dh if residual else None


def check(dx, dw, dy, x, r, w, dh):
    want, bound, want_w, size = _gradient64(dy, x, r, w, dh)
    within(dx, want, bound, "dx")
    # at most 8 rows of a thread one after another, four waves, 512 / 32 shares in a thread and
    # its wave's eight and the four waves; three roundings of a term (up to 64 rows: two of a
    # thread, 32 threads or more of one row)
    within(dw, want_w, (8 + 3 + 16 + 3 + 3 + 3) * U * size + 2.0 ** -140, "dw")


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_backward(T, H, residual, f32):
    case = _case(T, H, residual, f32)
    dy, x, r, w, dh = (None if t is None else t.cuda() for t in case)
    check(*ops.moe_rmsnorm_backward(dy, x, r, w, d_residual=dh), *case)


@pytest.mark.parametrize("where", ["dy", "d_residual"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H", [(9, 1024), (40, 7168), (1600, 1024), (1600, 4096), (1300, 7168), (1026, 8320)])
def test_in_place(where, f32, T, H):
    case = _case(T, H, True, f32)
    dy, x, r, w, dh = (t.cuda() for t in case)
    dx, dw = ops.moe_rmsnorm_backward(dy, x, r, w, d_residual=dh, dx=dy if where == "dy" else dh)
    assert dx.data_ptr() == (dy if where == "dy" else dh).data_ptr()
    check(dx, dw, *case)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", [(2000, 1024), (1600, 4096), (1300, 7168), (1026, 8320)])
def test_equal_bits_captured_and_again(T, H, residual):
    """Two launches, whose workspace takes the first one's shares."""
    case = _case(T, H, residual, False)
    dy, x, r, w, dh = (None if t is None else t.cuda() for t in case)
    need = ops.moe_rmsnorm_backward_workspace_bytes(T, H)
    work = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")

    def call():
        ops.moe_rmsnorm_backward(dy, x, r, w, d_residual=dh, dx=dx, d_weight=dw, workspace=work[:need])

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        dy.copy_(torch.randn(T, H, generator=gen(50 + k)).bfloat16())
        work[:need].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        again = ops.moe_rmsnorm_backward(dy, x, r, w, d_residual=dh)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
        check(dx, dw, dy.cpu(), *case[1:])
    assert (work[need:] == 255).all()
