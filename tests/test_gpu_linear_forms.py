"""Every form of moe_linear_fp8 against the product in 64 bits: each tile, K in parts, the
workspace that the parts go through."""

import pytest
import torch

from combine_top_route_moe_amd import ops
from tests.linear_forms import FORMS, PARTS
from tests.test_gpu_linear_fp8 import _case, check

pytestmark = pytest.mark.gpu
SOME = [f for f in PARTS if f[0] * f[1] * f[2] < 4e9]


@pytest.mark.parametrize("M,N,K,tile,parts", FORMS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_product(M, N, K, tile, parts, out):
    assert ops.moe_linear_fp8_parts(M, N, K) == (parts, tile)
    xq, xs, wq, ws = _case(M, N, K)
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    y = torch.full((M + 1, N), 7.0, dtype=out, device="cuda")
    check(ops.moe_linear_fp8(xq.cuda(), xs.cuda(), weights, y=y[:M]), xq, xs, wq, ws)
    assert (y[M] == 7).all()


@pytest.mark.parametrize("M,N,K,tile,parts", SOME)
def test_what_is_in_the_workspace_and_past_it(M, N, K, tile, parts):
    """What a workspace holds does not count, and of one that is larger the rest stays."""
    xq, xs, wq, ws = (t.cuda() for t in _case(M, N, K))
    weights = ops.linear_weights_from_codes(wq, ws)
    first = ops.moe_linear_fp8(xq, xs, weights)
    need = 4 * parts * M * N
    work = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(ops.moe_linear_fp8(xq, xs, weights, workspace=work[:need]), first)
    assert (work[need:] == 255).all()
    with pytest.raises(RuntimeError):
        ops.moe_linear_fp8(xq, xs, weights, workspace=work[: need - 1])


@pytest.mark.parametrize("M,N,K,tile,parts", SOME)
def test_equal_bits_on_any_stream_and_in_a_graph(M, N, K, tile, parts):
    xq, xs, wq, ws = (t.cuda() for t in _case(M, N, K))
    weights = ops.linear_weights_from_codes(wq, ws)
    first = ops.moe_linear_fp8(xq, xs, weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = ops.moe_linear_fp8(xq, xs, weights, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    work = torch.empty(ops.moe_linear_fp8_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_linear_fp8(xq, xs, weights, y=y, workspace=work)
    for k in range(3):
        xq.copy_(_case(M, N, K, seed=30 + k)[0])
        work.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ops.moe_linear_fp8(xq, xs, weights))


def test_products_in_parts_at_once():
    """Two streams, a workspace each (from each stream's own pool)."""
    M, N, K = 64, 4096, 7168
    assert ops.moe_linear_fp8_parts(M, N, K)[0] > 1
    dev = [[t.cuda() for t in _case(M, N, K, seed)] for seed in (1, 2)]
    packed = [ops.linear_weights_from_codes(c[2], c[3]) for c in dev]
    want = [ops.moe_linear_fp8(c[0], c[1], w) for c, w in zip(dev, packed)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [[ops.moe_linear_fp8(c[0], c[1], w, stream=s) for c, w, s in zip(dev, packed, streams)] for _ in range(10)]
        torch.cuda.synchronize()
        for pair in outs:
            assert all(torch.equal(a, b) for a, b in zip(pair, want))
