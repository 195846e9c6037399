"""MoELayer.decode's workspace, allocated at its first call."""

import numpy as np
import pytest
import torch

from combine_top_route_moe_amd import MoELayer, ops
from tests import few_util as fu
from tests.gpu_util import need_gpu, dev, dev_bf16

pytestmark = pytest.mark.gpu


def setup_module(module):
    need_gpu()
    assert ops.moe_device_check(0) == 0, "not a gfx950 device"


def test_a_first_call_that_is_captured():
    """The workspace then comes out of the graph's memory: replays, eager calls
    between them and after the graph is gone give a warmed-up layer's bits."""
    T, H, E, K, I = 50, 512, 16, 4, 256
    rng = np.random.default_rng(2)
    w13, w2 = (dev_bf16(m) for m in fu.make_weights(rng, E, H, I))
    layers = [MoELayer(T, H, E, K, I) for _ in range(2)]
    for layer in layers:
        layer.set_weights(w13, w2, fp4="mxfp4")
    ins = [(dev(rng.standard_normal((n, E)).astype(np.float32)), dev_bf16(fu.bf16(rng.standard_normal((n, H)))))
           for n in (30, 30, 50)]
    want = [layers[1].decode(*i).clone() for i in ins]
    logits, x = (t.clone() for t in ins[0])
    layer, graph = layers[0], torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.decode(logits, x)
    for i in (0, 1, 0, 1):
        logits.copy_(ins[i][0])
        x.copy_(ins[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out[:30], want[i])
        assert torch.equal(layer.decode(*ins[2]), want[2])
    del graph
    torch.cuda.empty_cache()
    other = [torch.full((1 << 22,), 3, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert torch.equal(layer.decode(*ins[2]), want[2])
    assert all((t == 3).all() for t in other)
