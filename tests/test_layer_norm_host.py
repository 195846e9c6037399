"""MoELayer behind its norm: which buffers the stages take and report, and what
is refused when.  No GPU needed: the buffers are host tensors, and the calls
that would launch kernels are stood in for."""

from contextlib import nullcontext
from types import SimpleNamespace

import pytest
import torch

from combine_top_route_moe_amd import MoELayer, ops

T, H, E, K, I, SI = 40, 256, 4, 2, 128, 256


@pytest.fixture
def calls(monkeypatch):
    """The names of the calls that the layer makes, in order."""
    made = []
    for name in ("moe_route", "moe_permute", "moe_quant_rows_fp8", "moe_fake_quant_rows", "moe_combine",
                 "moe_rmsnorm"):
        monkeypatch.setattr(ops, name, lambda *a, _name=name, **kw: made.append(_name))
    monkeypatch.setattr(MoELayer, "_ffn", lambda *a, **kw: made.append("ffn"))
    fields = ("format", "num_groups", "H", "I", "w13", "w2", "w13_scales", "w2_scales", "w13_tensor_scale",
              "w2_tensor_scale")
    monkeypatch.setattr(ops, "FFNWeights", lambda *a: SimpleNamespace(**dict(zip(fields, a))))
    monkeypatch.setattr(ops, "_one_device", lambda *a: 0)
    monkeypatch.setattr(ops, "moe_pack_ffn_weights", lambda a, b: (a, b))
    monkeypatch.setattr(ops, "moe_pack_ffn_weights_fp8", lambda a, b, k128=False: (a, a, b, b))
    side = SimpleNamespace(wait_stream=lambda s: None, cuda_stream=0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    monkeypatch.setattr(torch.cuda, "Stream", lambda device=None: side)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: side)
    return made


def _layer(fp8=False, shared=True, **kw):
    layer = MoELayer(T, H, E, K, I, device="cpu", shared_I=SI if shared else 0, **kw)
    _set(layer, fp8)
    return layer


def _set(layer, fp8=False):
    bf = dict(dtype=torch.bfloat16)
    w = [torch.zeros(E, 2 * I, H, **bf), torch.zeros(E, H, I, **bf)]
    if layer.shared_I:
        w += [torch.zeros(2 * SI, H, **bf), torch.zeros(H, SI, **bf)]
    layer.set_weights(*w, fp8=fp8)


X, W, LOGITS = torch.zeros(T, H, dtype=torch.bfloat16), torch.ones(H), torch.zeros(T, E)


def test_stage_outputs_names_the_codes_that_the_forward_ran_on(calls):
    layer = _layer("w8a8")
    codes = lambda: [layer.stage_outputs()[k].data_ptr() for k in ("hidden_codes", "hidden_scales")]  # noqa: E731
    layer.norm(X, W)
    layer.forward(LOGITS, None)
    normed = [layer.normed_q.data_ptr(), layer.normed_s.data_ptr()]
    assert codes() == normed
    layer.forward(LOGITS, X)
    assert codes() == [layer.hq.data_ptr(), layer.hs.data_ptr()]
    layer.norm(X, W)                                                # a norm alone changes nothing
    assert codes() == [layer.hq.data_ptr(), layer.hs.data_ptr()]
    for _, enqueue in layer.stages(LOGITS, None):
        enqueue()
    assert codes() == normed
    _set(layer)
    layer.forward(LOGITS, None)
    assert "hidden_codes" not in layer.stage_outputs()
    _set(layer, "w8a8")
    assert codes() == [layer.hq.data_ptr(), layer.hs.data_ptr()]    # new buffers


@pytest.mark.parametrize("fp8", [False, "w8a8"])
@pytest.mark.parametrize("overlap", [False, True])
def test_a_list_of_stages_does_not_run_on_other_rows_than_it_was_made_for(calls, fp8, overlap):
    """What norm() wrote is looked at when a stage reads it, not only when the list is made."""
    layer = _layer(fp8)
    layer.norm(X, W)
    stages = dict(layer.stages(LOGITS, None, overlap_shared=overlap))
    layer.norm(X[:5], W)                                            # a few tokens, for decode()
    calls.clear()
    for name in ("permute", "shared_ffn"):
        with pytest.raises(ValueError, match="all of the layer's rows"):
            stages[name]()
    assert not calls
    layer.norm(X, W)
    for enqueue in stages.values():
        enqueue()
    assert calls.count("moe_permute") == 1 and calls.count("ffn") == 3


def test_a_list_of_stages_on_codes_does_not_run_on_rows_without(calls):
    layer = _layer("w8a8")
    layer.norm(X, W)
    stages = dict(layer.stages(LOGITS, None))
    layer.w8a8 = False                                              # (as other weights leave it)
    layer.norm(X, W)
    with pytest.raises(ValueError, match="call it again"):
        stages["permute"]()


def test_a_list_of_stages_on_given_rows_does_not_look_at_the_norm(calls):
    layer = _layer(dispatch_fp4="mxfp4")
    layer.norm(X[:5], W)
    for _, enqueue in layer.stages(LOGITS, X):
        enqueue()
    with pytest.raises(ValueError, match="all of the layer's rows"):
        layer.stages(LOGITS, None)
    layer.norm(X, W)
    stages = dict(layer.stages(LOGITS, None))
    layer.norm(X[:5], W)
    with pytest.raises(ValueError, match="all of the layer's rows"):
        stages["dispatch_qdq"]()
