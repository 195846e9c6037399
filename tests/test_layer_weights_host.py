"""MoELayer's buffers as its weights change kind.  No GPU needed: the buffers
are host tensors, and the packing calls are stood in for."""

from contextlib import nullcontext
from types import SimpleNamespace

import pytest
import torch

from combine_top_route_moe_amd import MoELayer, ops

T, H, E, K, I, SI = 40, 256, 4, 2, 128, 256


@pytest.fixture
def layer(monkeypatch):
    fields = ("format", "num_groups", "H", "I", "w13", "w2", "w13_scales", "w2_scales", "w13_tensor_scale",
              "w2_tensor_scale")
    monkeypatch.setattr(ops, "FFNWeights", lambda *a: SimpleNamespace(**dict(zip(fields, a))))
    monkeypatch.setattr(ops, "_one_device", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    monkeypatch.setattr(torch.cuda, "Stream", lambda device=None: None)
    monkeypatch.setattr(ops, "moe_pack_ffn_weights", lambda a, b: (a, b))
    monkeypatch.setattr(ops, "moe_pack_ffn_weights_fp8", lambda a, b, k128=False: (a, a, b, b))
    monkeypatch.setattr(ops, "moe_pack_ffn_weights_fp4", lambda a, b, *rest: (a, a, None, b, b, None))
    return MoELayer(T, H, E, K, I, device="cpu", shared_I=SI)


def _weights():
    bf = dict(dtype=torch.bfloat16)
    return (torch.zeros(E, 2 * I, H, **bf), torch.zeros(E, H, I, **bf), torch.zeros(2 * SI, H, **bf),
            torch.zeros(H, SI, **bf))


@pytest.mark.parametrize("kw", [dict(), dict(pack=False), dict(fp8=True), dict(fp4="mxfp4"), dict(fp4="nvfp4")],
                         ids=lambda kw: "-".join(f"{k}={v}" for k, v in kw.items()) or "bf16")
def test_rows_are_whole_again_after_the_fp8_path(layer, kw):
    """"w8a8" moves the rows' codes, half the bytes of bf16 rows: with any
    other weights after it the permute must find buffers for whole rows, and
    the FFN its workspace."""
    layer.set_weights(*_weights(), fp8="w8a8")
    assert layer.perm.x_perm.shape == (layer.capacity, H // 2)
    layer.set_weights(*_weights(), **kw)
    assert not layer.w8a8
    assert layer.perm.x_perm.shape == (layer.capacity, H)
    size = ops.moe_grouped_ffn_fp4_workspace_bytes if "fp4" in kw else ops.moe_grouped_ffn_workspace_bytes
    assert layer.ffn_ws.numel() >= size(layer.capacity, E, H, I)
    assert layer.shared_ws.numel() >= size(T, 1, H, SI)


def test_decodes_workspace_is_of_its_first_call(layer, monkeypatch):
    """A layer that only runs prompts, or cannot decode, holds no workspace for
    decode(); one that does allocates it once, for its largest batch."""
    used = []
    monkeypatch.setattr(ops, "moe_decode", lambda *a, workspace, **kw: used.append(workspace))
    size = ops.moe_decode_workspace_bytes(T, H, I, K, E, SI)
    held = lambda: [n for n, t in vars(layer).items()  # noqa: E731
                    if torch.is_tensor(t) and t.dtype == torch.uint8 and n.startswith("decode")]
    assert not held()
    layer.set_weights(*_weights())
    assert not held()
    for n in (1, T, 7):
        layer.decode(torch.zeros(n, E), torch.zeros(n, H, dtype=torch.bfloat16))
    assert used[0] is used[1] is used[2] and used[0].numel() >= size


@pytest.mark.parametrize("kw", [dict(), dict(fp8=True), dict(fp8="w8a8"), dict(pack=False)],
                         ids=["bf16", "fp8", "w8a8", "rows"])
def test_weights_on_another_device_are_taken(layer, monkeypatch, kw):
    """These kinds of weights are packed on the current device's stream wherever
    they lie; only calls that were never made so refuse it."""
    def refuse(*a):
        raise ValueError("another device is current")

    monkeypatch.setattr(ops, "_one_device", refuse)
    layer.set_weights(*_weights(), **kw)
    with pytest.raises(ValueError, match="another device"):
        layer.set_weights(*_weights(), fp4="mxfp4")


def test_packed_weights_lie_where_the_layer_does(layer):
    bf = dict(dtype=torch.bfloat16, device="meta")
    w = ops._packed(torch.zeros(E, 2 * I, H, **bf), torch.zeros(E, H, I, **bf), "bf16")
    with pytest.raises(ValueError, match="weights on meta"):
        layer.set_packed_weights(w)
