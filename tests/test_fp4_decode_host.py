"""Refusals of moe_pack_ffn_weights_fp4, moe_grouped_ffn_fp4 and moe_decode,
and their size queries: everything the host can see is answered before any
device work (no GPU needed; the pointers are never read)."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from combine_top_route_moe_amd import _lib, ops
from tests import few_util as fu

P = 1 << 20            # a 16-byte aligned address, never read
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _weights(fmt=ops.MOE_W_MXFP4, **kw):
    f = dict(w13=P, w13_scales=P, w13_tensor_scale=P, w2=P, w2_scales=P, w2_tensor_scale=P)
    f.update(kw)
    return _lib.FFNWeightsStruct(fmt, f["w13"], f["w13_scales"], f["w13_tensor_scale"], f["w2"],
                                 f["w2_scales"], f["w2_tensor_scale"])


def _pack(lib, **kw):
    a = dict(w13=P, w2=P, G=2, H=256, I=128, mode=ops.MOE_FQ_MXFP4, g13=None, g2=None, q13=P, s13=P, q2=P, s2=P)
    a.update(kw)
    return lib.moe_pack_ffn_weights_fp4(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(G=0), INVALID), (dict(H=0), INVALID), (dict(I=-128), INVALID),
    (dict(H=200), UNSUPPORTED), (dict(I=64), UNSUPPORTED),
    (dict(mode=ops.MOE_FQ_BLOCK), INVALID), (dict(mode=9), INVALID),
    (dict(q13=None), INVALID), (dict(s2=None), INVALID), (dict(w2=None), INVALID),
    (dict(w13=P + 2), INVALID), (dict(s13=P + 8), INVALID),
    (dict(mode=ops.MOE_FQ_NVFP4), INVALID), (dict(mode=ops.MOE_FQ_NVFP4, g13=P), INVALID),
])
def test_pack_refusals(lib, kw, status):
    assert _pack(lib, **kw) == status


def _ffn(lib, weights="mx", **kw):
    w = _weights() if weights == "mx" else weights
    a = dict(x=P, cu=P, n=P, G=2, H=256, I=128, w=ctypes.addressof(w) if w is not None else None, scale=None, y=P,
             cap=4, flags=3, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    return lib.moe_grouped_ffn_fp4(*a.values(), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(G=0), INVALID), (dict(cap=-1), INVALID), (dict(flags=0), INVALID),
    (dict(flags=3 | ops.MOE_FFN_PACKED_WEIGHTS), INVALID), (dict(H=100), UNSUPPORTED),
    (dict(G=1025), UNSUPPORTED), (dict(cap=1 << 31), UNSUPPORTED), (dict(w=None), INVALID),
    (dict(cu=None), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(x=P + 4), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=P + 8), WORKSPACE),
    (dict(ws_bytes=16), WORKSPACE), (dict(cap=0, x=None, y=None, ws=None), OK),
])
def test_ffn_refusals(lib, kw, status):
    assert _ffn(lib, **kw) == status


@pytest.mark.parametrize("weights", [
    _weights(ops.MOE_W_BF16), _weights(ops.MOE_W_FP8), _weights(7), _weights(w13=None), _weights(w2_scales=None),
    _weights(w13=P + 8), _weights(ops.MOE_W_NVFP4, w13_tensor_scale=None)])
def test_ffn_refuses_other_weights(lib, weights):
    assert _ffn(lib, weights) == INVALID


def test_ffn_stage_needs_only_its_own_pointers(lib):
    # the workspace check comes after the pointer checks: reaching it shows they passed
    gate = _weights(w2=None, w2_scales=None)
    assert _ffn(lib, gate, flags=ops.MOE_FFN_GATE_UP, y=None, ws=None) == WORKSPACE
    down = _weights(w13=None, w13_scales=None)
    assert _ffn(lib, down, flags=ops.MOE_FFN_DOWN, x=None, ws=None) == WORKSPACE
    assert _ffn(lib, down, flags=ops.MOE_FFN_GATE_UP, ws=None) == INVALID


def _decode(lib, w=None, s=None, **kw):
    w = _weights(ops.MOE_W_BF16) if w is None else w
    routed = kw.pop("routed", ctypes.addressof(w))
    a = dict(logits=P, valid=None, x=P, T=4, H=256, I=128, E=8, K=2, begin=0, El=8, flags=1, idx=P, tw=P,
             w=routed, s=None if s is None else ctypes.addressof(s), sI=0, out=P + 4096, ws=P,
             ws_bytes=1 << 30)
    a.update(kw)
    return lib.moe_decode(*a.values(), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(T=65), UNSUPPORTED), (dict(K=9), INVALID), (dict(K=0), INVALID),
    (dict(E=64, K=33, El=1), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(begin=-1), INVALID),
    (dict(begin=1), INVALID), (dict(begin=2 ** 31 - 1, El=2), INVALID), (dict(El=0), INVALID),
    (dict(flags=2), INVALID), (dict(sI=128), INVALID), (dict(H=192), UNSUPPORTED), (dict(I=64), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(idx=None), INVALID), (dict(tw=None), INVALID), (dict(out=None), INVALID),
    (dict(routed=None), INVALID), (dict(x=P + 2), INVALID), (dict(out=P), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=256), WORKSPACE), (dict(ws=P + 4), WORKSPACE), (dict(T=0, x=None, out=None, ws=None), OK),
])
def test_decode_refusals(lib, kw, status):
    assert _decode(lib, **kw) == status


def test_decode_refuses_mismatched_weights(lib):
    assert _decode(lib, s=_weights(ops.MOE_W_FP8), sI=128) == INVALID        # another format than the routed
    assert _decode(lib, s=_weights(ops.MOE_W_BF16), sI=0) == INVALID
    assert _decode(lib, s=_weights(ops.MOE_W_BF16), sI=100) == UNSUPPORTED
    assert _decode(lib, _weights(ops.MOE_W_BF16, w2=None)) == INVALID
    assert _decode(lib, _weights(ops.MOE_W_FP8, w13_scales=None)) == INVALID
    assert _decode(lib, _weights(ops.MOE_W_NVFP4, w2_tensor_scale=None)) == INVALID
    assert _decode(lib, _weights(4)) == INVALID


def test_matrices_past_32_bit_offsets_are_refused(lib):
    """An expert's w13 in 4 GiB or more, or a dimension past 2^20; the largest
    below reach the workspace check."""
    for fmt, bits in ((ops.MOE_W_BF16, 16), (ops.MOE_W_FP8, 8), (ops.MOE_W_MXFP4, 4), (ops.MOE_W_NVFP4, 4)):
        w, H = _weights(fmt), 1 << 15
        I = (1 << 32) * 8 // bits // 2 // H                  # w13: 2^32 bytes
        for h, i, status in ((H, I, UNSUPPORTED), (H, I - 128, WORKSPACE), (1 << 20, 128, WORKSPACE),
                             ((1 << 20) + 128, 128, UNSUPPORTED), (128, (1 << 20) + 128, UNSUPPORTED)):
            assert _decode(lib, w, H=h, I=i, ws=None) == status, (fmt, h, i)
            if fmt in (ops.MOE_W_MXFP4, ops.MOE_W_NVFP4):
                assert _ffn(lib, w, H=h, I=i, ws=None) == status, (fmt, h, i)
        assert _decode(lib, w, s=w, H=H, sI=I, ws=None) == UNSUPPORTED


def test_launches_past_the_grid_are_refused(lib):
    big = dict(I=1 << 20, H=128, ws_bytes=1 << 60)
    assert _decode(lib, T=64, E=1024, K=32, El=1024, **big) == UNSUPPORTED
    assert _ffn(lib, cap=(1 << 31) - 1, G=1024, **big) == UNSUPPORTED
    assert _pack(lib, G=1 << 20, H=1 << 15, I=1 << 15) == UNSUPPORTED


def test_handles_do_not_change():
    q = torch.zeros(2, 256, 128, dtype=torch.uint8)
    for name in ("w13", "format", "H"):
        with pytest.raises(AttributeError):
            setattr(ops.FFNWeights.__new__(ops.FFNWeights), name, q)


def test_size_queries(lib):
    need = ops.moe_decode_workspace_bytes(64, 7168, 2048, 8, 256, 2048)
    assert need >= 64 * 9 * 2048 * 4
    assert ops.moe_decode_workspace_bytes(-1, 128, 128, 1, 1, 0) == 0
    need = ops.moe_decode_workspace_bytes(64, 7168, 2048, 8, 256)
    assert _decode(lib, T=64, H=7168, I=2048, E=256, K=8, El=256, ws_bytes=need - 1) == WORKSPACE
    assert ops.moe_grouped_ffn_fp4_workspace_bytes(1000, 4, 256, 128) >= 1000 * 128 * 2
    assert ops.moe_grouped_ffn_fp4_workspace_bytes(7, 4, 256, 128) >= 7 * 128 * 4
    assert ops.moe_grouped_ffn_fp4_workspace_bytes(0, 4, 256, 128) == 0
    for G, H, I in ((1, 128, 128), (4, 4096, 1536), (64, 2048, 1024), (1000, 256, 128)):   # one buffer for all batches
        sizes = [ops.moe_grouped_ffn_fp4_workspace_bytes(n, G, H, I)
                 for n in range(0, 140 * min(G, 64), 7 if G < 64 else 61)]
        assert sizes == sorted(sizes), (G, H, I)


def test_handles_check_their_tensors():
    q = torch.zeros(2, 256, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ops.FFNWeights(9, 2, 256, 128, q, q)
    with pytest.raises(ValueError):
        ops.FFNWeights(ops.MOE_W_MXFP4, 2, 256, 128, q, torch.zeros(2, 256, 64, dtype=torch.uint8))
    with pytest.raises(TypeError):
        ops.FFNWeights(ops.MOE_W_BF16, 2, 128, 128, q, q)
    with pytest.raises(ValueError):      # host tensors
        ops.FFNWeights(ops.MOE_W_BF16, 2, 128, 128, torch.zeros(2, 256, 128, dtype=torch.bfloat16),
                       torch.zeros(2, 128, 128, dtype=torch.bfloat16))
    w13, w2 = torch.zeros(2, 256, 128, dtype=torch.bfloat16), torch.zeros(2, 128, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.ffn_weights(w13, w2, "int4")
    with pytest.raises(ValueError):
        ops.ffn_weights(w13, w2[:1], "bf16")
    with pytest.raises(TypeError):
        ops.ffn_weights(w13.float(), w2, "bf16")
    with pytest.raises(ValueError):
        ops.moe_pack_ffn_weights_fp4(w13, w2, mode=ops.MOE_FQ_BLOCK)
    with pytest.raises(ValueError, match="device tensor"):
        ops.moe_pack_ffn_weights_fp4(w13, w2)


def test_fast_fake_quantizers_are_the_oracles():
    rng = np.random.default_rng(0)
    w = rng.standard_normal((64, 256)).astype(np.float32) * 0.1
    w[0, :32], w[1, :32], w[2] = 0.0, -0.0, w[2] * 2.0 ** -110
    w[3, :16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0.5]
    bits = fu.bf16(w)
    np.testing.assert_array_equal(fu.fake_quant(bits, "mxfp4"), oracle.fake_quant_mxfp4(bits)[0])
    g = fu.tensor_scale(bits)
    np.testing.assert_array_equal(fu.fake_quant(bits, "nvfp4"), oracle.fake_quant_nvfp4(bits, g)[0])
    np.testing.assert_array_equal(fu.fake_quant(bits, "nvfp4", 1e-3), oracle.fake_quant_nvfp4(bits, 1e-3)[0])
