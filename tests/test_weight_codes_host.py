"""Refusals of moe_pack_ffn_codes: answered on the host before any device work
(the pointers are never read)."""

import ctypes

import pytest
import torch

from combine_top_route_moe_amd import _lib, ops

P = 1 << 20            # a 16-byte aligned address, never read
INVALID, UNSUPPORTED = -1, -2


def _pack(fmt=ops.MOE_W_MXFP4, w13=P, s13=P, w2=P, s2=P, G=2, H=256, I=128, q13=P, o13=P, q2=P, o2=P, rows=True):
    w = _lib.FFNWeightsStruct(fmt, w13, s13, None, w2, s2, None)
    return _lib.load().moe_pack_ffn_codes(ctypes.addressof(w) if rows else None, G, H, I, q13, o13, q2, o2, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=False), INVALID), (dict(G=0), INVALID), (dict(H=0), INVALID), (dict(I=-128), INVALID),
    (dict(fmt=ops.MOE_W_BF16), INVALID), (dict(fmt=7), INVALID),
    (dict(H=200), UNSUPPORTED), (dict(I=64), UNSUPPORTED), (dict(H=(1 << 20) + 128), UNSUPPORTED),
    (dict(q13=None), INVALID), (dict(w13=None), INVALID), (dict(s13=None), INVALID), (dict(o2=None), INVALID),
    (dict(w13=P + 4), INVALID), (dict(q2=P + 8), INVALID), (dict(s2=P + 8), INVALID), (dict(o13=P + 4), INVALID),
    (dict(w13=None, q13=None, o13=None), INVALID), (dict(fmt=ops.MOE_W_FP8, q2=None), INVALID),
    (dict(fmt=ops.MOE_W_FP8, w2=P + 8), INVALID), (dict(G=1 << 20, H=1 << 15, I=1 << 15), UNSUPPORTED),
    (dict(G=(1 << 31) - 1, H=1 << 20, I=1 << 20), UNSUPPORTED),
])
def test_pack_codes_refusals(kw, status):
    assert _pack(**kw) == status


def test_codes_on_the_host_are_refused():
    q, q2 = torch.zeros(2, 256, 256, dtype=torch.uint8), torch.zeros(2, 256, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        ops.ffn_weights_from_codes("fp8", q, torch.zeros(2, 2, 2), q2, torch.zeros(2, 2, 1))
