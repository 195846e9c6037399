"""The few-token layer and the FFN on 4-bit weights at the sizes of a large
model: 256 experts of H = 7168, I = 2048, and prompts of 32768 rows.  Weights are
random codes and scales made on the GPU, the reference float64 there, on the
experts and rows that are looked at; the bounds are those of few_util.py."""

import pytest
import torch

from combine_top_route_moe_amd import ops
from tests import few_util as fu
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def setup_module(module):
    need_gpu()
    assert ops.moe_device_check(0) == 0, "not a gfx950 device"


class Stack:
    """G matrices [N, K] as codes and scales; [g]: the stored values, float64."""

    def __init__(self, gen, fmt, G, N, K):
        self.fmt, self.g = fmt, None
        byte = lambda *shape, lo=0, hi=256: torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda",  # noqa: E731
                                                          generator=gen)
        rand = lambda *shape: torch.rand(shape, generator=gen, device="cuda")  # noqa: E731
        if fmt == "fp8":
            self.codes = byte(G, N, K)
            self.codes.bitwise_and_(0xF7)                       # up to 240, no NaN
            self.scales = rand(G, N // 128, K // 128) * 2e-3 + 1e-4
        else:
            self.codes = byte(G, N, K // 2)
            mx = fmt == "mxfp4"
            self.scales = byte(G, N, K // (32 if mx else 16), lo=118 if mx else 0x30, hi=122 if mx else 0x48)
            if not mx:
                self.g = rand(G) * 0.01 + 0.002

    def __getitem__(self, g):
        c, s = self.codes[g], self.scales[g]
        if self.fmt == "fp8":
            s = s.repeat_interleave(128, 0).repeat_interleave(128, 1)
            return (c.view(torch.float8_e4m3fn).float() * s).bfloat16().double()
        lut = torch.tensor([*fu.E2M1, *(-fu.E2M1)], dtype=torch.float32, device="cuda")
        v = torch.stack([lut[(c & 15).int()], lut[(c >> 4).int()]], -1).flatten(1)
        if self.fmt == "mxfp4":
            return v.double() * torch.exp2(s.double() - 127).repeat_interleave(32, 1)
        S = s.view(torch.float8_e4m3fn).float() * self.g[g]
        return (v * S.repeat_interleave(16, 1)).bfloat16().double()


def _weights(gen, fmt, G, H, I):
    a, b = Stack(gen, fmt, G, 2 * I, H), Stack(gen, fmt, G, H, I)
    return ops.ffn_weights_from_codes(fmt, a.codes, a.scales, b.codes, b.scales, a.g, b.g), a, b


def _expert(x, w13, w2, a_step):
    """fu.expert on the GPU."""
    I, H = w13.shape[0] // 2, w13.shape[1]
    g, u = x @ w13[:I].t(), x @ w13[I:].t()
    eg = H * fu.F32_SUM * (x.abs() @ w13[:I].abs().t())
    eu = H * fu.F32_SUM * (x.abs() @ w13[I:].abs().t())
    s = g * torch.sigmoid(g)
    a = s * u
    ea = 1.1 * eg * u.abs() + s.abs() * eu + 1.1 * eg * eu + a.abs() * (2.0 ** -18 + a_step)
    aw2 = w2.abs().t()
    return a @ w2.t(), ea @ aw2 + (I + 64) * fu.F32_SUM * ((a.abs() + ea) @ aw2)


def _close(got, ref, bound):
    """Element by element; and the whole result's error, where those bounds of
    long sums are loose (test_gpu_decode.py's model-sized layer: one rounding to
    bf16, and the float32 sums' share)."""
    assert ((got.double() - ref).abs() <= bound + fu.BF16_HALF * (ref.abs() + bound)).all()
    return float((got.double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4", "nvfp4"])
def test_a_large_layer(fmt):
    H, I, E, K = 7168, 2048, 256, 8
    gen = torch.Generator(device="cuda").manual_seed(5)
    handle, w13, w2 = _weights(gen, fmt, E, H, I)
    shared, s13, s2 = _weights(gen, fmt, 1, H, I)
    for T in (1, 3, 20):
        x = (torch.randn(T, H, generator=gen, device="cuda") * 0.1).bfloat16()
        logits = torch.randn(T, E, generator=gen, device="cuda")
        out, idx, w = ops.moe_decode(logits, x, K, handle, shared=shared)
        ref, bound = _expert(x.double(), s13[0], s2[0], fu.PAIR)
        mag = ref.abs()
        for e in sorted(set(idx.flatten().tolist())):
            t, k = torch.nonzero(idx == e, as_tuple=True)
            y, ey = _expert(x[t].double(), w13[e], w2[e], fu.PAIR)
            wt = w[t, k].double()[:, None]
            ref[t] += wt * y
            bound[t] += wt * ey
            mag[t] += (wt * y).abs()
        off = _close(out, ref, bound + (K + 4) * fu.F32_SUM * (mag + bound))
        assert off <= 2.0 ** -8 + 2.0 ** -12, (T, off)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_large_prompt(fmt):
    H, I, G, rows = 4096, 1536, 64, 32768
    gen = torch.Generator(device="cuda").manual_seed(6)
    handle, w13, w2 = _weights(gen, fmt, G, H, I)
    p = torch.exp(1.5 * torch.randn(G, generator=gen, device="cuda"))
    counts = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=gen), minlength=G)
    cu = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    x = (torch.randn(rows, H, generator=gen, device="cuda") * 0.1).bfloat16()
    scale = torch.rand(rows, generator=gen, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.moe_grouped_ffn_fp4(x, cu.int(), counts.int(), handle, scale, dev_error=err)
    assert int(err.item()) == 0
    order = counts.argsort().tolist()
    for g in {0, G - 1, order[0], order[G // 2], order[-1]}:
        # up to 400 rows, across tiles of 128 and the segment's end
        r = slice(max(int(cu[g]), int(cu[g + 1]) - 400), int(cu[g + 1]))
        s = scale[r].double()[:, None]
        ref, bound = _expert(x[r].double(), w13[g], w2[g], fu.SINGLE)
        if len(ref):
            _close(y[r], ref * s, bound * s)
