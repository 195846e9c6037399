"""Expert weights handed over as codes and scales (ffn_weights_from_codes,
MoELayer.set_packed_weights): the packed order bit for bit that of the packing
calls, and the products on exactly the stored values, whatever scales a
checkpoint was written with."""

import numpy as np
import pytest
import torch

import oracle
from combine_top_route_moe_amd import MoELayer, ops
from oracle.numerics import bf16_bits_to_f32, bf16_bits_to_f64, e4m3fn_round
from tests import few_util as fu
from tests.gpu_util import need_gpu, dev, dev_bf16, host, host_bits

pytestmark = pytest.mark.gpu


def setup_module(module):
    need_gpu()
    assert ops.moe_device_check(0) == 0, "not a gfx950 device"


def _e4m3(values) -> torch.Tensor:
    """E4M3 codes of values that are E4M3 numbers."""
    t = torch.from_numpy(np.asarray(values, np.float32)).to(torch.float8_e4m3fn)
    assert np.array_equal(t.float().numpy(), values)
    return t.cuda()


def _fp8_checkpoint(w_bits):
    """(codes, scales, bf16 bits of the stored values) of a stack, its scales
    amax times the rounded reciprocal of 448: up to one float32 step from the
    quotient that the packing call takes."""
    q, s, v = [], [], []
    for w in w_bits:
        N, K = w.shape
        x = bf16_bits_to_f32(w).reshape(N // 128, 128, K // 128, 128)
        sg = (np.abs(x).max(axis=(1, 3)) * np.float32(1 / 448)).astype(np.float32)
        sb = sg[:, None, :, None]
        qg = e4m3fn_round(np.clip((x / sb).astype(np.float32), -448, 448)).astype(np.float32)
        q.append(qg.reshape(N, K))
        s.append(sg)
        v.append(fu.bf16(qg * sb).reshape(N, K))
    return np.stack(q), np.stack(s), np.stack(v)


def _fp4_checkpoint(rng, nv, G, N, K):
    """Codes (row-major, [G, N, K]), scale bytes, tensor scales and stored
    values that no quantizer need have written: any code, any scale."""
    codes = rng.integers(0, 16, (G, N, K)).astype(np.uint8)
    if nv:
        codes[:, ::3] &= 0xB                   # rows whose largest code is 3 (1.5)
        sb = rng.integers(0x20, 0x58, (G, N, K // 16)).astype(np.uint8)
        g = (rng.random(G) * 0.02 + 0.01).astype(np.float32)
    else:
        sb = rng.integers(119, 125, (G, N, K // 32)).astype(np.uint8)
        g = None
    return codes, sb, g, fu.fp4_values(codes, sb, nv, g)


def _nibbles(codes):
    return codes[..., 0::2] | codes[..., 1::2] << 4


def _handle(fmt, rng, G, H, I):
    """A checkpoint's handle and the bf16 bits of the values it stores."""
    if fmt == "fp8":
        (q13, s13, v13), (q2, s2, v2) = (_fp8_checkpoint(w) for w in fu.make_weights(rng, G, H, I))
        return ops.ffn_weights_from_codes("fp8", _e4m3(q13), dev(s13), _e4m3(q2), dev(s2)), v13, v2
    nv = fmt == "nvfp4"
    c13, s13, g13, v13 = _fp4_checkpoint(rng, nv, G, 2 * I, H)
    c2, s2, g2, v2 = _fp4_checkpoint(rng, nv, G, H, I)
    tensor = (dev(g13), dev(g2)) if nv else ()
    return ops.ffn_weights_from_codes(fmt, dev(_nibbles(c13)), dev(s13), dev(_nibbles(c2)), dev(s2),
                                      *tensor), v13, v2


@pytest.mark.parametrize("G,H,I", [(1, 128, 128), (3, 256, 384), (2, 640, 128)])
def test_fp8_order_is_the_packing_calls(G, H, I):
    w13, w2 = fu.make_weights(np.random.default_rng(G), G, H, I)
    want = ops.ffn_weights(dev_bf16(w13), dev_bf16(w2), "fp8")
    (q13, s13), (q2, s2) = (map(np.stack, zip(*[oracle.quantize_weight_blocks(m)[:2] for m in w])) for w in (w13, w2))
    q13, q2 = _e4m3(q13), _e4m3(q2)
    for a, b in ((q13, q2), (q13.view(torch.uint8), q2.view(torch.uint8))):
        got = ops.ffn_weights_from_codes("fp8", a, dev(s13), b, dev(s2))
        assert torch.equal(got.w13_scales, want.w13_scales) and torch.equal(got.w2_scales, want.w2_scales)
        # (a zero code's sign is not in the oracle's values)
        for x, y in ((got.w13, want.w13), (got.w2, want.w2)):
            assert torch.equal(x, y) or torch.equal(x.view(torch.float8_e4m3fn).float(),
                                                    y.view(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("G,H,I", [(1, 128, 128), (3, 256, 384), (2, 640, 128)])
def test_fp4_order_is_the_packing_calls(fmt, G, H, I):
    nv = fmt == "nvfp4"
    w13, w2 = fu.make_weights(np.random.default_rng(G), G, H, I)
    want = ops.ffn_weights(dev_bf16(w13), dev_bf16(w2), fmt)
    c13, s13 = fu.unpack_fp4(host(want.w13), host(want.w13_scales), nv, True)
    c2, s2 = fu.unpack_fp4(host(want.w2), host(want.w2_scales), nv, False)
    kind = torch.float8_e4m3fn if nv else torch.float8_e8m0fnu
    for cast in (lambda t: t, lambda t: t.view(kind)):
        got = ops.ffn_weights_from_codes(fmt, dev(_nibbles(c13)), cast(dev(s13)), dev(_nibbles(c2)), cast(dev(s2)),
                                         want.w13_tensor_scale, want.w2_tensor_scale)
        for n in ("w13", "w13_scales", "w2", "w2_scales"):
            assert torch.equal(getattr(got, n), getattr(want, n)), n
    # and row-major codes come back out of the packed order as they went in
    rng = np.random.default_rng(9)
    codes, sb, g, _ = _fp4_checkpoint(rng, nv, G, 2 * I, H)
    codes2, sb2, g2, _ = _fp4_checkpoint(rng, nv, G, H, I)
    got = ops.ffn_weights_from_codes(fmt, dev(_nibbles(codes)), dev(sb), dev(_nibbles(codes2)), dev(sb2),
                                     *((dev(g), dev(g2)) if nv else ()))
    for (q, s), (a, b), gu in (((codes, sb), (got.w13, got.w13_scales), True),
                               ((codes2, sb2), (got.w2, got.w2_scales), False)):
        back = fu.unpack_fp4(host(a), host(b), nv, gu)
        np.testing.assert_array_equal(back[0], q)
        np.testing.assert_array_equal(back[1], s)


def test_a_checkpoints_scales_are_not_the_packing_calls():
    """Why codes are handed over: quantizing the same weights with the quotient
    amax / 448 gives other scales and, at ties, codes a whole step away."""
    w = fu.make_weights(np.random.default_rng(0), 4, 512, 256)[0]
    q, s, _ = _fp8_checkpoint(w)
    again = [oracle.quantize_weight_blocks(m) for m in w]
    assert (s != np.stack([a[1] for a in again])).any()
    assert (q != np.stack([a[0] for a in again])).any()


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("T", [1, 13, 48])
def test_decode_on_a_checkpoint(fmt, T):
    H, E, K, I = 512, 12, 4, 256
    rng = np.random.default_rng(T)
    handle, v13, v2 = _handle(fmt, rng, E, H, I)
    shared, s13, s2 = _handle(fmt, rng, 1, H, 128)
    logits, x = rng.standard_normal((T, E)).astype(np.float32), fu.bf16(rng.standard_normal((T, H)))
    out, idx, w = ops.moe_decode(dev(logits), dev_bf16(x), K, handle, shared=shared)
    ref, bound = fu.layer(x, host(idx), host(w), E, 0, v13, v2, (s13[0], s2[0]))
    fu.check(host_bits(out), ref, bound)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4", "nvfp4"])
def test_a_layer_on_packed_weights(fmt):
    """Both paths of MoELayer, after weights of another kind and before them."""
    H, E, K, I, sI, T = 256, 8, 2, 128, 256, 300
    rng = np.random.default_rng(3)
    layer = MoELayer(T, H, E, K, I, shared_I=sI)
    if fmt == "bf16":
        v13, v2 = fu.make_weights(rng, E, H, I)
        s13, s2 = fu.make_weights(rng, 1, H, sI)
        handle, shared = (ops.ffn_weights(dev_bf16(a), dev_bf16(b)) for a, b in ((v13, v2), (s13, s2)))
    else:
        handle, v13, v2 = _handle(fmt, rng, E, H, I)
        shared, s13, s2 = _handle(fmt, rng, 1, H, sI)
    other = [dev_bf16(m) for m in (*fu.make_weights(rng, E, H, I), *fu.make_weights(rng, 1, H, sI))]
    logits, x = rng.standard_normal((T, E)).astype(np.float32), fu.bf16(rng.standard_normal((T, H)))
    layer.set_weights(*other, fp8=fmt == "bf16")
    before = layer.forward(dev(logits), dev_bf16(x)).clone()
    layer.set_packed_weights(handle, shared)
    prompt = host_bits(layer.forward(dev(logits), dev_bf16(x)))
    idx, w = host(layer.topk_idx), host(layer.topk_w)
    ref, bound = fu.layer(x, idx, w, E, 0, v13, v2, (s13[0], s2[0]), a_step=fu.SINGLE)
    # the staged path also rounds each routed row and the shared one to bf16
    rows = np.abs(fu.expert(bf16_bits_to_f64(x), s13[0], s2[0], fu.SINGLE)[0])
    for e in range(E):
        t, k = np.nonzero(idx == e)
        y, _ = fu.expert(bf16_bits_to_f64(x[t]), v13[e], v2[e], fu.SINGLE)
        np.add.at(rows, t, np.abs(w[t, k].astype(np.float64)[:, None] * y))
    fu.check(prompt, ref, bound + 1.01 * fu.BF16_HALF * (rows + bound), "prompt")
    out = host_bits(layer.decode(dev(logits[:9]), dev_bf16(x[:9])))
    ref, bound = fu.layer(x[:9], idx[:9], w[:9], E, 0, v13, v2, (s13[0], s2[0]))
    fu.check(out, ref, bound, "decode")
    layer.set_weights(*other, fp8=fmt == "bf16")
    assert torch.equal(layer.forward(dev(logits), dev_bf16(x)), before)
    assert int(layer.dev_error.item()) == 0


def test_refusals():
    rng = np.random.default_rng(1)
    handle, _, _ = _handle("fp8", rng, 2, 256, 128)
    other, _, _ = _handle("mxfp4", rng, 1, 256, 128)
    layer = MoELayer(4, 256, 2, 1, 128, shared_I=128)
    with pytest.raises(ValueError, match="another format"):
        layer.set_packed_weights(handle, other)
    with pytest.raises(ValueError, match="2 experts"):
        layer.set_packed_weights(other)
    with pytest.raises(ValueError, match="shared expert"):
        layer.set_packed_weights(handle, handle)
    q, q2 = torch.zeros(2, 256, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 256, 128, dtype=torch.uint8, device="cuda")
    s, s2 = torch.zeros(2, 2, 2, device="cuda"), torch.zeros(2, 2, 1, device="cuda")
    ops.ffn_weights_from_codes("fp8", q, s, q2, s2)
    bad = [(ValueError, ("bf16", q, s, q2, s2)), (ValueError, ("fp8", q, s[:, :1], q2, s2)),
           (ValueError, ("fp8", q, s, q2[:1], s2)), (TypeError, ("fp8", q, s.double(), q2, s2)),
           (TypeError, ("fp8", q.float(), s, q2, s2)), (ValueError, ("fp8", q.transpose(1, 2), s, q2, s2)),
           (ValueError, ("fp8", q[0], s, q2, s2)), (ValueError, ("fp8", q.cpu(), s, q2, s2)),
           (ValueError, ("mxfp4", q, s, q2, s2))]
    for err, args in bad:
        with pytest.raises(err):
            ops.ffn_weights_from_codes(*args)
    codes = [torch.zeros(2, n, dtype=torch.uint8, device="cuda") for n in (256 * 128, 256 * 16, 256 * 64, 256 * 8)]
    c13, b13, c2, b2 = (t.view(2, 256, -1) for t in codes)
    with pytest.raises(ValueError, match="tensor scales"):
        ops.ffn_weights_from_codes("nvfp4", c13, b13, c2, b2)


@pytest.mark.parametrize("kw", [dict(), dict(fp8=True), dict(fp4="nvfp4")], ids=["bf16", "fp8", "nvfp4"])
def test_weights_after_the_fp8_path(kw):
    """A layer that held "w8a8" weights gives the bits of a new one."""
    T, H, E, K, I, sI = 70, 512, 8, 2, 128, 128
    rng = np.random.default_rng(8)
    w = [dev_bf16(m) for m in (*fu.make_weights(rng, E, H, I), *fu.make_weights(rng, 1, H, sI))]
    logits, x = dev(rng.standard_normal((T, E)).astype(np.float32)), dev_bf16(fu.bf16(rng.standard_normal((T, H))))
    outs = []
    for first in (False, True):
        layer = MoELayer(T, H, E, K, I, shared_I=sI)
        if first:
            layer.set_weights(*w, fp8="w8a8")
            layer.forward(logits, x)
        layer.set_weights(*w, **kw)
        outs.append(layer.forward(logits, x).clone())
        assert int(layer.dev_error.item()) == 0
    assert torch.equal(outs[0], outs[1])
