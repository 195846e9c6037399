"""4-bit expert weights: moe_pack_ffn_weights_fp4 against the oracle's FP4
fake-quantizers (codes and scales read back through the packed order, values
bit for bit), moe_grouped_ffn_fp4 against the float64 FFN on those values
within element-wise bounds (tests/few_util.py)."""

import numpy as np
import pytest
import torch

from combine_top_route_moe_amd import ops
from oracle.numerics import bf16_bits_to_f32, bf16_bits_to_f64
from tests import few_util as fu
from tests.gpu_util import need_gpu, dev, dev_bf16, host, host_bits

pytestmark = pytest.mark.gpu

FMTS = ("mxfp4", "nvfp4")


def setup_module(module):
    need_gpu()
    assert ops.moe_device_check(0) == 0, "not a gfx950 device"


# ---- packing -----------------------------------------------------------------
def _planted(rng, G, N, K):
    """Weights with edge groups: all zero, negative zeros, one large value over
    tiny ones, exact ties between codes, tiny magnitudes."""
    w = rng.standard_normal((G, N, K)).astype(np.float32) * 0.05
    w[0, 0, :32] = 0.0
    w[0, 1, :32] = -0.0
    w[0, 2, :32] = 1e-4
    w[0, 2, 5] = 3.0
    ties = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0.5])
    w[0, 3, :32] = np.tile(ties, 2)
    w[0, 4, :32] = np.tile(ties, 2) * 2.0 ** -9
    w[0, 5, :32] = 2.0 ** -120
    w[0, N - 1, K - 32:] = np.tile(ties[::-1], 2)
    return fu.bf16(w)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G,H,I", [(1, 128, 128), (3, 256, 384), (2, 640, 128)])
def test_pack_matches_the_fake_quantizer(fmt, G, H, I):
    rng = np.random.default_rng(G * H + I)
    w13, w2 = _planted(rng, G, 2 * I, H), _planted(rng, G, H, I)
    nv = fmt == "nvfp4"
    mode = ops.MOE_FQ_NVFP4 if nv else ops.MOE_FQ_MXFP4
    q13, s13, g13, q2, s2, g2 = ops.moe_pack_ffn_weights_fp4(dev_bf16(w13), dev_bf16(w2), mode)
    for w, q, s, g, gu in ((w13, q13, s13, g13, True), (w2, q2, s2, g2, False)):
        g = host(g) if nv else None
        if nv:
            np.testing.assert_array_equal(g, [fu.tensor_scale(m) for m in w])
        codes, sb = fu.unpack_fp4(host(q), host(s), nv, gu)
        want = np.stack([fu.fake_quant(m, fmt) for m in w])
        got = fu.fp4_values(codes, sb, nv, g)
        # a zero keeps its sign in a code; the fake-quant writes +0 for an all-zero group
        np.testing.assert_array_equal(bf16_bits_to_f32(got), bf16_bits_to_f32(want))
    # packing the stored values again gives them back
    v13 = np.stack([fu.fake_quant(m, fmt) for m in w13])
    v2 = np.stack([fu.fake_quant(m, fmt) for m in w2])
    again = ops.moe_pack_ffn_weights_fp4(dev_bf16(v13), dev_bf16(v2), mode, g13, g2)
    for v, q, s, g, gu in ((v13, again[0], again[1], g13, True), (v2, again[3], again[4], g2, False)):
        codes, sb = fu.unpack_fp4(host(q), host(s), nv, gu)
        got = bf16_bits_to_f32(fu.fp4_values(codes, sb, nv, host(g) if nv else None))
        ref = bf16_bits_to_f32(v)
        if nv:   # guaranteed where the block's largest code is 6
            top = np.abs(codes & 7).reshape(codes.shape[:2] + (-1, 16)).max(-1).repeat(16, -1) == 7
            np.testing.assert_array_equal(got[top], ref[top])
        else:
            np.testing.assert_array_equal(got, ref)


def test_pack_one_matrix_alone():
    rng = np.random.default_rng(5)
    w13, w2 = fu.make_weights(rng, 2, 256, 128)
    both = ops.moe_pack_ffn_weights_fp4(dev_bf16(w13), dev_bf16(w2))
    a = ops.moe_pack_ffn_weights_fp4(dev_bf16(w13), None)
    b = ops.moe_pack_ffn_weights_fp4(None, dev_bf16(w2))
    assert a[3] is None and b[0] is None and both[2] is None
    assert torch.equal(a[0], both[0]) and torch.equal(a[1], both[1])
    assert torch.equal(b[3], both[3]) and torch.equal(b[4], both[4])


# ---- the FFN -----------------------------------------------------------------
def _segments(counts, pad=0):
    """cu_seqlens and capacity with `pad` unused rows after every segment."""
    cu = np.zeros(len(counts) + 1, np.int32)
    cu[1:] = np.cumsum(np.asarray(counts) + pad)
    return cu, int(cu[-1])


def _weights(rng, fmt, G, H, I):
    w13, w2 = fu.make_weights(rng, G, H, I)
    handle = ops.ffn_weights(dev_bf16(w13), dev_bf16(w2), fmt)
    return handle, fu.Stored(w13, fmt), fu.Stored(w2, fmt)


def _check(y_bits, x, cu, counts, v13, v2, scale, a_step, sentinel=None):
    covered = np.zeros(len(x), bool)
    for g, n in enumerate(counts):
        if n <= 0:
            continue
        r = slice(cu[g], cu[g] + n)
        covered[r] = True
        ref, err = fu.expert(bf16_bits_to_f64(x[r]), v13[g], v2[g], a_step)
        if scale is not None:
            ref, err = ref * scale[r, None].astype(np.float64), err * np.abs(scale[r, None])
        fu.check(y_bits[r], ref, err + fu.BF16_HALF * (np.abs(ref) + err), f"group {g}")
    if sentinel is not None:
        np.testing.assert_array_equal(y_bits[~covered], sentinel[~covered])


# (counts, H, I): few rows a group or few groups, which the few-row kernels take;
# more of both; and as many as only the tile kernel takes
FEW = [([1], 128, 128), ([1], 2048, 256), ([16], 256, 128), ([0, 3, 0, 1, 17, 0], 384, 256),
       ([33, 0, 0, 2, 0], 256, 384), ([0] * 70 + [5, 0, 1], 128, 128), ([2] * 130, 128, 128),
       ([0, 0, 1], 1152, 640), ([17, 9], 128, 128), ([8, 129], 384, 256), ([5, 20], 1152, 1152)]
MANY = [([64] * 80, 128, 128), ([1, 0, 130, 65, 64, 63, 16, 17] * 6, 384, 256), ([0, 50] * 18, 640, 1152),
        ([5000], 128, 128), ([300, 0, 5, 77, 640, 800], 256, 640), ([127, 1, 128, 130, 257, 0], 1152, 896)]
TILE = [([40] * 150, 256, 384), ([1, 0, 130, 65, 64, 63, 16, 17] * 20, 384, 256), ([0, 50] * 60, 640, 1152),
        ([20000], 128, 128), ([300, 0, 5, 77, 640, 800] * 6, 256, 640),
        ([127, 1, 128, 130, 257, 0] * 8, 1152, 896)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", range(len(FEW) + len(MANY) + len(TILE)))
@pytest.mark.parametrize("scaled", [True, False])
def test_ffn_matches_float64(fmt, case, scaled):
    counts, H, I = (FEW + MANY + TILE)[case]
    rng = np.random.default_rng(100 + case)
    G = len(counts)
    handle, v13, v2 = _weights(rng, fmt, G, H, I)
    cu, cap = _segments(counts)
    x = fu.bf16(rng.standard_normal((cap, H)))
    scale = rng.standard_normal(cap).astype(np.float32) if scaled else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.moe_grouped_ffn_fp4(dev_bf16(x), dev(cu), dev(np.array(counts, np.int32)), handle,
                                None if scale is None else dev(scale), dev_error=err)
    assert int(err.item()) == 0
    _check(host_bits(y), x, cu, counts, v13, v2, scale, fu.PAIR if case < len(FEW) else fu.SINGLE)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,I", [([3, 0, 9], 128), ([1000, 0, 429], 2048), ([4000, 0, 429], 2048)])
def test_rows_outside_the_segments_stay_and_do_not_matter(fmt, counts, I):
    """Unused rows between segments hold NaN and are neither read into other
    rows nor written; a NaN or inf in one row reaches that row only; the
    workspace is not written past its size."""
    rng = np.random.default_rng(7)
    H, G = 256, len(counts)
    handle, v13, v2 = _weights(rng, fmt, G, H, I)
    cu, cap = _segments(counts, pad=3)
    x = fu.bf16(rng.standard_normal((cap, H)))
    used = np.zeros(cap, bool)
    for g, n in enumerate(counts):
        used[cu[g]:cu[g] + n] = True
    x[~used] = 0x7FC0
    bad = cu[2] + 1
    x_bad = x.copy()
    x_bad[bad, 3], x_bad[bad, 9] = 0x7FC0, 0x7F80
    need = ops.moe_grouped_ffn_fp4_workspace_bytes(cap, G, H, I)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    sentinel = rng.integers(0, 1 << 16, (cap, H)).astype(np.uint16)
    outs = []
    for xb in (x, x_bad):
        y = dev_bf16(sentinel)
        ops.moe_grouped_ffn_fp4(dev_bf16(xb), dev(cu), dev(np.array(counts, np.int32)), handle, None,
                                y=y, workspace=ws)
        outs.append(host_bits(y))
    _check(outs[0], x, cu, counts, v13, v2, None, fu.SINGLE, sentinel)
    other = np.arange(cap) != bad
    np.testing.assert_array_equal(outs[1][other], outs[0][other])
    assert np.isnan(bf16_bits_to_f32(outs[1][bad])).all()
    assert (ws[need:] == 0x5A).all()


@pytest.mark.parametrize("rows,I", [(5, 128), (3000, 768), (9000, 768)])
def test_bad_segments_are_skipped_and_reported(rows, I):
    rng = np.random.default_rng(9)
    H = 128
    handle, v13, v2 = _weights(rng, "mxfp4", 3, H, I)
    x = fu.bf16(rng.standard_normal((rows, H)))
    half = rows // 2
    counts = np.array([half, 4, rows - half], np.int32)
    for cu in ([0, rows - 1, half, rows], [0, -2, half, rows]):
        cu = np.array(cu, np.int32)
        sentinel = rng.integers(0, 1 << 16, (rows, H)).astype(np.uint16)
        y, err = dev_bf16(sentinel), torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.moe_grouped_ffn_fp4(dev_bf16(x), dev(cu), dev(counts), handle, None, y=y, dev_error=err)
        assert int(err.item()) == ops.MOE_DEVERR_ROW_RANGE
        keep = counts.copy()
        keep[1] = 0
        _check(host_bits(y), x, cu, keep, v13, v2, None, fu.SINGLE, sentinel)
    # overlapping segments that need more runs than disjoint ones could: reported
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    counts = np.array([rows, rows, rows], np.int32)
    ops.moe_grouped_ffn_fp4(dev_bf16(x), dev(np.zeros(4, np.int32)), dev(counts), handle, None, dev_error=err)
    torch.cuda.synchronize()
    if rows >= 90:
        ops.moe_grouped_ffn_fp4(dev_bf16(x), dev(np.zeros(4, np.int32)),
                                dev(np.full(3, 1 << 30, np.int32)), handle, None, dev_error=err)
        assert int(err.item()) == ops.MOE_DEVERR_ROW_RANGE


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,I", [([2, 5], 256), ([760, 350], 1280), ([2000, 900], 1280)])
def test_stages_streams_graphs_and_repeats(fmt, counts, I):
    """GATE_UP then DOWN equals ALL; another stream; a captured graph replayed
    between eager calls on other inputs; the same bits every time."""
    rng = np.random.default_rng(11)
    H = 384
    handle, v13, v2 = _weights(rng, fmt, 2, H, I)
    cu, cap = _segments(counts)
    cu_d, n_d = dev(cu), dev(np.array(counts, np.int32))
    xs = [dev_bf16(fu.bf16(rng.standard_normal((cap, H)))) for _ in range(3)]
    ws = torch.empty(ops.moe_grouped_ffn_fp4_workspace_bytes(cap, 2, H, I), dtype=torch.uint8, device="cuda")
    want = [ops.moe_grouped_ffn_fp4(x, cu_d, n_d, handle) for x in xs]
    y = torch.zeros_like(want[0])
    ops.moe_grouped_ffn_fp4(xs[0], cu_d, n_d, handle, y=y, workspace=ws, flags=ops.MOE_FFN_GATE_UP)
    assert not y.any()
    ops.moe_grouped_ffn_fp4(xs[0], cu_d, n_d, handle, y=y, workspace=ws, flags=ops.MOE_FFN_DOWN)
    assert torch.equal(y, want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = torch.zeros_like(y)
    ops.moe_grouped_ffn_fp4(xs[1], cu_d, n_d, handle, y=y2, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y2, want[1])
    x_in, graph = xs[0].clone(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ops.moe_grouped_ffn_fp4(x_in, cu_d, n_d, handle, y=y, workspace=ws)
    for i in (1, 2, 0, 2):
        x_in.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(ops.moe_grouped_ffn_fp4(xs[0], cu_d, n_d, handle, workspace=ws), want[0])


def test_empty_batch():
    handle, _, _ = _weights(np.random.default_rng(1), "mxfp4", 2, 128, 128)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert ops.moe_grouped_ffn_fp4(x, z, z[:2], handle).shape == (0, 128)
