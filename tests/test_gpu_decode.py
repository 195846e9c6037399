"""moe_decode, the whole layer for a few tokens, against the float64 layer on
the weights its format stores, within element-wise bounds (tests/few_util.py);
routes bit for bit as moe_route gives them."""

import numpy as np
import pytest
import torch

import oracle
from combine_top_route_moe_amd import MoELayer, ops
from oracle.numerics import bf16_bits_to_f32, bf16_bits_to_f64
from tests import few_util as fu
from tests.gpu_util import need_gpu, dev, dev_bf16, host, host_bits

pytestmark = pytest.mark.gpu

FMTS = ("bf16", "fp8", "mxfp4", "nvfp4")


def setup_module(module):
    need_gpu()
    assert ops.moe_device_check(0) == 0, "not a gfx950 device"


class Layer:
    """Seeded weights of one layer: device handle and the values it stores."""

    def __init__(self, seed, fmt, El, H, I, sI=0, spoil=None):
        rng = np.random.default_rng(seed)
        self.H, self.I, self.El, self.sI = H, I, El, sI
        w13, w2 = fu.make_weights(rng, El, H, I)
        if spoil is not None:
            spoil(w13, w2)
        self.handle = ops.ffn_weights(dev_bf16(w13), dev_bf16(w2), fmt)
        self.v13, self.v2 = fu.Stored(w13, fmt), fu.Stored(w2, fmt)
        self.shared = self.shared_v = None
        if sI:
            s13, s2 = fu.make_weights(rng, 1, H, sI)
            self.shared = ops.ffn_weights(dev_bf16(s13), dev_bf16(s2), fmt)
            self.shared_v = (fu.fake_quant(s13[0], fmt), fu.fake_quant(s2[0], fmt))

    def check(self, out, x, idx, w, begin=0, what=""):
        ref, bound = fu.layer(x, idx, w, self.El, begin, self.v13, self.v2, self.shared_v)
        fu.check(host_bits(out), ref, bound, what)


def _inputs(rng, T, E, H):
    return rng.standard_normal((T, E)).astype(np.float32), fu.bf16(rng.standard_normal((T, H)))


# T, H, E, K, I, shared_I, local experts, first local, padding rows
SHAPES = [
    (1, 128, 1, 1, 128, 0, 1, 0, 0),
    (1, 256, 8, 2, 128, 128, 8, 0, 0),
    (1, 1152, 60, 6, 384, 640, 60, 0, 0),
    (2, 128, 1000, 32, 128, 0, 1000, 0, 0),
    (7, 384, 5, 3, 256, 0, 5, 0, 2),
    (15, 256, 8, 8, 128, 256, 8, 0, 0),
    (16, 128, 16, 2, 256, 0, 8, 8, 0),
    (17, 256, 4, 1, 128, 128, 4, 0, 1),
    (32, 256, 3, 2, 128, 0, 3, 0, 0),
    (33, 128, 130, 5, 256, 128, 65, 30, 3),
    (48, 640, 40, 8, 128, 0, 40, 0, 0),
    (64, 256, 2, 2, 128, 128, 2, 0, 0),
    (64, 128, 200, 10, 128, 0, 200, 0, 5),
    (64, 256, 7, 3, 384, 128, 3, 2, 0),
    # enough experts at work for the row tiles; a few with many tokens
    (40, 128, 300, 8, 128, 128, 300, 0, 0),
    (64, 640, 40, 6, 896, 256, 40, 0, 3),
    (64, 384, 3, 2, 4096, 0, 3, 0, 0),
    (64, 128, 1024, 32, 128, 128, 1024, 0, 0),      # all the entries there can be
    (20, 1152, 4, 2, 1152, 0, 4, 0, 0),             # few tiles, long reductions
    (2, 1152, 100, 2, 1152, 128, 100, 0, 0),
    (8, 1536, 2, 2, 256, 128, 2, 0, 0),             # a few experts for all, or long rows
    (8, 19200, 100, 8, 128, 0, 2, 50, 1),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_layer_matches_float64(fmt, shape):
    T, H, E, K, I, sI, El, begin, pad = shape
    rng = np.random.default_rng(sum(shape))
    L = Layer(sum(shape) + 1, fmt, El, H, I, sI)
    logits, x = _inputs(rng, T, E, H)
    valid = None
    if pad:
        valid = np.ones(T, np.uint8)
        valid[rng.permutation(T)[:pad]] = 0
    renorm = T % 2 == 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, idx, w = ops.moe_decode(dev(logits), dev_bf16(x), K, L.handle, expert_begin=begin,
                                 row_valid=None if valid is None else dev(valid), renormalize=renorm,
                                 shared=L.shared, dev_error=err)
    assert int(err.item()) == 0
    ri, rw = ops.moe_route(dev(logits), K, None if valid is None else dev(valid), renorm)
    assert torch.equal(idx, ri) and torch.equal(w, rw)
    np.testing.assert_array_equal(host(idx), oracle.route(logits, valid, K, renorm)[0])
    L.check(out, x, host(idx), host(w), begin)


def test_a_model_sized_layer():
    """Long reductions: the bound of single elements is loose there, so the
    whole result's error too: one rounding, at most 2^-8 relative, and the
    float32 sums' share, taken as 2^-12 (sums of a few thousand terms of
    random sign are off by far less than their worst case)."""
    T, H, E, K, I, sI = 3, 4096, 3, 2, 1536, 1536
    rng = np.random.default_rng(3)
    for fmt in FMTS:
        L = Layer(4, fmt, E, H, I, sI)
        logits, x = _inputs(rng, T, E, H)
        out, idx, w = ops.moe_decode(dev(logits), dev_bf16(x), K, L.handle, shared=L.shared)
        ref, _ = fu.layer(x, host(idx), host(w), E, 0, L.v13, L.v2, L.shared_v)
        d = np.linalg.norm(bf16_bits_to_f64(host_bits(out)) - ref) / np.linalg.norm(ref)
        assert d <= 2.0 ** -8 + 2.0 ** -12, (fmt, d)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_given_routes(T):
    """Ids of the caller's: padding slots, other ranks' experts, ids past the
    last expert (reported), one expert named in several slots."""
    H, I, El, begin, E, K = 256, 128, 6, 4, 12, 5
    rng = np.random.default_rng(T)
    L = Layer(8, "bf16", El, H, I, 128)
    _, x = _inputs(rng, T, E, H)
    idx = rng.integers(-1, E, (T, K)).astype(np.int32)
    idx[0] = [5, 5, -1, 5, 9]
    w = rng.standard_normal((T, K)).astype(np.float32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ti, tw = dev(idx), dev(w)
    run = lambda: ops.moe_decode(None, dev_bf16(x), K, L.handle, expert_begin=begin, num_experts=E,  # noqa: E731
                                 shared=L.shared, topk_idx=ti, topk_w=tw, dev_error=err)[0]
    L.check(run(), x, idx, w, begin)
    assert int(err.item()) == 0
    np.testing.assert_array_equal(host(ti), idx)          # inputs stay
    np.testing.assert_array_equal(host(tw), w)
    idx2 = idx.copy()
    idx2[T - 1, 1], idx2[0, 0] = E, 0x7FFFFFFF
    ti.copy_(dev(idx2))
    out = run()
    assert int(err.item()) == ops.MOE_DEVERR_EXPERT_RANGE
    L.check(out, x, np.where(idx2 >= E, -1, idx2), w, begin)
    # all rows masked: the shared expert alone
    out = ops.moe_decode(None, dev_bf16(x), K, L.handle, expert_begin=begin, num_experts=E, shared=L.shared,
                         topk_idx=ti, topk_w=tw, row_valid=torch.zeros(T, dtype=torch.uint8, device="cuda"))[0]
    L.check(out, x, np.full_like(idx, -1), w, begin)


@pytest.mark.parametrize("fmt", FMTS)
def test_no_expert_here_gives_plus_zero(fmt):
    L = Layer(2, fmt, 2, 128, 128)
    rng = np.random.default_rng(2)
    logits, x = _inputs(rng, 9, 8, 128)
    logits[:, 4:6] = -50.0
    out, idx, w = ops.moe_decode(dev(logits), dev_bf16(x), 3, L.handle, expert_begin=4)
    assert not np.isin(host(idx), [4, 5]).any()
    assert (host_bits(out) == 0).all()
    out, idx, _ = ops.moe_decode(dev(logits), dev_bf16(x), 3, L.handle,
                                 row_valid=torch.zeros(9, dtype=torch.uint8, device="cuda"))
    assert (host(idx) == -1).all() and (host_bits(out) == 0).all()


@pytest.mark.parametrize("T", [1, 12, 50])
def test_infinities_and_nan_stay_where_they_belong(T):
    """NaN and inf weights of one expert reach only the tokens that chose it;
    NaN in one token's hidden row reaches only that token; NaN and infinite
    logits route as moe_route says."""
    H, I, E, K = 256, 128, 6, 2

    def spoil(w13, w2):
        w13[3, 5, 7], w13[3, I + 9, 11] = 0x7FC0, 0x7F80
        w2[3, 2, 2] = 0xFF80

    L = Layer(5, "bf16", E, H, I, 0, spoil)
    rng = np.random.default_rng(T)
    logits, x = _inputs(rng, T, E, H)
    logits[:, 3] -= 1.0
    logits[0, 3] = -np.inf
    if T > 1:
        logits[1] = [np.nan, 1.0, -np.inf, np.nan, 0.5, -np.inf]
        logits[2] = [np.inf, np.inf, 0, 0, 0, 0]
        x[4, 10] = 0x7FC0
        logits[5] = -np.inf
        logits[5, 3] = np.nan
    out, idx, w = ops.moe_decode(dev(logits), dev_bf16(x), K, L.handle)
    ri, rw = ops.moe_route(dev(logits), K)
    assert torch.equal(idx, ri) and torch.equal(w, rw)
    idx, got = host(idx), bf16_bits_to_f32(host_bits(out))
    clean = ~(idx == 3).any(1)
    if T > 1:
        clean[4] = False
        assert np.isnan(got[4]).all()
    assert np.isfinite(got[clean]).all() and clean.any()
    v13, v2 = list(L.v13), list(L.v2)
    v13[3], v2[3] = np.zeros_like(v13[3]), np.zeros_like(v2[3])
    xc = x.copy()
    xc[~clean] = 0
    ref, bound = fu.layer(xc, idx, host(w), E, 0, v13, v2)
    fu.check(host_bits(out)[clean], ref[clean], bound[clean])
    assert np.isnan(got[(idx == 3).any(1)]).any(axis=1).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,E", [(1, 2), (1, 300), (12, 2), (3, 2)])
def test_an_intermediate_past_the_range_is_an_infinity(fmt, T, E):
    """One intermediate element overflows (float32, or its rounding to bf16):
    the outputs are the infinities that it times w2's column gives, no NaN."""
    H, I = 128, 128
    w13, w2 = np.zeros((E, 2 * I, H), np.float32), np.full((E, H, I), 0.5, np.float32)
    w13[:, 5, 0] = w13[:, I + 5, 1] = 1.0
    w2[:, ::2, 5] = -0.5
    h = ops.ffn_weights(dev_bf16(fu.bf16(w13)), dev_bf16(fu.bf16(w2)), fmt)
    logits = np.zeros((T, E), np.float32)
    # a = g u: past float32; below 2^128, but rounding past bf16 (from 2^128 (1 - 2^-9))
    for big in ((1e30, 1e30), (2.0 ** 64 * 129 / 128, 2.0 ** 64 * 127 / 128)):
        x = np.zeros((T, H), np.float32)
        x[:, :2] = big
        got = bf16_bits_to_f64(host_bits(ops.moe_decode(dev(logits), dev_bf16(fu.bf16(x)), 1, h)[0]))
        assert np.isinf(got).all() and (got[:, ::2] < 0).all() and (got[:, 1::2] > 0).all(), big


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_graphs_streams_and_repeats(fmt):
    """Two captured batch sizes that share a workspace and the weights,
    replayed in turn between eager calls; another stream; the same bits every
    time; nothing written past the outputs or the workspace."""
    H, I, E, K, sI = 384, 256, 20, 4, 128
    L = Layer(6, fmt, E, H, I, sI)
    rng = np.random.default_rng(6)
    cases = {}
    need = max(ops.moe_decode_workspace_bytes(T, H, I, K, E, sI) for T in (3, 41))
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for T in (3, 41):
        ins = []
        for _ in range(3):
            logits, x = _inputs(rng, T, E, H)
            ins.append((dev(logits), dev_bf16(x)))
        want = [ops.moe_decode(a, b, K, L.handle, shared=L.shared) for a, b in ins]
        for a, b in zip(ins, want):
            again = ops.moe_decode(a[0], a[1], K, L.handle, shared=L.shared, workspace=ws)
            assert all(torch.equal(p, q) for p, q in zip(again, b))
        buf = dict(logits=ins[0][0].clone(), x=ins[0][1].clone(),
                   idx=torch.zeros(T + 1, K, dtype=torch.int32, device="cuda"),
                   w=torch.zeros(T + 1, K, device="cuda"),
                   out=torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device="cuda"))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ops.moe_decode(buf["logits"], buf["x"], K, L.handle, shared=L.shared, topk_idx=buf["idx"][:T],
                           topk_w=buf["w"][:T], out=buf["out"][:T], workspace=ws)
        cases[T] = (graph, buf, ins, want)
    for i in (0, 2, 1, 2):
        for T, (graph, buf, ins, want) in cases.items():
            buf["logits"].copy_(ins[i][0])
            buf["x"].copy_(ins[i][1])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(buf["out"][:T], want[i][0]) and torch.equal(buf["idx"][:T], want[i][1])
            assert torch.equal(buf["w"][:T], want[i][2])
            assert (buf["out"][T] == 7.0).all() and not buf["idx"][T].any()
        other = cases[41][2][0]
        eager = ops.moe_decode(other[0], other[1], K, L.handle, shared=L.shared, workspace=ws)
        assert torch.equal(eager[0], cases[41][3][0][0])
    assert (ws[need:] == 0x5A).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = cases[3][2][1]
    out = torch.empty(3, H, dtype=torch.bfloat16, device="cuda")
    ops.moe_decode(a, b, K, L.handle, shared=L.shared, out=out, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, cases[3][3][1][0])


@pytest.mark.parametrize("T", [2, 30])
def test_two_calls_at_once(T):
    """Calls on two streams at a time, each with workspace and outputs of its
    own, allocated by the binding on the call's stream: the bits of a call
    alone.  The side stream's packing, too."""
    H, I, E, K = 512, 1024, 32, 4
    rng = np.random.default_rng(T)
    w13, w2 = (dev_bf16(m) for m in fu.make_weights(rng, E, H, I))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    handles = [ops.ffn_weights(w13, w2, "nvfp4", stream=s) for s in streams]
    torch.cuda.synchronize()
    for n in ("w13", "w13_scales", "w13_tensor_scale", "w2", "w2_scales", "w2_tensor_scale"):
        assert torch.equal(getattr(handles[0], n), getattr(handles[1], n))
    ins = [tuple(f(a) for f, a in zip((dev, dev_bf16), _inputs(rng, T, E, H))) for _ in range(2)]
    want = [ops.moe_decode(a, b, K, handles[0])[0] for a, b in ins]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(12):
        for i in (0, 1):
            got[i].append(ops.moe_decode(*ins[i], K, handles[i], stream=streams[i])[0])
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_expert_parallel_shares_add_up():
    """The shares of two ranks, added, are the whole layer: each share is off
    by its own bound."""
    T, H, E, K, I = 21, 256, 10, 4, 128
    rng = np.random.default_rng(12)
    w13, w2 = fu.make_weights(rng, E, H, I)
    logits, x = _inputs(rng, T, E, H)
    parts, bounds = [], []
    for begin, n in ((0, 3), (3, 7)):
        h = ops.ffn_weights(dev_bf16(w13[begin:begin + n]), dev_bf16(w2[begin:begin + n]), "bf16")
        out, idx, w = ops.moe_decode(dev(logits), dev_bf16(x), K, h, expert_begin=begin)
        parts.append(bf16_bits_to_f64(host_bits(out)))
        bounds.append(fu.layer(x, host(idx), host(w), n, begin, w13[begin:], w2[begin:])[1])
    ref, _ = fu.layer(x, host(idx), host(w), E, 0, w13, w2)
    assert (np.abs(sum(parts) - ref) <= sum(bounds)).all()


def test_no_tokens():
    L = Layer(1, "bf16", 2, 128, 128)
    out, idx, w = ops.moe_decode(torch.empty(0, 4, device="cuda"),
                                 torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), 2, L.handle)
    assert out.shape == (0, 128) and idx.shape == (0, 2)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 16, 17, 64])
@pytest.mark.parametrize("E,K", [(1, 1), (16, 16), (40, 17), (60, 7), (64, 8), (64, 32), (65, 8), (128, 4),
                                 (200, 9), (256, 8), (257, 3), (700, 20)])
def test_routes_are_moe_routes(T, E, K, renorm):
    """Every routing path (in gate/up, in the plan by a wave or by 16 lanes, in
    a launch of its own) on logits with ties, +-0, infinities and NaN."""
    rng = np.random.default_rng(T * E + K)
    logits = rng.integers(-3, 4, (T, E)).astype(np.float32)
    logits[rng.random((T, E)) < 0.1] = -0.0
    logits[0, 0] = np.inf
    logits[T - 1] = rng.standard_normal(E)
    if T > 2:
        logits[1] = -np.inf
        logits[2, ::2] = np.nan
    valid = (rng.random(T) < 0.8).astype(np.uint8)
    handle = ops.ffn_weights(torch.zeros(E, 256, 128, dtype=torch.bfloat16, device="cuda"),
                             torch.zeros(E, 128, 128, dtype=torch.bfloat16, device="cuda"))
    x = dev_bf16(fu.bf16(rng.standard_normal((T, 128))))
    _, idx, w = ops.moe_decode(dev(logits), x, K, handle, row_valid=dev(valid), renormalize=renorm)
    ri, rw = ops.moe_route(dev(logits), K, dev(valid), renorm)
    assert torch.equal(idx, ri)
    np.testing.assert_array_equal(host(w).view(np.uint32), host(rw).view(np.uint32))


# ---- through the layer ---------------------------------------------------------
def _layer(fmt, T, H, E, K, I, sI, seed=3):
    rng = np.random.default_rng(seed)
    w13, w2 = fu.make_weights(rng, E, H, I)
    s13, s2 = fu.make_weights(rng, 1, H, sI)
    layer = MoELayer(T, H, E, K, I, shared_I=sI)
    kw = {} if fmt == "bf16" else {"fp8": True} if fmt == "fp8" else {"fp4": fmt}
    layer.set_weights(dev_bf16(w13), dev_bf16(w2), dev_bf16(s13), dev_bf16(s2), **kw)
    q = lambda m: [fu.fake_quant(x, fmt) for x in m]  # noqa: E731
    return layer, q(w13), q(w2), (fu.fake_quant(s13[0], fmt), fu.fake_quant(s2[0], fmt)), rng


@pytest.mark.parametrize("fmt,T", [(f, 600) for f in FMTS] + [("mxfp4", 6000)])
def test_a_prompt_then_decode_steps(fmt, T):
    """The layer as it is served: a prompt through the staged path (for 4-bit
    weights the grouped FFN on them), then decode steps of changing batches
    eagerly and from a captured graph, in one layer's buffers."""
    H, E, K, I, sI = 256, 8, 2, 384, 128
    layer, v13, v2, sv, rng = _layer(fmt, T, H, E, K, I, sI)
    logits, x = _inputs(rng, T, E, H)
    prompt = host_bits(layer.forward(dev(logits), dev_bf16(x)))
    idx, w = host(layer.topk_idx), host(layer.topk_w)
    ref, bound = fu.layer(x, idx, w, E, 0, v13, v2, sv, a_step=fu.SINGLE)
    # the staged path also rounds each routed row and the shared one to bf16
    rows = np.zeros_like(ref)
    for e in range(E):
        t, k = np.nonzero(idx == e)
        y, _ = fu.expert(bf16_bits_to_f64(x[t]), v13[e], v2[e], fu.SINGLE)
        np.add.at(rows, t, np.abs(w[t, k].astype(np.float64)[:, None] * y))
    rows += np.abs(fu.expert(bf16_bits_to_f64(x), *sv, fu.SINGLE)[0])
    fu.check(prompt, ref, bound + 1.01 * fu.BF16_HALF * (rows + bound), "prompt")
    buf_l, buf_x = torch.zeros(5, E, device="cuda"), torch.zeros(5, H, dtype=torch.bfloat16, device="cuda")
    layer.decode(buf_l, buf_x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.decode(buf_l, buf_x)
    for n in (1, 5, 64, 5, 9):
        logits, x = _inputs(rng, n, E, H)
        if n == 5:
            buf_l.copy_(dev(logits))
            buf_x.copy_(dev_bf16(x))
            graph.replay()
            out = layer.out[:5]
        else:
            out = layer.decode(dev(logits), dev_bf16(x))
        torch.cuda.synchronize()
        idx, w = host(layer.topk_idx[:n]), host(layer.topk_w[:n])
        np.testing.assert_array_equal(idx, oracle.route(logits, None, K, True)[0])
        ref, bound = fu.layer(x, idx, w, E, 0, v13, v2, sv)
        fu.check(host_bits(out), ref, bound, n)
    # the caller's routes, as another router left them
    layer.topk_idx[:3] = dev(np.array([[1, 1], [7, 0], [-1, 4]], np.int32))
    layer.topk_w[:3] = 0.5
    out = layer.decode(None, dev_bf16(x[:3]))
    ref, bound = fu.layer(x[:3], host(layer.topk_idx[:3]), host(layer.topk_w[:3]), E, 0, v13, v2, sv)
    fu.check(host_bits(out), ref, bound, "given")
    assert int(layer.dev_error.item()) == 0


def test_layer_refusals():
    w13, w2 = fu.make_weights(np.random.default_rng(0), 4, 256, 128)
    w13, w2 = dev_bf16(w13), dev_bf16(w2)
    l1 = torch.zeros(1, 4, device="cuda")
    x1 = torch.zeros(1, 256, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(pack=False), dict(fp8="w8a8")):
        layer = MoELayer(8, 256, 4, 2, 128)
        layer.set_weights(w13, w2, **kw)
        with pytest.raises(ValueError, match="packed weights"):
            layer.decode(l1, x1)
    for kw in (dict(combine_qdq=True), dict(dispatch_block=128), dict(dispatch_fp4="mxfp4")):
        layer = MoELayer(8, 256, 4, 2, 128, **kw)
        layer.set_weights(w13, w2)
        with pytest.raises(ValueError, match="quantizers"):
            layer.decode(l1, x1)
    layer = MoELayer(8, 256, 4, 2, 128)
    layer.set_weights(w13, w2)
    with pytest.raises(ValueError, match="up to 8 tokens"):
        layer.decode(torch.zeros(9, 4, device="cuda"), torch.zeros(9, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="unknown FP4"):
        layer.set_weights(w13, w2, fp4="int4")
    with pytest.raises(ValueError, match="neither"):
        layer.set_weights(w13, w2, fp4="mxfp4", fp8=True)


def test_binding_refusals(monkeypatch):
    w13, w2 = fu.make_weights(np.random.default_rng(0), 4, 256, 128)
    h = ops.ffn_weights(dev_bf16(w13), dev_bf16(w2), "mxfp4")
    l2, x2 = torch.zeros(2, 4, device="cuda"), torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = [
        (ValueError, lambda: ops.moe_decode(l2[:1], x2, 2, h)),
        (ValueError, lambda: ops.moe_decode(l2, x2[:, :128].contiguous(), 2, h)),
        (TypeError, lambda: ops.moe_decode(l2.double(), x2, 2, h)),
        (ValueError, lambda: ops.moe_decode(l2, x2.t().contiguous().t(), 2, h)),       # strides
        (ValueError, lambda: ops.moe_decode(None, x2, 2, h)),
        (ValueError, lambda: ops.moe_decode(l2, x2, 2, h, topk_idx=torch.zeros(2, 3, **i32))),
        (ValueError, lambda: ops.moe_decode(l2, x2, 2, h, out=x2[:1])),
        (ValueError, lambda: ops.moe_decode(l2, x2, 2, h, shared=h)),
        (ValueError, lambda: ops.moe_decode(l2.cpu(), x2, 2, h)),
        (RuntimeError, lambda: ops.moe_decode(l2, x2, 2, h, expert_begin=1)),
        (RuntimeError, lambda: ops.moe_decode(l2, x2, 2, h, out=x2)),
        (TypeError, lambda: ops.moe_decode(l2, x2, 2, h, workspace=torch.zeros(1 << 20, device="cuda"))),
        (TypeError, lambda: ops.moe_decode(l2, x2, 2, h, dev_error=torch.zeros(1, device="cuda"))),
        (RuntimeError, lambda: ops.moe_decode(l2, x2, 2, h, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))),
        (ValueError, lambda: ops.moe_grouped_ffn_fp4(x2, torch.zeros(4, **i32), torch.zeros(4, **i32), h)),
        (ValueError, lambda: ops.moe_grouped_ffn_fp4(x2, torch.zeros(5, **i32), torch.zeros(4, **i32), h,
                                                     torch.zeros(1, device="cuda"))),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)      # another device is current
    with pytest.raises(ValueError, match="current device"):
        ops.moe_decode(l2, x2, 2, h)
    with pytest.raises(ValueError, match="current device"):
        ops.moe_grouped_ffn_fp4(x2, torch.zeros(5, **i32), torch.zeros(4, **i32), h)
