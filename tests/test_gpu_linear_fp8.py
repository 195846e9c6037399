"""moe_linear_fp8 and its packing against the product in 64 bits."""

import pytest
import torch

from combine_top_route_moe_amd import ops
from combine_top_route_moe_amd._lib import load
from tests.around_util import BF16, TINY, U, e4m3, gen, product_slack, quant_rows, quant_tiles, rows64, tiles64, within

pytestmark = pytest.mark.gpu


def _case(M, N, K, seed=0):
    g = gen(seed)
    xq, xs = quant_rows(torch.randn(M, K, generator=g))
    wq, ws = quant_tiles(0.02 * torch.randn(N, K, generator=g))
    return xq, xs, wq, ws


def check(y, xq, xs, wq, ws):
    """Each output is a sum of K products, those of a block added by the matrix core
    (``product_slack``), the blocks one after another and at most 64 parts of K at the end,
    a block's scale rounded once; then y's own rounding."""
    X, W = rows64(xq, xs), tiles64(wq, ws)
    want = X @ W.t()
    size = X.abs() @ W.abs().t()
    own = BF16 if y.dtype == torch.bfloat16 else U
    slack = product_slack(X, W) + (xq.shape[1] / 128 + 64 + 2) * U * size
    bound = want.abs() * own + slack * (1 + own) + TINY
    within(y, want, bound)


SIZES = [
    (1, 128, 128), (1, 16, 128), (1, 1, 256), (2, 17, 128), (1, 7168, 2048), (3, 200, 640), (16, 256, 1024),
    (13, 576, 7168), (17, 129, 384), (31, 130, 512), (33, 1000, 1280), (64, 640, 2048), (65, 384, 256),
    (100, 2112, 1536), (127, 128, 4096), (128, 257, 128), (129, 512, 896), (200, 64, 8192), (255, 255, 640),
    (257, 1024, 512), (333, 4096, 2048), (512, 320, 2176), (1000, 777, 640), (1025, 2048, 256), (2048, 1280, 1024),
    (3000, 130, 384), (2300, 4098, 512), (300, 6000, 384), (700, 3001, 512), (4101, 4098, 256), (4200, 4224, 640),
    (16385, 1030, 128), (30, 64, 16384), (4095, 4090, 384), (3900, 3841, 640), (4096, 4096, 128),
]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_product(M, N, K, out):
    xq, xs, wq, ws = _case(M, N, K)
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    y = ops.moe_linear_fp8(xq.cuda(), xs.cuda(), weights, out_dtype=out)
    assert y.shape == (M, N) and y.dtype == out
    check(y, xq, xs, wq, ws)


def _unpack(weights):
    """Row-major codes [N, K] of packed weights."""
    N, K = weights.N, weights.K
    n = -(-N // 16)
    t = weights.packed.cpu().reshape(n, K // 128, 2, 4, 16, 16)      # tile, block, half, lane / 16, row, byte
    return t.permute(0, 4, 1, 2, 3, 5).reshape(n * 16, K)[:N]


@pytest.mark.parametrize("N,K", [(128, 128), (256, 640), (384, 256)])
def test_packing(N, K):
    _, _, wq, ws = _case(1, N, K)
    a = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    assert torch.equal(_unpack(a), wq) and torch.equal(a.scales.cpu(), ws)
    t = ops.linear_weights_from_codes(wq.cuda().view(torch.float8_e4m3fn), ws.cuda(), transpose=True)
    assert (t.N, t.K) == (K, N)
    assert torch.equal(_unpack(t), wq.t()) and torch.equal(t.scales.cpu(), ws.t())


@pytest.mark.parametrize("N,K", [(1, 128), (17, 256), (300, 384), (256, 512)])
def test_packing_bf16(N, K):
    """The codes and tile scales of the expert weights' quantizer, a tile at the edge
    from the rows that it has."""
    w = (0.02 * torch.randn(N, K, generator=gen(3))).bfloat16()
    if N > 16:
        w[:, 128:256] = 0                                            # tiles of zeros
        w[5] *= 100
    a = ops.linear_weights(w.cuda())
    wq, ws = quant_tiles(w.float())
    assert torch.equal(a.scales.cpu(), ws)
    assert torch.equal(e4m3(_unpack(a)), e4m3(wq))
    if N % 128 == 0:
        t = ops.linear_weights(w.cuda(), transpose=True)
        assert torch.equal(e4m3(_unpack(t)), e4m3(wq.t().contiguous())) and torch.equal(t.scales.cpu(), ws.t())
        _, _, q2, s2 = ops.moe_pack_ffn_weights_fp8(None, w.cuda()[None])
        assert torch.equal(s2.cpu().reshape(ws.shape), ws)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_packing_what_is_not_finite(bad):
    """Its tile has no scale: NaN, and so has every output that the tile is part of."""
    w = (0.02 * torch.randn(384, 512, generator=gen(5))).bfloat16()
    clean = ops.linear_weights(w.cuda())
    w[200, 300] = bad
    a = ops.linear_weights(w.cuda())
    assert torch.isnan(a.scales[1, 2]) and (_unpack(a)[128:256, 256:384] == 0x7F).all()
    rest = torch.ones(3, 4, dtype=torch.bool)
    rest[1, 2] = False
    assert torch.equal(a.scales.cpu()[rest], clean.scales.cpu()[rest])
    x = ops.moe_quant_rows_fp8(torch.randn(40, 512, generator=gen(6)).bfloat16().cuda())
    y, z = ops.moe_linear_fp8(*x, a), ops.moe_linear_fp8(*x, clean)
    assert torch.isnan(y[:, 128:256]).all()
    assert torch.equal(y[:, :128], z[:, :128]) and torch.equal(y[:, 256:], z[:, 256:])


def test_rows_past_n_are_zero():
    _, _, wq, ws = _case(1, 20, 128)
    packed = ops.linear_weights_from_codes(wq.cuda(), ws.cuda()).packed.cpu().reshape(2, 2, 4, 16, 16)
    assert (packed[1, :, :, 4:] == 0).all()


@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (50, 384, 256), (300, 512, 1024)])
def test_gradient_of_the_rows(M, N, K):
    """dx = dy W on transposed weights: against the formula, and against differences of
    the loss sum(dy y), which is linear in x (any step gives the same difference)."""
    g = gen(4)
    _, _, wq, ws = _case(1, N, K)
    dy = torch.randn(M, N, generator=g).bfloat16()
    dq, ds = ops.moe_quant_rows_fp8(dy.cuda())
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda(), transpose=True)
    dx = ops.moe_linear_fp8(dq, ds, weights, out_dtype=torch.float32)
    check(dx, dq.cpu(), ds.cpu(), wq.t().contiguous(), ws.t().contiguous())
    W, D = tiles64(wq, ws), rows64(dq.cpu(), ds.cpu())
    loss = lambda X: (D * (X @ W.t())).sum()  # noqa: E731
    X = torch.randn(M, K, generator=g, dtype=torch.float64)
    for m, k in [(0, 0), (M - 1, K - 1), (M // 2, 130)]:
        E = torch.zeros_like(X)
        E[m, k] = 1.0
        diff = float((loss(X + E) - loss(X - E)) / 2)
        size = float((D[m].abs() * W[:, k].abs()).sum())
        slack = float(product_slack(D[m:m + 1], W[:, k:k + 1].t()))
        assert abs(float(dx[m, k]) - diff) <= slack + (N / 128 + 66) * U * size + 1e-9 * abs(float(loss(X)))


def test_wide_scales_and_given_output():
    M, N, K = 70, 260, 512
    xq, xs, wq, ws = _case(M, N, K)
    wide = torch.full((K // 128, M + 37), float("nan"))
    wide[:, :M] = xs
    y = torch.empty(M + 2, N, dtype=torch.bfloat16, device="cuda").fill_(7)
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    got = ops.moe_linear_fp8(xq.cuda(), wide.cuda(), weights, y=y[:M])
    assert got.data_ptr() == y.data_ptr() and (y[M:] == 7).all()
    check(got, xq, xs, wq, ws)


@pytest.mark.parametrize("M", [5, 40, 200, 1500])
@pytest.mark.parametrize("N", [255, 1024])
def test_a_nan_stays_in_its_row(M, N):
    K = 1024
    xq, xs, wq, ws = _case(M, N, K)
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    clean = ops.moe_linear_fp8(xq.cuda(), xs.cuda(), weights)
    xq[2, 700] = 0x7F
    xs[3, M - 1] = float("nan")
    xs[0, 1] = float("inf")
    y = ops.moe_linear_fp8(xq.cuda(), xs.cuda(), weights)
    rest = [m for m in range(M) if m not in (1, 2, M - 1)]
    assert torch.equal(y[rest], clean[rest])
    assert torch.isnan(y[2]).all() and torch.isnan(y[M - 1]).all() and not torch.isfinite(y[1]).any()


def test_zero_rows_and_zero_tiles():
    M, N, K = 40, 300, 512
    xq, xs, wq, ws = _case(M, N, K)
    xq[7], xs[:, 7] = 0, 0
    wq[128:256], ws[1] = 0, 0
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    y = ops.moe_linear_fp8(xq.cuda(), xs.cuda(), weights)
    assert (y[7] == 0).all() and (y[:, 128:256] == 0).all()
    check(y, xq, xs, wq, ws)


def test_no_rows():
    _, _, wq, ws = _case(1, 128, 128)
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    x = torch.empty(0, 128, dtype=torch.uint8, device="cuda")
    assert ops.moe_linear_fp8(x, torch.empty(1, 0, device="cuda"), weights).shape == (0, 128)


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (13, 576, 7168), (200, 640, 2048), (1100, 1024, 512)])
def test_equal_calls_give_equal_bits_on_any_stream_and_in_a_graph(M, N, K):
    xq, xs, wq, ws = (t.cuda() for t in _case(M, N, K))
    weights = ops.linear_weights_from_codes(wq, ws)
    first = ops.moe_linear_fp8(xq, xs, weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = ops.moe_linear_fp8(xq, xs, weights, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    need = ops.moe_linear_fp8_workspace_bytes(M, N, K)
    work = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_linear_fp8(xq, xs, weights, y=y, workspace=work)
    for k in range(3):
        xq.copy_(_case(M, N, K, seed=30 + k)[0])
        work.fill_(255)                                              # what is in the workspace does not count
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ops.moe_linear_fp8(xq, xs, weights))


def test_two_calls_at_once():
    a, b = _case(300, 512, 2048, 1), _case(300, 512, 2048, 2)
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    dev = [[t.cuda() for t in c] for c in (a, b)]
    packed = [ops.linear_weights_from_codes(c[2], c[3]) for c in dev]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [ops.moe_linear_fp8(c[0], c[1], w, stream=s) for c, w, s in zip(dev, packed, streams)]
    torch.cuda.synchronize()
    for y, c in zip(outs, (a, b)):
        check(y, *c)


def test_the_norm_feeds_the_product():
    """As they are used: the stream's norm writes the codes that the product reads."""
    g = gen(8)
    T, H, N = 130, 1024, 300
    x, res = torch.randn(T, H, generator=g).bfloat16(), torch.randn(T, H, generator=g).bfloat16()
    w = torch.ones(H).bfloat16()
    wq, ws = quant_tiles(0.02 * torch.randn(N, H, generator=g))
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    n = ops.moe_rmsnorm(x.cuda(), w.cuda(), residual=res.cuda(), y=False, codes=True)
    y = ops.moe_linear_fp8(n.codes, n.scales, weights)
    check(y, n.codes.cpu(), n.scales.cpu(), wq, ws)
    h = (x.float() + res.float()).bfloat16().double()
    v = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)
    W = tiles64(wq, ws)
    # the codes are each off by at most 2^-4 of the value (or 2^-10 of the scale, which is at
    # most amax / 448): the outputs by that times |v| |W|
    s = v.reshape(T, -1, 128).abs().amax(2).repeat_interleave(128, 1) / 448
    off = torch.maximum(v.abs() * 2.0 ** -4, s * 2.0 ** -10) * 1.001
    within(y, v @ W.t(), (off @ W.abs().t() + product_slack(v, W)) * (1 + BF16) + BF16 * (v @ W.t()).abs() + 1e-5)


def _random_codes(*shape):
    """E4M3 codes without NaN, made on the GPU."""
    return torch.randint(0, 0x70, shape, dtype=torch.uint8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))


def test_rows_past_32_bits():
    """4.4e9 codes of x: the last rows against the same rows alone (bit for bit: both
    calls take the same tiles)."""
    M, N, K = 1_100_000, 130, 4096
    x, xs = _random_codes(M, K), torch.ones(K // 128, M, device="cuda")
    _, _, wq, ws = _case(1, N, K)
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    y = ops.moe_linear_fp8(x, xs, weights)
    tail = x[-5:].contiguous()
    check(y[-5:], tail.cpu(), torch.ones(K // 128, 5), wq, ws)
    check(y[:5], x[:5].cpu(), torch.ones(K // 128, 5), wq, ws)


@pytest.mark.parametrize("M", [3, 40])
def test_weights_past_32_bits(M):
    """4.5e9 codes of W: its last rows."""
    N, K = 1 << 20, 4352
    codes, scales = _random_codes(N, K), torch.rand(N // 128, K // 128, device="cuda") + 0.5
    weights = ops.linear_weights_from_codes(codes, scales)
    xq, xs, _, _ = _case(M, 16, K)
    y = ops.moe_linear_fp8(xq.cuda(), xs.cuda(), weights)
    last = slice(N - 128, N)
    check(y[:, last], xq, xs, codes[last].cpu(), scales[-1:].cpu())
    check(y[:, :128], xq, xs, codes[:128].cpu(), scales[:1].cpu())


@pytest.mark.parametrize("M,N,K", [(17, 64, 128), (333, 4096, 2048), (2048, 1280, 1024)])
def test_without_a_workspace_where_none_is_used(M, N, K):
    """In one part: the C call takes NULL, the binding allocates the output alone."""
    xq, xs, wq, ws = _case(M, N, K)
    weights = ops.linear_weights_from_codes(wq.cuda(), ws.cuda())
    assert ops.moe_linear_fp8_parts(M, N, K)[0] == 1
    x, s, y = xq.cuda(), xs.cuda(), torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    status = load().moe_linear_fp8(x.data_ptr(), s.data_ptr(), M, M, N, K, weights.packed.data_ptr(),
                                   weights.scales.data_ptr(), 0, y.data_ptr(), None, 0,
                                   torch.cuda.current_stream().cuda_stream)
    assert status == 0
    made = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]  # noqa: E731
    before = made()
    z = ops.moe_linear_fp8(x, s, weights)
    assert made() == before + 1
    assert torch.equal(y, z)
    check(y, xq, xs, wq, ws)
