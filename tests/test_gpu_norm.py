"""moe_rmsnorm and its gradient against the formulas in 64 bits."""

import pytest
import torch

from combine_top_route_moe_amd import ops
from tests.around_util import BF16, TINY, U, e4m3, gen, rows64, within

pytestmark = pytest.mark.gpu
EPS = 1e-6

# one wave a row to 2048 channels, four to 8192, sixteen beyond; rows of 4, 5 and more a
# workgroup; widths that leave some of the threads without a vector
SHAPES = [(1, 128), (1, 2048), (3, 384), (5, 2048), (333, 640), (4, 2176), (17, 4096), (64, 7168), (2, 8192),
          (3, 8320), (5, 16384), (2, 32768), (4097, 256)]


def _inputs(T, H, seed=0, f32=False):
    g = gen(seed)
    x = torch.randn(T, H, generator=g).bfloat16()
    res = (3 * torch.randn(T, H, generator=g)).bfloat16()
    w = 1 + 0.2 * torch.randn(H, generator=g)
    return x, res, w if f32 else w.bfloat16()


def _formula(x, res, w, eps=EPS):
    h = x if res is None else (x.float() + res.float()).bfloat16()
    r = 1 / torch.sqrt(h.double().square().mean(1) + eps)
    return h, r, h.double() * r[:, None] * w.double()


def check_forward(out, h, r, v):
    """A sum of H squares has at most 64 additions one after another (32 in a
    thread, its row of lanes, the wave's four, 16 waves), so r is off by at most 32
    + 5 roundings; v by three more, a scale by one more."""
    if out.h is not None:
        assert torch.equal(out.h.cpu().view(torch.int16), h.view(torch.int16))
    if out.rstd is not None:
        within(out.rstd, r, 40 * U * r, "rstd")
    if out.y is not None:
        within(out.y, v, v.abs() * (BF16 + 48 * U) + TINY, "y")
    if out.codes is not None:
        T, H = v.shape
        t = v.reshape(T, H // 128, 128)
        s = t.abs().amax(2) / 448
        within(out.scales[:, :T].t(), s, 48 * U * s + 2.0 ** -149, "scales")
        got = rows64(out.codes, out.scales)
        half = torch.maximum(t.abs() * 2.0 ** -4, s[:, :, None] * 2.0 ** -10) * (1 + 2.0 ** -16)
        within(got, v, (half + t.abs() * 2.0 ** -16 + 2.0 ** -140).reshape(T, H), "codes")


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual,f32", [(True, False), (False, True)])
def test_forward(T, H, residual, f32):
    x, res, w = _inputs(T, H, f32=f32)
    res = res if residual else None
    out = ops.moe_rmsnorm(x.cuda(), w.cuda(), EPS, residual=None if res is None else res.cuda(), y=True, codes=True,
                          rstd=True)
    assert (out.h is None) == (res is None)
    check_forward(out, *_formula(x, res, w))


def _nearest_codes(p):
    """E4M3 values nearest to 448 p / amax |p| per 128 channels, half way to the even one.
    p in float64 is exact (8 + 24 bits), and so are both sides of the comparison with
    a midpoint: 448 p has 41 bits, a midpoint of 5 times the largest 37."""
    T, H = p.shape
    t = p.reshape(T, H // 128, 128)
    top = t.abs().amax(2, keepdim=True)
    q = (448 * t).abs() / torch.where(top > 0, top, torch.ones_like(top))
    step = torch.exp2((torch.frexp(q).exponent - 4).clamp(min=-9).double())
    low = torch.floor(q / step)
    over = (448 * t).abs() - (low + 0.5) * step * top
    return ((low + ((over > 0) | ((over == 0) & (low % 2 == 1)))) * step * t.sign()).reshape(T, H)


@pytest.mark.parametrize("T,H", [(333, 640), (64, 7168), (5, 16384), (4097, 256)])
@pytest.mark.parametrize("gain", ["bf16", "f32", "f32 of few bits", "ones"])
def test_codes_are_the_nearest(T, H, gain):
    """Not one code on the wrong side, half-way quotients included (a bf16 gain and a gain
    of few bits have thousands of them)."""
    x, _, w = _inputs(T, H, f32=True)
    w = {"bf16": w.bfloat16(), "f32": w, "f32 of few bits": w.bfloat16().float(), "ones": torch.ones(H)}[gain]
    out = ops.moe_rmsnorm(x.cuda(), w.cuda(), EPS, y=False, codes=True)
    assert torch.equal(e4m3(out.codes.cpu()).double(), _nearest_codes(x.double() * w.double()))


@pytest.mark.parametrize("want", ["y", "codes", "rstd", "h"])
def test_one_output(want):
    x, res, w = _inputs(37, 1024)
    kw = {"y": False, "h": False} | {want: True}
    out = ops.moe_rmsnorm(x.cuda(), w.cuda(), EPS, residual=res.cuda(), **kw)
    assert [k for k in ("h", "y", "codes", "rstd") if getattr(out, k) is not None] == [want]
    check_forward(out, *_formula(x, res, w))


def test_codes_are_those_of_the_row_quantizer_where_v_is_bf16():
    """With a gain of powers of two and rows of +-1 (r = 1 but for eps), v is a bf16
    number, and the codes and scales are bit for bit moe_quant_rows_fp8's."""
    g = gen(1)
    x = torch.where(torch.rand(9, 512, generator=g) < 0.5, 1.0, -1.0).bfloat16().cuda()
    w = torch.exp2(torch.randint(-8, 8, (512,), generator=g).float()).cuda()
    out = ops.moe_rmsnorm(x, w, 1e-30, y=True, codes=True, rstd=True)
    assert torch.equal(out.rstd, torch.ones_like(out.rstd))
    codes, scales = ops.moe_quant_rows_fp8(out.y)
    assert torch.equal(out.codes, codes) and torch.equal(out.scales, scales)


def test_wide_scales_keep_what_lies_past_the_rows():
    x, res, w = _inputs(5, 256)
    scales = torch.full((2, 9), 7.0, device="cuda")
    out = ops.moe_rmsnorm(x.cuda(), w.cuda(), EPS, codes=True, scales=scales)
    assert out.scales is scales and (scales[:, 5:] == 7).all()
    check_forward(out, *_formula(x, None, w))


@pytest.mark.parametrize("T,H", [(7, 2048), (6, 4096), (3, 16384)])
@pytest.mark.parametrize("where", ["residual", "x"])
def test_in_place(T, H, where):
    x, res, w = _inputs(T, H)
    xd, rd = x.cuda(), res.cuda()
    h = rd if where == "residual" else xd
    out = ops.moe_rmsnorm(xd, w.cuda(), EPS, residual=rd, h=h, y=xd if where == "residual" else True, codes=True)
    assert out.h.data_ptr() == h.data_ptr()
    check_forward(out, *_formula(x, res, w))


def test_large_and_small_rows():
    """Rows of zeros, of one channel, of tiny and of large numbers side by side."""
    x = torch.zeros(6, 256)
    x[1, 5] = 3.0
    x[2] = 1e-30 * torch.randn(256, generator=gen(2))
    x[3] = 1e15 * torch.randn(256, generator=gen(3))
    x[4, :128] = torch.randn(128, generator=gen(4))
    x[5] = 1e-3
    x = x.bfloat16()
    w = torch.ones(256).bfloat16()
    out = ops.moe_rmsnorm(x.cuda(), w.cuda(), EPS, y=True, codes=True, rstd=True)
    check_forward(out, *_formula(x, None, w))
    assert (out.codes[0] == 0).all() and (out.scales[:, 0] == 0).all() and (out.scales[1, 4] == 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_row_and_shows(bad):
    x, _, w = _inputs(7, 2304)
    clean = ops.moe_rmsnorm(x.cuda(), w.cuda(), EPS, codes=True, rstd=True)
    x[3, 1000] = bad
    out = ops.moe_rmsnorm(x.cuda(), w.cuda(), EPS, codes=True, rstd=True)
    rows = [0, 1, 2, 4, 5, 6]
    for a, b in ((out.y, clean.y), (out.codes, clean.codes), (out.scales.t(), clean.scales.t()), (out.rstd, clean.rstd)):
        assert torch.equal(a[rows], b[rows])
    assert torch.isnan(out.y[3, 1000])
    values = rows64(out.codes, out.scales)[3]
    block = slice(896, 1024)
    assert torch.isnan(values[block]).all() and torch.isnan(out.scales[7, 3])


def test_no_rows():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    out = ops.moe_rmsnorm(x, w, EPS, codes=True, rstd=True)
    assert out.y.shape == (0, 256) and out.rstd.shape == (0,)
    dx, dw = ops.moe_rmsnorm_backward(x, x, out.rstd, w)
    assert dx.shape == (0, 256) and (dw == 0).all()


def _gradient64(dy, h, r, w, dh):
    hat = h.double() * r.double()[:, None]
    g = dy.double() * w.double()
    c = (g * hat).mean(1, keepdim=True)
    dx = r.double()[:, None] * (g - hat * c)
    # every float32 step's share: g, hat and their product once each, the mean's sum by at
    # most 64 additions, the last additions
    r = r.double()[:, None]
    slack = r * (4 * g.abs() + hat.abs() * (80 * (g * hat).abs().mean(1, keepdim=True) + 4 * c.abs())) * U
    if dh is not None:
        dx, slack = dx + dh.double(), slack + dh.double().abs() * U
    return dx, dx.abs() * (BF16 + U) + slack * (1 + BF16) + TINY, (dy.double() * hat).sum(0), (dy.double() * hat).abs().sum(0)


@pytest.mark.parametrize("T,H", SHAPES + [(20000, 128), (1500, 4096), (300, 9216), (1024, 384), (1025, 384),
                                        (700, 16384), (5000, 1024), (3000, 1536), (1300, 7168), (1030, 2176), (1100, 20480)])
@pytest.mark.parametrize("residual,f32", [(True, True), (False, False)])
def test_backward(T, H, residual, f32):
    x, res, w = _inputs(T, H, f32=f32)
    g = gen(9)
    dy = torch.randn(T, H, generator=g).bfloat16()
    dh = torch.randn(T, H, generator=g).bfloat16() if residual else None
    r = (1 / torch.sqrt(x.double().square().mean(1) + EPS)).float()
    dx, dw = ops.moe_rmsnorm_backward(dy.cuda(), x.cuda(), r.cuda(), w.cuda(),
                                      d_residual=None if dh is None else dh.cuda())
    want, bound, want_w, size = _gradient64(dy, x, r, w, dh)
    within(dx, want, bound, "dx")
    # up to 1024 rows each 32nd in a thread (32 additions), 32 threads (wide rows: 8 and 128);
    # else at most 12 rows of a workgroup's share one after another up to 20000 rows, four
    # waves, 512 / 32 shares in a thread and 32 threads; two roundings of a term
    within(dw, want_w, (8 + 128 + 2) * U * size + 2.0 ** -140, "dw")


def test_backward_against_differences():
    T, H = 3, 256
    x, _, w = _inputs(T, H, f32=True)
    dy = torch.randn(T, H, generator=gen(5)).bfloat16()
    f = lambda x, w: ((x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * w) * dy.double()).sum()  # noqa: E731
    out = ops.moe_rmsnorm(x.cuda(), w.cuda(), EPS, rstd=True)
    dx, dw = ops.moe_rmsnorm_backward(dy.cuda(), x.cuda(), out.rstd, w.cuda())
    d, X, W = 1e-5, x.double(), w.double()
    for t, c in [(0, 0), (0, 255), (1, 77), (2, 128)]:
        e = torch.zeros(T, H, dtype=torch.float64)
        e[t, c] = d
        diff = (f(X + e, W) - f(X - e, W)) / (2 * d)
        # third derivatives are of order one here: the difference is right to d^2 and 1e-16 / d
        assert abs(float(dx[t, c]) - float(diff)) <= BF16 * abs(float(diff)) + 1e-5
    for c in (0, 130, 255):
        e = torch.zeros(H, dtype=torch.float64)
        e[c] = d
        diff = (f(X, W + e) - f(X, W - e)) / (2 * d)
        assert abs(float(dw[c]) - float(diff)) <= 1e-5


@pytest.mark.parametrize("where", ["dy", "d_residual"])
@pytest.mark.parametrize("T,H", [(9, 1024), (9, 4096), (3000, 1024), (1300, 4096)])
def test_backward_in_place(where, T, H):
    x, dy, w = _inputs(T, H)
    dh = torch.randn(T, H, generator=gen(6)).bfloat16()
    r = (1 / torch.sqrt(x.double().square().mean(1) + EPS)).float()
    a, b = dy.cuda(), dh.cuda()
    dx, _ = ops.moe_rmsnorm_backward(a, x.cuda(), r.cuda(), w.cuda(), d_residual=b, dx=a if where == "dy" else b)
    want, bound, _, _ = _gradient64(dy, x, r, w, dh)
    within(dx, want, bound)


def test_equal_calls_give_equal_bits():
    x, res, w = (t.cuda() for t in _inputs(3000, 2048))
    r = torch.rand(3000, device="cuda") + 0.5
    first = ops.moe_rmsnorm_backward(res, x, r, w)
    for _ in range(3):
        again = ops.moe_rmsnorm_backward(res, x, r, w)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_captured_and_replayed():
    x, res, w = (t.cuda() for t in _inputs(50, 4096))
    dy = torch.randn(50, 4096, generator=gen(7)).bfloat16().cuda()
    out = ops.moe_rmsnorm(x, w, EPS, residual=res, codes=True, rstd=True)
    ws = torch.empty(ops.moe_rmsnorm_backward_workspace_bytes(50, 4096), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(4096, device="cuda")

    def both():
        ops.moe_rmsnorm(x, w, EPS, residual=res, h=out.h, y=out.y, codes=out.codes, scales=out.scales, rstd=out.rstd)
        ops.moe_rmsnorm_backward(dy, out.h, out.rstd, w, dx=dx, d_weight=dw, workspace=ws)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        x.copy_(torch.randn(50, 4096, generator=gen(20 + k)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out.h, out.y, out.codes, out.scales, out.rstd, dx, dw)]
        both()
        assert all(torch.equal(a, b) for a, b in zip(got, (out.h, out.y, out.codes, out.scales, out.rstd, dx, dw)))


def test_on_another_stream():
    x, res, w = (t.cuda() for t in _inputs(200, 2048))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = ops.moe_rmsnorm(x, w, EPS, residual=res, codes=True, rstd=True, stream=side)
    dx, dw = ops.moe_rmsnorm_backward(res, out.h, out.rstd, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    here = ops.moe_rmsnorm(x, w, EPS, residual=res, codes=True, rstd=True)
    hx, hw = ops.moe_rmsnorm_backward(res, here.h, here.rstd, w)
    for a, b in ((out.y, here.y), (out.codes, here.codes), (out.scales, here.scales), (dx, hx), (dw, hw)):
        assert torch.equal(a, b)
    assert float(e4m3(out.codes).abs().max()) == 448


def test_offsets_past_32_bits():
    """2.2e9 channels: the last rows, forward and backward, against the same rows alone."""
    T, H = 270_000, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.ones(H, device="cuda")
    out = ops.moe_rmsnorm(x, w, EPS, y=False, codes=True, rstd=True)
    some = ops.moe_rmsnorm(x[-3:].contiguous(), w, EPS, codes=True, rstd=True)
    assert torch.equal(out.codes[-3:], some.codes) and torch.equal(out.scales[:, -3:], some.scales)
    assert torch.equal(out.rstd[-3:], some.rstd)
    del out.codes
    dx, dw = ops.moe_rmsnorm_backward(x, x, out.rstd, w)
    few, _ = ops.moe_rmsnorm_backward(x[-3:].contiguous(), x[-3:].contiguous(), some.rstd, w)
    assert torch.equal(dx[-3:], few) and torch.isfinite(dw).all()
