"""A layer with the norm in front of it, its router's product and losses: the
operators one after another, as a model uses them."""

import pytest
import torch

from combine_top_route_moe_amd import MoELayer, ops
from tests.around_util import gen, quant_tiles, rows64, tiles64

pytestmark = pytest.mark.gpu
T, H, E, K, I = 96, 512, 16, 4, 256


def _layer(fp8=False, shared=False):
    g = gen(1)
    layer = MoELayer(T, H, E, K, I, shared_I=I if shared else 0)
    w = lambda *s: (0.05 * torch.randn(*s, generator=g)).bfloat16().cuda()  # noqa: E731
    args = [w(E, 2 * I, H), w(E, H, I)]
    if shared:
        args += [w(2 * I, H), w(H, I)]
    layer.set_weights(*args, fp8=fp8)
    return layer


def _inputs(seed=2):
    g = gen(seed)
    x, res = torch.randn(T, H, generator=g).bfloat16().cuda(), (2 * torch.randn(T, H, generator=g)).bfloat16().cuda()
    return x, res, (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda(), torch.randn(T, E, generator=g).cuda()


@pytest.mark.parametrize("shared", [False, True])
def test_norm_then_forward(shared):
    layer, (x, res, w, logits) = _layer(shared=shared), _inputs()
    plain = ops.moe_rmsnorm(x, w, residual=res)
    want = layer.forward(logits, plain.y).clone()
    rows = layer.norm(x, w, residual=res)
    assert torch.equal(rows, plain.y) and torch.equal(res, plain.h)           # the stream in place
    assert torch.equal(layer.forward(logits, None), want)


@pytest.mark.parametrize("shared", [False, True])
def test_norm_then_the_fp8_path(shared):
    """The codes of the norm are what the experts read: bit for bit the layer's other
    stages on them, and no row quantizer runs."""
    layer, (x, res, w, logits) = _layer("w8a8", shared), _inputs()
    n = ops.moe_rmsnorm(x, w, residual=res, codes=True)
    other = _layer("w8a8", shared)
    other.hq.copy_(n.codes), other.hs.copy_(n.scales)
    for name, enqueue in other.stages(logits, n.y):
        if name != "dispatch_quant":
            enqueue()
    layer.norm(x, w, residual=res, h=torch.empty_like(res))
    assert "dispatch_quant" not in [name for name, _ in layer.stages(logits, None)]
    assert torch.equal(layer.forward(logits, None), other.out)
    layer.forward(logits, n.h)                       # rows of its own are quantized beside the norm's
    assert torch.equal(layer.forward(logits, None), other.out)


def test_norm_then_decode():
    layer, (x, res, w, logits) = _layer(), _inputs()
    rows = layer.norm(x[:5], w, residual=res[:5])
    got = layer.decode(logits[:5], rows).clone()
    assert torch.equal(got, layer.decode(logits[:5], rows.clone()))
    with pytest.raises(ValueError, match="all of the layer's rows"):
        layer.forward(logits, None)


def test_refusals():
    layer, (x, res, w, logits) = _layer(), _inputs()
    with pytest.raises(ValueError, match="norm"):
        layer.forward(logits, None)
    with pytest.raises(ValueError, match="x must be"):
        layer.norm(torch.cat([x, x]), w)
    layer.norm(x, w)
    layer.set_weights(torch.zeros(E, 2 * I, H).bfloat16().cuda(), torch.zeros(E, H, I).bfloat16().cuda(), fp8="w8a8")
    with pytest.raises(ValueError, match="call it again"):
        layer.forward(logits, None)


def test_a_block_in_training_captured_and_replayed():
    """Stream -> norm with codes -> router's product on the codes -> layer -> losses -> the
    router's gradient -> its rows' gradient -> the norm's gradient, in one graph."""
    layer = _layer("w8a8", shared=True)
    x, res, w, _ = _inputs()
    wq, ws = quant_tiles(0.2 * torch.randn(128, H, generator=gen(3)))
    wq[E:] = 0
    router = ops.linear_weights_from_codes(wq[:E].contiguous().cuda(), ws.cuda())
    back = ops.linear_weights_from_codes(wq.cuda(), ws.cuda(), transpose=True)     # [H, 128]: rows past E are zero
    n = ops.moe_rmsnorm(x, w, residual=res, codes=True, rstd=True)
    logits = torch.empty(T, E, device="cuda")
    d_topk_w = torch.randn(T, K, generator=gen(4)).cuda()
    d_loss = torch.tensor([0.1, 0.01], device="cuda")
    padded = torch.zeros(T, 128, dtype=torch.bfloat16, device="cuda")
    dq, ds = ops.moe_quant_rows_fp8(padded)
    losses = ops.moe_balance_loss(logits.zero_(), torch.zeros(T, K, dtype=torch.int32, device="cuda"))
    dl, dy = torch.empty_like(logits), torch.empty_like(x)
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    work = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def step():
        ops.moe_rmsnorm(x, w, residual=res, h=n.h, y=n.y, codes=n.codes, scales=n.scales, rstd=n.rstd)
        layer.norm(x, w, residual=res, h=n.h)
        ops.moe_linear_fp8(n.codes, n.scales, router, y=logits, workspace=work)
        layer.forward(logits, None)
        ops.moe_balance_loss(logits, layer.topk_idx, out=losses, workspace=work, dev_error=layer.dev_error)
        layer.route_backward(logits, d_topk_w, d_loss=d_loss, losses=losses, d_logits=dl)
        padded[:, :E].copy_(dl)
        ops.moe_quant_rows_fp8(padded, None, dq, ds)
        ops.moe_linear_fp8(dq, ds, back, y=dy, workspace=work)
        ops.moe_rmsnorm_backward(dy, n.h, n.rstd, w, d_residual=x, dx=dx, d_weight=dw, workspace=work)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (n.h, n.y, logits, layer.out, losses.loss, losses.counts, losses.probs, dl, dy, dx, dw)
    for k in range(3):
        x.copy_(torch.randn(T, H, generator=gen(30 + k)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs[2:]:
            t.zero_()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, outs))
    assert int(layer.dev_error) == 0
    # the logits are the codes' product with the router's weights
    want = rows64(n.codes, n.scales) @ tiles64(wq[:E], ws).t()
    assert float((logits.cpu().double() - want).norm() / want.norm()) < 1e-3      # 2^-11 of the sum, at worst
    assert int(losses.counts.sum()) == T * K


def test_stage_outputs_after_the_norm_hold_its_codes():
    layer, (x, res, w, logits) = _layer("w8a8", True), _inputs()
    n = ops.moe_rmsnorm(x, w, codes=True)
    layer.norm(x, w)
    layer.forward(logits, None)
    outs = layer.stage_outputs()
    assert torch.equal(outs["hidden_codes"], n.codes) and torch.equal(outs["hidden_scales"], n.scales)
    layer.forward(logits, res)
    codes, scales = ops.moe_quant_rows_fp8(res)
    outs = layer.stage_outputs()
    assert torch.equal(outs["hidden_codes"], codes) and torch.equal(outs["hidden_scales"], scales)


@pytest.mark.parametrize("fp8", [False, "w8a8"])
@pytest.mark.parametrize("n", [5, T])
def test_the_gradient_of_the_layers_norm(fp8, n):
    """One norm a step: its gradient starts from what the layer's call wrote."""
    layer, (x, res, w, _) = _layer(fp8), _inputs()
    dy = torch.randn(n, H, generator=gen(7)).bfloat16().cuda()
    want = ops.moe_rmsnorm(x[:n], w, residual=res[:n], rstd=True)
    rstd, h = torch.full((T,), 7.0, device="cuda"), torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
    rows = layer.norm(x[:n], w, residual=res[:n], h=h, rstd=rstd[:n])
    assert torch.equal(rows, want.y) and torch.equal(rstd[:n], want.rstd) and (rstd[n:] == 7).all()
    for a, b in zip(ops.moe_rmsnorm_backward(dy, h, rstd[:n], w), ops.moe_rmsnorm_backward(dy, want.h, want.rstd, w)):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="rstd"):
        layer.norm(x[:n], w, rstd=rstd[: n - 1])


KINDS = [dict(dispatch_block=128), dict(combine_qdq=True), dict(dispatch_fp4="mxfp4"), dict(combine_fp4="mxfp4"),
         dict(fp8=True), dict(fp4="mxfp4"), dict(fp4="nvfp4"), dict(pack=False)]


def _layer_of(kw, shared=True):
    kw, g = dict(kw), gen(1)
    weights = {k: kw.pop(k) for k in ("fp8", "fp4", "pack") if k in kw}
    layer = MoELayer(T, H, E, K, I, shared_I=I if shared else 0, **kw)
    w = lambda *s: (0.05 * torch.randn(*s, generator=g)).bfloat16().cuda()  # noqa: E731
    layer.set_weights(w(E, 2 * I, H), w(E, H, I), *((w(2 * I, H), w(H, I)) if shared else ()), **weights)
    return layer


@pytest.mark.parametrize("kw", KINDS, ids=lambda kw: "-".join(f"{k}={v}" for k, v in kw.items()))
@pytest.mark.parametrize("shared", [False, True])
def test_norm_then_forward_of_any_kind(kw, shared):
    """Quantizers of the dispatched and of the combined rows, weights of every format: on the
    norm's rows as on the same rows given."""
    layer, (x, res, w, logits) = _layer_of(kw, shared), _inputs()
    valid = torch.ones(T, dtype=torch.uint8, device="cuda")
    valid[[3, 50]] = 0
    rows = ops.moe_rmsnorm(x, w, residual=res).y
    if layer.combine_scale is not None:
        layer.calibrate_combine_scale(logits, rows, valid)
    want = layer.forward(logits, rows, valid).clone()
    assert want.any()
    layer.norm(x, w, residual=res)
    layer.out.zero_()
    assert torch.equal(layer.forward(logits, None, valid), want) and int(layer.dev_error) == 0


def _router_check(layer, logits, valid, n):
    """The layer's losses and gradient against those of the operators on its routes."""
    idx, top = layer.topk_idx[:n].clone(), layer.topk_w[:n].clone()
    if valid is not None:
        assert (idx[valid == 0] == -1).all() and (valid == 0).any()
    want = ops.moe_balance_loss(logits, idx, valid)
    got = layer.balance_loss(logits, valid)
    for name in ("loss", "counts", "probs", "num_tokens"):
        assert torch.equal(getattr(got, name), getattr(want, name)), name
    real = n if valid is None else int(valid.sum())
    assert int(got.num_tokens) == real and int(got.counts.sum()) == real * K
    dw, d = torch.randn(n, K, generator=gen(4)).cuda(), torch.tensor([0.1, 0.01], device="cuda")
    a = layer.route_backward(logits, dw, valid, d_loss=d, losses=got)
    b = ops.moe_route_backward(logits, idx, top, dw, valid, d_loss=d, counts=want.counts, num_tokens=want.num_tokens)
    assert torch.equal(a, b) and a.shape == (n, E) and a.any()
    if valid is not None:
        assert not a[valid == 0].any()
    with pytest.raises(ValueError, match="counts"):
        layer.route_backward(logits, dw, valid, d_loss=d)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("n", [1, 7, 64, T])
def test_the_routers_training_behind_forward_and_decode(n, padded):
    """With padding, and for fewer tokens than the layer's: decode's."""
    layer, (x, _, _, logits) = _layer(shared=True), _inputs()
    valid = None
    if padded:
        valid = torch.ones(n, dtype=torch.uint8, device="cuda")
        valid[n // 2] = 0
    if n == T:
        layer.forward(logits, x, valid)
    else:
        layer.decode(logits[:n], x[:n], valid)
    if padded and n == 1:                                            # no token at all
        losses = layer.balance_loss(logits[:1], valid)
        assert not losses.loss.any() and not losses.counts.any() and int(losses.num_tokens) == 0
        return
    _router_check(layer, logits[:n].contiguous(), valid, n)
