"""moe_balance_loss and moe_route_backward against the formulas in 64 bits."""

import pytest
import torch

from combine_top_route_moe_amd import ops
from tests.around_util import U, gen, within

pytestmark = pytest.mark.gpu
INF = float("inf")


def _route(T, E, K, pad=0, renorm=True, seed=0, spread=1.0):
    g = gen(seed)
    logits = spread * torch.randn(T, E, generator=g) + torch.randn(E, generator=g)
    valid = None
    if pad:
        valid = torch.ones(T, dtype=torch.uint8)
        valid[torch.randperm(T, generator=g)[:pad]] = 0
    idx, w = ops.moe_route(logits.cuda(), K, None if valid is None else valid.cuda(), renorm)
    return logits, valid, idx, w


def _softmax64(logits):
    l = torch.where(torch.isnan(logits), -INF, logits.double())
    top = l.amax(1, keepdim=True)
    e = torch.where(l == top, 1.0, torch.exp(l - top))
    z = e.sum(1, keepdim=True)
    lse = (top + torch.log(z))[:, 0]
    span = torch.where(torch.isfinite(l - top), (top - l), torch.zeros_like(l))
    # a probability: the difference and two exponentials' ends (each |l - top| + 2 steps of
    # float32), a sum of at most 16 + 8 additions, two more roundings
    return e / z, lse, (2 * span.amax(1, keepdim=True) + 2 + 2 + 24 + 2) * U


def _losses64(logits, valid, idx, E, K):
    real = torch.ones(len(logits), dtype=torch.bool) if valid is None else valid.bool()
    n = int(real.sum())
    p, lse, rel = _softmax64(logits)
    ids = idx[real].flatten()
    counts = torch.bincount(ids[(ids >= 0) & (ids < E)].long(), minlength=E)
    m = max(n, 1)
    P = p[real].sum(0) / m
    fine = torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[real]
    return counts, n, P, E * (counts.double() * P).sum() / (m * K), fine.square().sum() / m, (p * rel)[real].sum(0) / m, fine


CASES = [(1, 1, 1, 0), (1, 2, 1, 0), (1, 64, 8, 0), (5, 7, 3, 1), (64, 64, 8, 0), (37, 65, 4, 9), (100, 128, 8, 13),
         (333, 200, 6, 50), (257, 256, 8, 0), (50, 300, 32, 3), (40, 512, 10, 0), (33, 1000, 4, 2), (20, 1024, 32, 0),
         (3000, 64, 8, 700), (5000, 33, 2, 0)]


@pytest.mark.parametrize("T,E,K,pad", CASES)
def test_losses(T, E, K, pad):
    logits, valid, idx, _ = _route(T, E, K, pad)
    r = ops.moe_balance_loss(logits.cuda(), idx, None if valid is None else valid.cuda())
    counts, n, P, balance, z, slack, lse = _losses64(logits, valid, idx.cpu(), E, K)
    assert torch.equal(r.counts.cpu(), counts.int()) and int(r.num_tokens) == n
    adds = T / 16 / min(128, -(-T // 16)) + 5                        # a wave's tokens, the waves of a workgroup
    within(r.probs, P, slack + (adds + 1) * U * P, "probs")
    bound = E * (counts.double() * (slack + (adds + 1) * U * P)).sum() / max(n * K, 1)
    within(r.loss[0], balance, bound + U * balance, "balance")
    # lse = top + log(sum): the log to two steps and the sum's error, both terms' roundings
    off = (lse.abs() + 32) * U + 2 * U * lse.abs()
    within(r.loss[1], z, (2 * lse.abs() * off + off ** 2).sum() / max(n, 1) + U * z, "z")


def test_even_routing_has_balance_one():
    logits = torch.zeros(64, 16, device="cuda")
    idx = (torch.arange(128, dtype=torch.int32, device="cuda") % 16).reshape(64, 2)
    r = ops.moe_balance_loss(logits, idx)
    assert float(r.loss[0]) == 1 and torch.equal(r.counts, torch.full_like(r.counts, 8))
    assert torch.equal(r.probs, torch.full_like(r.probs, 1 / 16))


def test_no_real_tokens():
    logits, idx = torch.randn(9, 40, device="cuda"), torch.full((9, 3), -1, dtype=torch.int32, device="cuda")
    none = torch.zeros(9, dtype=torch.uint8, device="cuda")
    for l, i, v in ((logits, idx, none), (logits[:0], idx[:0], None)):
        r = ops.moe_balance_loss(l, i, v)
        assert not r.loss.any() and not r.counts.any() and not r.probs.any() and not r.num_tokens.any()
        g = ops.moe_route_backward(l, i, torch.zeros_like(i).float(), torch.ones_like(i).float(), v,
                                   d_loss=torch.ones(2, device="cuda"), counts=r.counts, num_tokens=r.num_tokens)
        assert g.shape == l.shape and not g.any()


def test_ids_that_name_no_expert():
    logits = torch.randn(20, 10, generator=gen(1))
    idx = torch.randint(0, 10, (20, 3), generator=gen(2), dtype=torch.int32)
    idx[4, 1], idx[5, 0], idx[6] = -1, -7, -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = ops.moe_balance_loss(logits.cuda(), idx.cuda(), dev_error=err)
    assert torch.equal(r.counts.cpu(), torch.bincount(idx[idx >= 0].long(), minlength=10).int()) and int(err) == 0
    idx[7, 2], idx[8, 0] = 10, 2 ** 31 - 1
    r = ops.moe_balance_loss(logits.cuda(), idx.cuda(), dev_error=err)
    good = idx[(idx >= 0) & (idx < 10)]
    assert torch.equal(r.counts.cpu(), torch.bincount(good.long(), minlength=10).int())
    assert int(err) == ops.MOE_DEVERR_EXPERT_RANGE
    err.zero_()
    w, dw = torch.rand(20, 3, generator=gen(3)), torch.randn(20, 3, generator=gen(4))
    hole = (idx < 0) | (idx >= 10)
    w[hole], dw[hole] = float("nan"), INF                            # what lies there is not read into anything
    g = ops.moe_route_backward(logits.cuda(), idx.cuda(), w.cuda(), dw.cuda(), dev_error=err)
    assert int(err) == ops.MOE_DEVERR_EXPERT_RANGE
    want, bound = _gradient64(logits, None, idx, w, dw, True, None, None, 20)
    within(g, want, bound)


def _gradient64(logits, valid, idx, w, dw, renorm, d, counts, n):
    T, E = logits.shape
    K = idx.shape[1]
    p, lse, rel = _softmax64(logits)
    want = torch.zeros(T, E, dtype=torch.float64)
    bound = torch.zeros(T, E, dtype=torch.float64)
    if d is not None:
        m = max(n, 1)
        b = E * counts.double() / (m * K) - 1
        mean = (p * b).sum(1, keepdim=True)
        size = (p * (b.abs() + 2)).sum(1, keepdim=True)
        fine = torch.isfinite(lse)[:, None]
        z = torch.where(fine, lse[:, None], torch.zeros(1, dtype=torch.float64))
        d0, d1 = float(d[0]) / m, 2 * float(d[1]) / m
        want += torch.where(fine, p * (d0 * (b - mean) + d1 * z), 0.0)
        # each factor's share: the probability, the difference and the mean's sum (24
        # additions), the logsumexp, and some ten roundings of products
        bound += p * (abs(d0) * ((b - mean).abs() * (rel + 10 * U) + (b.abs() + 2) * 4 * U + size * (rel + 26 * U))
                      + abs(d1) * (z.abs() * (rel + 12 * U) + 32 * U))
    if dw is not None:
        on = (idx >= 0) & (idx < E)
        zero = torch.zeros(1, dtype=torch.float64)
        W, wd = torch.where(on, w.double(), zero), torch.where(on, w.double() * dw.double(), zero)
        dot, size = wd.sum(1, keepdim=True), wd.abs().sum(1, keepdim=True)
        part, off = wd, wd.abs() * 3 * U
        if renorm:
            part, off = wd - W * dot, off + (W * size).abs() * 12 * U + 2 * U * (wd.abs() + (W * dot).abs())
        else:
            want -= p * dot
            bound += p * (dot.abs() * (rel + 4 * U) + size * 10 * U)
        at = torch.where(on, idx, 0).long()
        many = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, at, part.abs())
        want.scatter_add_(1, at, part)
        bound.scatter_add_(1, at, off)
        bound += 4 * U * many
    bound += 4 * U * want.abs() + 2.0 ** -140
    if valid is not None:
        want[valid == 0], bound[valid == 0] = 0, 0
    return want, bound


@pytest.mark.parametrize("T,E,K,pad", CASES + [(10000, 16, 4, 100)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("what", ["both", "weights", "losses"])
def test_gradient(T, E, K, pad, renorm, what):
    logits, valid, idx, w = _route(T, E, K, pad, renorm)
    v = None if valid is None else valid.cuda()
    r = ops.moe_balance_loss(logits.cuda(), idx, v)
    dw = None if what == "losses" else torch.randn(T, K, generator=gen(5))
    d = None if what == "weights" else torch.tensor([0.7, -0.3])
    g = ops.moe_route_backward(logits.cuda(), idx, w, None if dw is None else dw.cuda(), v, renorm,
                               d_loss=None if d is None else d.cuda(), counts=r.counts, num_tokens=r.num_tokens)
    want, bound = _gradient64(logits, valid, idx.cpu(), w.cpu(), dw, renorm, d, r.counts.cpu(), T - pad)
    within(g, want, bound)


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    """Of a loss in 64 bits through the softmax and the chosen experts, which the step is
    too small to change."""
    T, E, K = 6, 12, 3
    logits, _, idx, w = _route(T, E, K, renorm=renorm, seed=3)
    r = ops.moe_balance_loss(logits.cuda(), idx)
    dw, d = torch.randn(T, K, generator=gen(6)), torch.tensor([0.5, 0.25])
    g = ops.moe_route_backward(logits.cuda(), idx, w, dw.cuda(), None, renorm, d_loss=d.cuda(), counts=r.counts,
                               num_tokens=r.num_tokens)
    f, at = r.counts.cpu().double() / (T * K), idx.cpu().long()

    def loss(l):
        p, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)
        c = l.gather(1, at)
        weights = torch.softmax(c, 1) if renorm else p.gather(1, at)
        return (weights * dw.double()).sum() + 0.5 * E * (f * p.mean(0)).sum() + 0.25 * lse.square().mean()

    l, step = logits.double(), 1e-5
    for t in range(T):
        for e in range(E):
            x = torch.zeros(T, E, dtype=torch.float64)
            x[t, e] = step
            diff = float((loss(l + x) - loss(l - x)) / (2 * step))
            assert abs(float(g[t, e]) - diff) <= 1e-5 * abs(diff) + 3e-6    # float32 weights; the difference to 1e-9


def test_without_logits():
    logits, _, idx, w = _route(30, 20, 4)
    dw = torch.randn(30, 4, generator=gen(7)).cuda()
    a = ops.moe_route_backward(logits.cuda(), idx, w, dw)
    b = ops.moe_route_backward(None, idx, w, dw, num_experts=20)
    assert torch.equal(a, b)


def test_an_expert_in_two_slots():
    logits = torch.randn(8, 70, generator=gen(8))
    idx = torch.tensor([[3, 3, 69], [1, 2, 1]] * 4, dtype=torch.int32)
    w, dw = torch.rand(8, 3, generator=gen(9)), torch.randn(8, 3, generator=gen(10))
    for renorm in (True, False):
        g = ops.moe_route_backward(logits.cuda(), idx.cuda(), w.cuda(), dw.cuda(), renormalize=renorm)
        want, bound = _gradient64(logits, None, idx, w, dw, renorm, None, None, 8)
        within(g, want, bound)


def test_logits_that_are_not_finite():
    logits = torch.randn(8, 100, generator=gen(11))
    logits[0, 5:] = -INF                                             # experts that are masked
    logits[1] = -INF                                                 # a row that the mask leaves empty
    logits[2] = float("nan")
    logits[3, 7] = float("nan")
    logits[4, 9] = INF
    logits[5, [2, 90]] = INF
    logits[6, 3] = torch.finfo(torch.float32).min
    idx, w = ops.moe_route(logits.cuda(), 4)
    r = ops.moe_balance_loss(logits.cuda(), idx)
    counts, n, P, balance, z, slack, lse = _losses64(logits, None, idx.cpu(), 100, 4)
    assert torch.equal(r.counts.cpu(), counts.int()) and int(r.num_tokens) == 8
    within(r.probs, P, slack + 8 * U * P)
    within(r.loss[0], balance, 100 * (counts.double() * (slack + 8 * U * P)).sum() / 32 + U * balance)
    off = (lse.abs() + 32) * U + 2 * U * lse.abs()
    within(r.loss[1], z, (2 * lse.abs() * off + off ** 2).sum() / 8 + U * z)
    dw, d = torch.randn(8, 4, generator=gen(12)), torch.tensor([1.0, 1.0])
    for renorm in (True, False):
        g = ops.moe_route_backward(logits.cuda(), idx, w, dw.cuda(), renormalize=renorm, d_loss=d.cuda(),
                                   counts=r.counts, num_tokens=r.num_tokens)
        want, bound = _gradient64(logits, None, idx.cpu(), w.cpu(), dw, renorm, d, r.counts.cpu(), 8)
        within(g, want, bound)
        assert torch.isfinite(g).all()


def test_equal_calls_give_equal_bits_on_any_stream_and_in_a_graph():
    logits, valid, idx, w = _route(2000, 96, 6, 100)
    l, v = logits.cuda(), valid.cuda()
    dw, d = torch.randn(2000, 6, generator=gen(13)).cuda(), torch.tensor([0.1, 0.01], device="cuda")

    def call(stream=None, out=None, ws=None, g=None):
        r = ops.moe_balance_loss(l, idx, v, out=out, workspace=ws, stream=stream)
        g = ops.moe_route_backward(l, idx, w, dw, v, d_loss=d, counts=r.counts, num_tokens=r.num_tokens, d_logits=g,
                                   stream=stream)
        return r.loss, r.counts, r.probs, r.num_tokens, g

    first = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    out = ops.RouterLosses(*other[:4])
    ws = torch.empty(ops.moe_balance_loss_workspace_bytes(2000, 96), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(None, out, ws, other[4])
    for k in range(3):
        l.copy_(torch.randn(2000, 96, generator=gen(40 + k)))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(other, call()))


def test_offsets_past_32_bits():
    """2.2e9 logits: the counts of all, and the gradient of the last tokens."""
    T, E = 2_200_000, 1024
    logits = torch.zeros(T, E, device="cuda")
    logits[-4:] = torch.randn(4, E, generator=gen(1)).cuda()
    idx = torch.full((T, 1), 3, dtype=torch.int32, device="cuda")
    idx[-1] = 1023
    r = ops.moe_balance_loss(logits, idx)
    assert int(r.num_tokens) == T and int(r.counts[3]) == T - 1 and int(r.counts[1023]) == 1
    d = torch.tensor([float(T), float(T)], device="cuda")
    g = ops.moe_route_backward(logits, idx, torch.ones(T, 1, device="cuda"), None, d_loss=d, counts=r.counts,
                               num_tokens=r.num_tokens)
    want, bound = _gradient64(logits[-4:].cpu(), None, idx[-4:].cpu(), None, None, True, d.cpu(), r.counts.cpu(), T)
    # (the routing has one slot: K of the formula is idx's)
    within(g[-4:], want, bound)
