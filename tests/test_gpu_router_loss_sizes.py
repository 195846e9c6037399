"""moe_balance_loss and moe_route_backward for more than 256 experts and more tokens than
one workgroup takes, and for the longest sums of a wave, against the formulas in 64 bits."""

import pytest
import torch

from combine_top_route_moe_amd import ops
from tests.around_util import U, gen, within
from tests.test_gpu_router_loss import _gradient64, _losses64, _route, _softmax64

pytestmark = pytest.mark.gpu

CASES = [(65, 257, 8, 0), (65, 512, 3, 11), (700, 300, 8, 33), (1000, 512, 10, 200), (65, 513, 4, 1), (200, 700, 32, 0),
         (2000, 1000, 4, 500), (3001, 1024, 1, 7), (65, 64, 8, 64), (65, 2, 1, 0), (4000, 3, 2, 1)]


def _additions(T, E):
    """Of a probability to a float32 sum, one after another: the tokens of a wave, of 16 a
    workgroup, and the workgroup's waves in halves; the workgroups' sums meet in 64 bits."""
    groups = min(-(-T // 16), 256, max(32, 32768 // E))
    return -(-T // (16 * groups)) + 4


def check_losses(r, counts, n, P, balance, z, slack, lse, T, E, K):
    assert torch.equal(r.counts.cpu(), counts.int()) and int(r.num_tokens) == n
    per = slack + (_additions(T, E) + 1) * U * P
    within(r.probs, P, per, "probs")
    within(r.loss[0], balance, E * (counts.double() * per).sum() / max(n * K, 1) + U * balance, "balance")
    off = (lse.abs() + 32) * U + 2 * U * lse.abs()
    within(r.loss[1], z, (2 * lse.abs() * off + off ** 2).sum() / max(n, 1) + U * z, "z")


@pytest.mark.parametrize("T,E,K,pad", CASES)
def test_losses(T, E, K, pad):
    assert ops.moe_balance_loss_workspace_bytes(T, E) > 0              # (more than one workgroup)
    logits, valid, idx, _ = _route(T, E, K, pad)
    r = ops.moe_balance_loss(logits.cuda(), idx, None if valid is None else valid.cuda())
    check_losses(r, *_losses64(logits, valid, idx.cpu(), E, K), T, E, K)


@pytest.mark.parametrize("T,E,K,pad", CASES)
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient(T, E, K, pad, renorm):
    logits, valid, idx, w = _route(T, E, K, pad, renorm)
    v = None if valid is None else valid.cuda()
    r = ops.moe_balance_loss(logits.cuda(), idx, v)
    dw, d = torch.randn(T, K, generator=gen(5)), torch.tensor([0.7, -0.3])
    g = ops.moe_route_backward(logits.cuda(), idx, w, dw.cuda(), v, renorm, d_loss=d.cuda(), counts=r.counts,
                               num_tokens=r.num_tokens)
    want, bound = _gradient64(logits, valid, idx.cpu(), w.cpu(), dw, renorm, d, r.counts.cpu(), T - pad)
    within(g, want, bound)


@pytest.mark.parametrize("T,E,K", [(300_000, 1024, 2), (1_000_000, 40, 3), (400_000, 300, 1)])
def test_the_longest_sums(T, E, K):
    """Hundreds of tokens a wave, whose probabilities no sum holds exactly."""
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.empty(T, E, device="cuda").normal_(generator=g)
    idx = torch.randint(0, E, (T, K), dtype=torch.int32, device="cuda", generator=g)
    r = ops.moe_balance_loss(logits, idx)
    P, part = (torch.zeros(E, dtype=torch.float64, device="cuda") for _ in range(2))
    lse = []
    for rows in logits.split(50_000):
        l = rows.double()
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - top)
        s = e.sum(1, keepdim=True)
        rel = (2 * (top - l.amin(1, keepdim=True)) + 30) * U           # (as _softmax64)
        P += (e / s).sum(0) / T
        part += (e / s * rel).sum(0) / T
        lse.append((top + torch.log(s))[:, 0].cpu())
    counts = torch.bincount(idx.flatten().long(), minlength=E).cpu()
    P, part, lse = P.cpu(), part.cpu(), torch.cat(lse)
    check_losses(r, counts, T, P, E * (counts.double() * P).sum() / (T * K), lse.square().mean(), part, lse, T, E, K)


def test_the_chunked_reference_is_the_other_ones():
    logits = torch.randn(50, 30, generator=gen(2))
    p, lse, rel = _softmax64(logits)
    l = logits.double()
    assert torch.equal(rel, (2 * (l.amax(1, keepdim=True) - l.amin(1, keepdim=True)) + 30) * U)
