"""Shared by the tests of the norm, the FP8 product and the router's losses:
inputs, the formulas in 64 bits and the error bounds of float32 arithmetic."""

import torch

U = 2.0 ** -24          # half a step of float32, relative
BF16 = 2.0 ** -8        # of bf16
TINY = 2.0 ** -133      # half a step of bf16's subnormals


def gen(seed):
    return torch.Generator().manual_seed(seed)


def e4m3(codes):
    """The values of E4M3 codes (uint8), in 64 bits."""
    return codes.cpu().view(torch.float8_e4m3fn).double()


def quant_rows(x):
    """float32 rows -> codes uint8, scales [H/128, T]."""
    T, H = x.shape
    t = x.reshape(T, H // 128, 128)
    s = t.abs().amax(2) / 448.0
    q = torch.where(s[:, :, None] > 0, t / s[:, :, None], torch.zeros_like(t)).clamp(-448, 448)
    return q.reshape(T, H).to(torch.float8_e4m3fn).view(torch.uint8), s.t().contiguous()


def quant_tiles(w):
    """float32 [N, K] -> codes uint8, scales [ceil(N/128), K/128]."""
    N, K = w.shape
    nb = -(-N // 128)
    x = torch.zeros(nb * 128, K)
    x[:N] = w
    t = x.reshape(nb, 128, K // 128, 128)
    s = t.abs().amax((1, 3)) / 448.0
    safe = torch.where(s > 0, s, torch.ones_like(s))[:, None, :, None]
    q = (t / safe).clamp(-448, 448).reshape(nb * 128, K)[:N]
    return q.to(torch.float8_e4m3fn).view(torch.uint8), s


def rows64(codes, scales):
    T, K = codes.shape
    return (e4m3(codes).reshape(T, K // 128, 128) * scales[:, :T].t().double().cpu()[:, :, None]).reshape(T, K)


def tiles64(codes, scales):
    N, K = codes.shape
    s = scales.double().cpu().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    return e4m3(codes) * s


def within(got, want, bound, what=""):
    """Every element of got within `bound` of want (all in 64 bits)."""
    d = (got.double().cpu() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((d - bound)[bad].max()), float(d.max()))


def product_slack(X, W):
    """What the FP8 matrix instruction may lose of X W^T.  It adds 8 neighbouring
    products exactly but for their low bits: each is cut off at 2^-13 of 2^e, e
    the largest exponent sum among the 8 (measured bit by bit: 2^16, -2^16 and
    2^3 give 2^3, with 2^2 in its place 0).  The product with that exponent sum is
    at least 2^e, so each of the other 7 loses less than 2^-13 of the largest
    product, which is at most the largest |x| times the largest |w| of the 8.  The
    sums of 8 are then added in float32, by truncation at worst: 16 additions a
    block of 128, two half steps each."""
    top = lambda A: A.abs().reshape(A.shape[0], -1, 8).amax(2)  # noqa: E731
    return 7 * 2.0 ** -13 * (top(X) @ top(W).t()) + 32 * U * (X.abs() @ W.abs().t())
