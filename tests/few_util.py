"""Float64 references and error bounds for the few-token layer and the FFN on
4-bit weights, and the packed 4-bit layout read back.

Bounds (element-wise, in magnitudes of the same products):
  * a float32 sum of n products is off by at most n 2^-23 times the sum of
    their magnitudes (2^-24 an addition; twice that leaves room for additions
    that truncate);
  * a = silu(g) u: |silu'| <= 1.1, exp and the division a few float32 steps
    (exp's argument reduction at most |g| 2^-24 <= 2^-18 for |g| <= 64), and
    the rounding of a itself, ``a_step`` relative (2^-16 for the pair of bf16
    numbers, 2^-8 for one);
  * the result's one rounding to bf16: half a step, 2^-8 relative.
"""

from __future__ import annotations

import numpy as np
import torch

import oracle
from oracle.ffn import silu
from oracle.numerics import bf16_bits_to_f32, bf16_bits_to_f64, e4m3fn_round

F32_SUM = 2.0 ** -23
BF16_HALF = 2.0 ** -8
PAIR, SINGLE = 2.0 ** -16, 2.0 ** -8


def bf16(a) -> np.ndarray:
    """bf16 bits of finite values (the host's conversion: large stacks)."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return t.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def tensor_scale(w_bits) -> np.float32:
    return oracle.nvfp4_tensor_scale(np.abs(bf16_bits_to_f32(w_bits)).max())


def _e2m1(r) -> np.ndarray:
    """E2M1 values of float32 r, |r| <= 6 (ties to the even code)."""
    a = np.abs(r)
    q = ((a > .25) * np.float32(.5) + (a >= .75) * np.float32(.5) + (a > 1.25) * np.float32(.5)
         + (a >= 1.75) * np.float32(.5) + (a > 2.5) + (a >= 3.5) + (a > 5.0) * np.float32(2))
    return np.copysign(q.astype(np.float32), r)


def fake_quant(w_bits, fmt: str, g=None) -> np.ndarray:
    """bf16 bits [N, K] of the values that ``fmt`` stores a matrix as: the
    oracle's fake-quantizers (4-bit ones restated here without their tables, a
    hundred times faster; test_fp4_decode_host.py holds them to the oracle's)."""
    if fmt == "bf16":
        return w_bits
    if fmt == "fp8":
        return oracle.quantize_weight_blocks(w_bits)[2]
    N, K = w_bits.shape
    x = bf16_bits_to_f32(w_bits).reshape(N, -1, 32 if fmt == "mxfp4" else 16)
    amax = np.abs(x).max(axis=2)
    if fmt == "mxfp4":
        e = np.clip(np.frexp(np.where(amax > 0, amax, 1))[1] - 3, -127, 127)
        S = np.where(amax > 0, np.ldexp(np.float32(1), e), 0).astype(np.float32)[..., None]
        r = np.ldexp(x, -e[..., None])
    else:
        g = np.float32(tensor_scale(w_bits) if g is None else g)
        with np.errstate(divide="ignore", invalid="ignore"):
            q = amax / np.float32(np.float32(6) * g)
        b = e4m3fn_round(np.minimum(np.where(np.isnan(q), 0, q).astype(np.float64), 448.0))
        S = (b.astype(np.float32) * g)[..., None]
        r = x / np.where(S > 0, S, np.float32(1))
    v = np.where(S > 0, _e2m1(np.clip(r, -6, 6)) * S, np.float32(0))
    return bf16(v).reshape(N, K)


class Stored:
    """fake_quant of each matrix of a stack, when it is first asked for."""

    def __init__(self, w_bits, fmt: str):
        self.w, self.fmt, self.done = w_bits, fmt, {}

    def __getitem__(self, e):
        if e not in self.done:
            self.done[e] = fake_quant(self.w[e], self.fmt)
        return self.done[e]


def make_weights(rng, G: int, H: int, I: int, std: float = 0.06):
    """(w13 [G, 2I, H], w2 [G, H, I]) bf16 bits."""
    def normal(*shape):   # matrix by matrix: the large stacks stay in cache
        w = np.empty(shape, np.uint16)
        for g in range(G):
            w[g] = bf16(rng.standard_normal(shape[1:], dtype=np.float32) * np.float32(std))
        return w

    return normal(G, 2 * I, H), normal(G, H, I)


def expert(x, w13_bits, w2_bits, a_step: float):
    """One expert on rows x (float64 [n, H]): (y, bound of |y - y_computed|)."""
    w13, w2 = bf16_bits_to_f64(w13_bits), bf16_bits_to_f64(w2_bits)
    I, H = w13.shape[0] // 2, w13.shape[1]
    g, u = x @ w13[:I].T, x @ w13[I:].T
    eg = H * F32_SUM * (np.abs(x) @ np.abs(w13[:I]).T)
    eu = H * F32_SUM * (np.abs(x) @ np.abs(w13[I:]).T)
    s = silu(g)
    a = s * u
    ea = 1.1 * eg * np.abs(u) + np.abs(s) * eu + 1.1 * eg * eu + np.abs(a) * (2.0 ** -18 + a_step)
    aw2 = np.abs(w2).T
    return a @ w2.T, ea @ aw2 + (I + 64) * F32_SUM * ((np.abs(a) + ea) @ aw2)


def layer(x_bits, idx, w, El: int, begin: int, w13, w2, shared=None, a_step: float = PAIR):
    """The layer on given routes: (out, bound) float64 [T, H].  w13, w2: bf16
    bits per local expert, as stored."""
    x = bf16_bits_to_f64(x_bits)
    T, K = idx.shape
    out, err, mag = np.zeros((3,) + x.shape)
    for e in range(El):
        t, k = np.nonzero(idx == e + begin)
        if not len(t):
            continue
        y, ey = expert(x[t], w13[e], w2[e], a_step)
        wt = w[t, k].astype(np.float64)[:, None]
        np.add.at(out, t, wt * y)
        np.add.at(err, t, np.abs(wt) * ey)
        np.add.at(mag, t, np.abs(wt * y))
    if shared is not None:
        y, ey = expert(x, shared[0], shared[1], a_step)
        out, err, mag = out + y, err + ey, mag + np.abs(y)
    err = err + (K + 4) * F32_SUM * (mag + err)
    return out, err + BF16_HALF * (np.abs(out) + err)


def check(got_bits, ref, bound, what=""):
    got = bf16_bits_to_f64(got_bits)
    assert got.shape == ref.shape
    over = np.abs(got - ref) > bound
    assert not over.any(), (what, int(over.sum()), got.size, np.argwhere(over)[:4].tolist(),
                            got[over][:4].tolist(), ref[over][:4].tolist(), bound[over][:4].tolist())


def _rows(p, gate_up: bool, N: int):
    """[.., ct, f, r16, rest] with G first -> rows in matrix order."""
    G, n_ct = p.shape[:2]
    rest = p.shape[4:]
    if not gate_up:
        return p.reshape((G, N) + rest)
    half = (G, N // 2) + rest
    return np.concatenate([p[:, :, :2].reshape(half), p[:, :, 2:].reshape(half)], axis=1)


def unpack_fp4(q, s, mode_nv: bool, gate_up: bool):
    """Packed codes and scale bytes -> (codes [G, N, K] 0..15, scale bytes
    [G, N, K/group]).  q [G, N, K/2], s [G, N, K/group] uint8 as packed."""
    G, N, half = q.shape
    K = 2 * half
    nkb, n_ct = K // 128, N // 64
    u = q.reshape(G, n_ct, nkb, 4, 4, 16, 4, 4)          # g ct kb f q4 r p byte
    c = np.stack([u & 15, u >> 4], axis=-1).reshape(G, n_ct, nkb, 4, 4, 16, 4, 8)
    c = c.transpose(0, 1, 3, 5, 2, 6, 4, 7)              # g ct f r kb p q4 j
    codes = _rows(c.reshape(G, n_ct, 4, 16, K), gate_up, N)
    if mode_nv:
        v = s.reshape(G, n_ct, nkb, 2, 16, 4, 4).transpose(0, 1, 5, 4, 2, 6, 3)   # g ct f r kb p h
        return codes, _rows(v.reshape(G, n_ct, 4, 16, K // 16), gate_up, N)
    v = s.reshape(G, n_ct, nkb, 16, 4, 4).transpose(0, 1, 4, 3, 2, 5)     # g ct f r kb p
    return codes, _rows(v.reshape(G, n_ct, 4, 16, K // 32), gate_up, N)


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def fp4_values(codes, scale_bytes, mode_nv: bool, g=None) -> np.ndarray:
    """bf16 bits of the values that codes and scale bytes stand for."""
    v = (E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)).astype(np.float32)
    if not mode_nv:
        X = np.ldexp(1.0, scale_bytes.astype(np.int64) - 127).repeat(32, axis=-1)
        return bf16(v * X)
    b = scale_bytes.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    b = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1.0 + m / 8.0) * 2.0 ** (e - 7.0)).astype(np.float32)
    S = (b * np.asarray(g, dtype=np.float32)[:, None, None]).astype(np.float32).repeat(16, axis=-1)
    return bf16(v * S)
