"""Refusals of moe_rmsnorm, moe_linear_fp8, moe_balance_loss, their gradients
and packing, and their size queries: everything the host can see is answered
before any device work (no GPU needed; the pointers are never read)."""

import pytest
import torch

from combine_top_route_moe_amd import _lib, ops

P = 1 << 20            # a 16-byte aligned address, never read
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _norm(lib, **kw):
    a = dict(x=P, res=P, w=P, T=4, H=256, eps=1e-6, flags=0, h=2 * P, y=3 * P, codes=P, scales=P, stride=4, rstd=P)
    a.update(kw)
    return lib.moe_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(flags=2), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(H=100), UNSUPPORTED), (dict(H=32768 + 128), UNSUPPORTED), (dict(T=(1 << 26) - 3, stride=1 << 40), UNSUPPORTED),
    (dict(T=1 << 24, H=4096, stride=1 << 40), UNSUPPORTED), (dict(T=1 << 22, H=16384), UNSUPPORTED),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(stride=3), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(x=P + 2), INVALID), (dict(res=P + 8), INVALID),
    (dict(h=P + 2), INVALID), (dict(y=P + 4), INVALID), (dict(codes=P + 8), INVALID), (dict(w=P + 4), INVALID),
    (dict(h=None, y=None, codes=None, scales=None, rstd=None), INVALID),
    (dict(y=2 * P), INVALID), (dict(res=3 * P), INVALID),
    (dict(T=0, x=None, w=None, stride=0), OK),
])
def test_norm_refusals(lib, kw, status):
    assert _norm(lib, **kw) == status


def _norm_back(lib, **kw):
    a = dict(dy=P, h=2 * P, rstd=P, w=P, T=4, H=256, flags=0, dres=P, dx=3 * P, dw=P, ws=P, bytes=1 << 30)
    a.update(kw)
    return lib.moe_rmsnorm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(flags=4), INVALID), (dict(H=100), UNSUPPORTED), (dict(T=1 << 40), UNSUPPORTED),
    (dict(dw=None), INVALID), (dict(dw=P + 4), INVALID), (dict(dy=None), INVALID), (dict(h=None), INVALID),
    (dict(rstd=None), INVALID), (dict(w=None), INVALID), (dict(dx=None), INVALID), (dict(dx=2 * P), INVALID),
    (dict(dy=P + 2), INVALID), (dict(dres=P + 2), INVALID), (dict(T=2000, ws=None), WORKSPACE),
    (dict(T=2000, ws=P + 8), WORKSPACE), (dict(T=2000, bytes=256 * 4 - 1), WORKSPACE), (dict(dx=2 * P, ws=None), INVALID),
    (dict(dx=P, ws=None), WORKSPACE),                                # in place: never without
])
def test_norm_gradient_refusals(lib, kw, status):
    assert _norm_back(lib, **kw) == status


def _pack(lib, **kw):
    a = dict(w=P, codes=None, scales=None, N=256, K=128, flags=0, packed=2 * P, packed_scales=3 * P)
    a.update(kw)
    return lib.moe_pack_linear_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), INVALID), (dict(K=-128), INVALID), (dict(flags=2), INVALID), (dict(K=100), UNSUPPORTED),
    (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=(1 << 20) + 128), UNSUPPORTED), (dict(N=200, flags=1), UNSUPPORTED),
    (dict(w=None), INVALID), (dict(codes=P, scales=P), INVALID), (dict(w=None, codes=P), INVALID),
    (dict(w=None, scales=P), INVALID), (dict(packed=None), INVALID), (dict(packed_scales=None), INVALID),
    (dict(w=P + 2), INVALID), (dict(packed=P + 8), INVALID), (dict(w=None, codes=2 * P, scales=P), INVALID),
    (dict(w=None, codes=P, scales=3 * P), INVALID),
])
def test_pack_refusals(lib, kw, status):
    assert _pack(lib, **kw) == status


def _linear(lib, **kw):
    a = dict(x=P, xs=P, stride=40, M=40, N=256, K=512, packed=P, scales=P, flags=0, y=2 * P, ws=P, bytes=1 << 40)
    a.update(kw)
    return lib.moe_linear_fp8(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(stride=39), INVALID),
    (dict(flags=1), INVALID), (dict(flags=4), INVALID), (dict(K=130), UNSUPPORTED),
    (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=(1 << 20) + 128), UNSUPPORTED),
    (dict(M=1 << 31, stride=1 << 31), UNSUPPORTED), (dict(x=None), INVALID), (dict(xs=None), INVALID),
    (dict(packed=None), INVALID), (dict(scales=None), INVALID), (dict(y=None), INVALID), (dict(x=P + 8), INVALID),
    (dict(y=P + 2), INVALID), (dict(y=P), INVALID), (dict(packed=P + 4), INVALID), (dict(M=0, x=None, y=None, ws=None), OK),
    (dict(M=(1 << 31) - 1, stride=1 << 31, N=1 << 20, K=128), UNSUPPORTED),
])
def test_linear_refusals(lib, kw, status):
    assert _linear(lib, **kw) == status


def test_sizes(lib):
    assert lib.moe_linear_fp8_packed_bytes(576, 7168) == 576 * 7168
    assert lib.moe_linear_fp8_packed_bytes(17, 128) == 32 * 128
    assert lib.moe_linear_fp8_packed_bytes(1 << 20, 1 << 20) == 1 << 40
    assert [lib.moe_linear_fp8_packed_bytes(*a) for a in ((0, 128), (16, 100), (1 << 21, 128))] == [0, 0, 0]
    assert lib.moe_rmsnorm_backward_workspace_bytes(0, 256) == 0
    assert lib.moe_rmsnorm_backward_workspace_bytes(100, 200) == 0
    for T, H in ((1, 128), (10 ** 6, 2048), (10 ** 6, 8192), (10 ** 6, 32768)):
        assert 4 * H <= lib.moe_rmsnorm_backward_workspace_bytes(T, H) <= 4096 * 4 * H
    assert lib.moe_balance_loss_workspace_bytes(0, 64) == 0 and lib.moe_balance_loss_workspace_bytes(9, 2000) == 0
    assert lib.moe_balance_loss_workspace_bytes(ops.MOE_LOSS_FEW_TOKENS, 1024) == 0
    assert lib.moe_linear_fp8_workspace_bytes(ops.MOE_LINEAR_FEW_ROWS, 8192, 8192) == 0
    sizes = [lib.moe_balance_loss_workspace_bytes(T, 64) for T in (1, 64, 65, 1000, 10 ** 4, 10 ** 6)]
    assert sizes[0] == 0 and sizes == sorted(sizes) and sizes[2] > 0 and sizes[-1] < 1 << 20
    sizes = [lib.moe_linear_fp8_workspace_bytes(M, 576, 7168) for M in (1, 16, 17, 64, 500, 5000, 10 ** 6)]
    assert sizes[1] == 0 and sizes == sorted(sizes) and sizes[-1] == 32 << 20    # one for all smaller batches
    assert lib.moe_linear_fp8_workspace_bytes(0, 128, 128) == 0 and lib.moe_linear_fp8_workspace_bytes(1, 1, 100) == 0


def _loss(lib, **kw):
    a = dict(logits=P, valid=None, idx=P, T=4, E=8, K=2, loss=P, counts=P, probs=P, n=P, ws=P, bytes=1 << 30, err=None)
    a.update(kw)
    return lib.moe_balance_loss(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(K=0), INVALID), (dict(K=9), INVALID),
    (dict(E=2000), UNSUPPORTED), (dict(E=64, K=33), UNSUPPORTED), (dict(loss=None), INVALID), (dict(counts=None), INVALID),
    (dict(probs=None), INVALID), (dict(n=None), INVALID), (dict(logits=None), INVALID), (dict(idx=None), INVALID),
    (dict(T=4000, ws=None), WORKSPACE), (dict(T=4000, ws=P + 8), WORKSPACE), (dict(T=4000, bytes=8), WORKSPACE),
])
def test_loss_refusals(lib, kw, status):
    assert _loss(lib, **kw) == status


def _back(lib, **kw):
    a = dict(logits=P, valid=None, idx=P, w=P, dw=P, T=4, E=8, K=2, flags=1, d=P, counts=P, n=P, out=2 * P, err=None)
    a.update(kw)
    return lib.moe_route_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(K=9), INVALID), (dict(flags=2), INVALID), (dict(E=1025), UNSUPPORTED),
    (dict(E=64, K=33), UNSUPPORTED), (dict(out=None), INVALID), (dict(out=P), INVALID), (dict(dw=None, d=None), INVALID), (dict(w=None), INVALID),
    (dict(idx=None), INVALID), (dict(counts=None), INVALID), (dict(n=None), INVALID), (dict(logits=None), INVALID),
    (dict(logits=None, d=None, flags=0), INVALID), (dict(T=0, logits=None, out=None), OK),
])
def test_route_gradient_refusals(lib, kw, status):
    assert _back(lib, **kw) == status


BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


def test_binding_checks():
    x, w = torch.zeros(4, 256, dtype=BF), torch.ones(256)
    with pytest.raises(ValueError, match="device tensor"):
        ops.moe_rmsnorm(x, w)
    with pytest.raises(ValueError, match="weight: expected shape"):
        ops.moe_rmsnorm(x, w[:128])
    with pytest.raises(ValueError, match="residual does not match"):
        ops.moe_rmsnorm(x, w, residual=x[:2])
    with pytest.raises(ValueError, match=r"x must be \[T, H\]"):
        ops.moe_rmsnorm(x[0], w)
    with pytest.raises(ValueError, match="h or d_residual does not match"):
        ops.moe_rmsnorm_backward(x, x[:3], torch.ones(4), w)
    with pytest.raises(ValueError, match=r"rstd must be \[T\]"):
        ops.moe_rmsnorm_backward(x, x, torch.ones(3), w)
    with pytest.raises(ValueError, match="either w, or codes"):
        ops.moe_pack_linear_fp8(None)
    with pytest.raises(ValueError, match="scales must be"):
        ops.linear_weights_from_codes(torch.zeros(200, 256, dtype=U8), torch.ones(1, 2))
    with pytest.raises(ValueError, match="N % 128"):
        ops.linear_weights(torch.zeros(200, 256, dtype=BF), transpose=True)
    with pytest.raises(ValueError, match="device tensor"):
        ops.linear_weights(torch.zeros(200, 256, dtype=BF))
    with pytest.raises(ValueError, match="logits must be"):
        ops.moe_balance_loss(torch.zeros(4), torch.zeros(4, 2, dtype=I32))
    with pytest.raises(ValueError, match="topk_idx must be"):
        ops.moe_balance_loss(torch.zeros(4, 8), torch.zeros(3, 2, dtype=I32))
    idx, k = torch.zeros(4, 2, dtype=I32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="row_valid must be"):
        ops.moe_balance_loss(torch.zeros(4, 8), idx, torch.ones(3, dtype=U8))
    with pytest.raises(ValueError, match="num_experts is needed"):
        ops.moe_route_backward(None, idx, k, k)
    with pytest.raises(ValueError, match="needs counts"):
        ops.moe_route_backward(torch.zeros(4, 8), idx, k, k, d_loss=torch.ones(2))
    with pytest.raises(ValueError, match="one shape"):
        ops.moe_route_backward(torch.zeros(4, 8), idx, k, torch.zeros(4, 3))


def test_sizes_past_the_interface():
    """What a 32-bit argument would take modulo 2^32 (tensors without memory of that size)."""
    far = (1 << 32) + 128
    with pytest.raises(ValueError, match="below 2"):
        ops.moe_rmsnorm(torch.zeros(1, 1, dtype=BF).expand(1, far), torch.zeros(1).expand(far))
    with pytest.raises(ValueError, match="below 2"):
        ops.moe_balance_loss(torch.zeros(1, 1).expand(far, 8), torch.zeros(1, 1, dtype=I32).expand(far, 2))
    with pytest.raises(ValueError, match="below 2"):
        ops.moe_route_backward(torch.zeros(1, 1).expand(far, 8), *(torch.zeros(1, 1).expand(far, 2),) * 3)
    for size in (lambda: ops.moe_linear_fp8_packed_bytes(far, 128), lambda: ops.moe_linear_fp8_workspace_bytes(1, 16, far),
                 lambda: ops.moe_rmsnorm_backward_workspace_bytes(1, far),
                 lambda: ops.moe_balance_loss_workspace_bytes(far, 8)):
        with pytest.raises(ValueError, match="below 2"):
            size()


def test_a_product_uses_what_its_parts_take():
    """The size query is enough for what a product uses, and only that is asked of a caller."""
    lib = _lib.load()
    several = 0
    for M in (1, 16, 17, 40, 64, 128, 333, 1000, 4096):
        for N in (1, 64, 333, 576, 2048, 4096, 8192):
            for K in (128, 256, 1024, 2048, 7168):
                parts, (rows, columns) = ops.moe_linear_fp8_parts(M, N, K)
                assert parts in (1, 2, 4, 8) and parts <= K // 128 and rows >= 16 and columns >= 16
                if parts > 1:
                    several += 1
                    need = 4 * parts * M * N
                    assert need <= lib.moe_linear_fp8_workspace_bytes(M, N, K)
                    kw = dict(M=M, N=N, K=K, stride=M)
                    for bad in (dict(ws=None), dict(bytes=need - 1), dict(ws=P + 8)):
                        assert _linear(lib, **kw, **bad) == WORKSPACE
    assert several > 20
    assert ops.moe_linear_fp8_parts(16, 8192, 8192) == (1, (16, 16))
    for sizes in ((0, 128, 128), (1 << 31, 128, 128), (1, 0, 128), (1, 128, 130), (1, (1 << 20) + 1, 128)):
        assert ops.moe_linear_fp8_parts(*sizes) == (0, (0, 0))
    with pytest.raises(ValueError, match="below 2"):
        ops.moe_linear_fp8_parts(1, 1 << 32, 128)


def test_packing_on_the_weights_is_refused(lib):
    """Workgroups would read what others have written; codes and scales are refused as well."""
    assert _pack(lib, packed=P) == INVALID
