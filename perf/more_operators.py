"""What stands around the experts in a layer: the norm in front of it, the dense
FP8 product beside it, the router's losses and its gradient.  Cases, inputs,
plain forms and the framework's calls.

  norm      h = bf16(x + residual); v = h / sqrt(mean(h^2) + eps) * weight per
            row; v in bf16, and v as E4M3 codes with a scale per row and 128
            channels (the rows that the FP8 products read).
  norm_grad the gradients of v's bf16 form with respect to h and weight, the
            residual stream's own gradient added to h's.
  linear    y = x W^T on E4M3 codes: a float32 scale per row and 128 columns of
            x, per 128 x 128 tile of W.
  balance   the router's losses over the tokens that are real: the balance loss
            E * sum_e (share of slots of e) * (mean probability of e), the mean
            of logsumexp(logits)^2, and the counts and means themselves.
  route_grad the gradient with respect to the logits of the routing weights
            (softmax over the chosen experts, or over all) and of both losses.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    n = lambda name, T, H, residual=1, y=1, codes=1: {  # noqa: E731
        "name": name, "op": "norm", "T": T, "H": H, "residual": residual, "y": y, "codes": codes, "wf32": 0}
    ng = lambda name, T, H, residual=1, wf32=0: {  # noqa: E731
        "name": name, "op": "norm_grad", "T": T, "H": H, "residual": residual, "wf32": wf32}
    li = lambda name, M, N, K: {"name": name, "op": "linear", "M": M, "N": N, "K": K}  # noqa: E731
    b = lambda name, T, E, K, pad: {"name": name, "op": "balance", "T": T, "E": E, "K": K, "pad": pad}  # noqa: E731
    rg = lambda name, T, E, K, pad, renorm: {  # noqa: E731
        "name": name, "op": "route_grad", "T": T, "E": E, "K": K, "pad": pad, "renorm": renorm}
    return [
        # one user's next token in front of a layer whose rows travel as codes
        n("norm 1 row", 1, 2048, y=0),
        # a prompt: the router's product reads bf16, the experts read the codes
        n("norm 4096 rows", 4096, 7168),
        # a training step's micro-batches, a ragged one and a full one
        ng("norm gradient 333 rows", 333, 2048, wf32=1),
        ng("norm gradient 16384 rows", 16384, 4096),
        # one user's next token through a dense projection: weights read once
        li("linear 1 row", 1, 7168, 2048),
        # a ragged decode batch into a narrow projection that ends inside a tile
        li("linear 13 rows narrow", 13, 576, 7168),
        # a short prompt
        li("linear 333 rows", 333, 4096, 2048),
        # a prompt through a dense feed-forward's first product
        li("linear 4096 rows", 4096, 4096, 7168),
        # the smallest batch that a router sees in training, and a full one with padding
        b("balance 64 tokens", 64, 64, 8, 0),
        b("balance 16384 tokens", 16384, 128, 8, 1638),
        rg("route gradient 512 tokens", 512, 64, 8, 0, 1),
        rg("route gradient 4096 tokens", 4096, 256, 8, 100, 1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm", "norm_grad", "linear", "linear", "linear", "balance", "route_grad"])
        if op in ("norm", "norm_grad"):
            c = {"op": op, "T": _log(rng, 1, 16384), "H": 128 * _log(rng, 1, 128),
                 "residual": rng.randint(0, 1), "wf32": rng.randint(0, 1)}
            if op == "norm":
                c["y"], c["codes"] = rng.choice([(1, 0), (0, 1), (1, 1)])
            if c["T"] * c["H"] <= 3e7:
                return c
        elif op == "linear":
            c = {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 16, 8192), "K": 128 * _log(rng, 1, 64)}
            if c["M"] * c["N"] * c["K"] <= 1.2e11:
                return c
        else:
            T, E = _log(rng, 1, 16384), _log(rng, 2, 512)
            c = {"op": op, "T": T, "E": E, "K": rng.randint(1, min(E, 10)), "pad": rng.randint(0, T // 4)}
            if op == "route_grad":
                c["renorm"] = rng.randint(0, 1)
            if T * E <= 2.1e6:
                return c


def work(case):
    c = case
    if c["op"] == "norm":
        n, wide = c["T"] * c["H"], 4 if c["wf32"] else 2
        per = 2 + (4 if c["residual"] else 0) + 2 * c["y"] + (1 + 4 / 128) * c["codes"]
        return {"bytes": n * per + wide * c["H"] + 4 * c["T"], "flops": n * (6 + 4 * c["codes"])}
    if c["op"] == "norm_grad":
        n, wide = c["T"] * c["H"], 4 if c["wf32"] else 2
        return {"bytes": n * (6 + 2 * c["residual"]) + (4 + wide) * c["H"] + 4 * c["T"], "flops": n * 11}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        tiles = -(-N // 128) * (K // 128)
        return {"bytes": M * K + 4 * M * K / 128 + N * K + 4 * tiles + 2 * M * N, "flops": 2 * M * N * K}
    T, E, K = c["T"], c["E"], c["K"]
    real = T - c["pad"]
    if c["op"] == "balance":
        return {"bytes": 4 * real * (E + K) + T + 8 * E + 12, "flops": 5 * real * E}
    return {"bytes": 4 * real * (E + 3 * K) + 4 * T * E + T + 4 * E + 12, "flops": 10 * real * E}


# ---------------------------------------------------------------- the inputs
def _tiles(w):
    """A bf16 matrix as a checkpoint in 128 x 128 blocks holds it: codes, scales."""
    N, K = w.shape
    nb = -(-N // 128)
    x = torch.zeros(nb * 128, K, device=w.device)
    x[:N] = w
    t = x.reshape(nb, 128, K // 128, 128)
    s = t.abs().amax((1, 3)) / 448.0
    q = (t / s[:, None, :, None]).clamp(-448, 448).reshape(nb * 128, K)[:N]
    return q.to(torch.float8_e4m3fn), s


def _rows8(x):
    """float32 rows as codes with a scale per 128 channels, scales block by block."""
    T, H = x.shape
    t = x.reshape(T, H // 128, 128)
    s = t.abs().amax(2) / 448.0
    q = torch.where(s[:, :, None] > 0, t / s[:, :, None], 0.0).clamp(-448, 448)
    return q.reshape(T, H).to(torch.float8_e4m3fn), s.t().contiguous()


def prepare(case, seed):
    c, s = case, dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    if c["op"] in ("norm", "norm_grad"):
        T, H = c["T"], c["H"]
        # a residual stream grows with depth and has a few large channels
        wide = torch.exp(0.5 * randn(H))
        s["weight"] = 1.0 + 0.1 * randn(H)
        s["weight"] = s["weight"] if c["wf32"] else s["weight"].bfloat16()
        if c["op"] == "norm":
            s["x"] = randn(T, H).bfloat16()
            s["stream"] = (4.0 * wide * randn(T, H)).bfloat16() if c["residual"] else None
        else:
            s["h"] = (4.0 * wide * randn(T, H)).bfloat16()
            s["rstd"] = (1 / torch.sqrt(s["h"].double().square().mean(1) + EPS)).float()
            s["dy"] = (0.01 * randn(T, H)).bfloat16()
            s["dh"] = (0.01 * randn(T, H)).bfloat16() if c["residual"] else None
        return s
    if c["op"] == "linear":
        s["x"], s["x_scales"] = _rows8(randn(c["M"], c["K"]))
        s["w"], s["w_scales"] = _tiles((0.02 * randn(c["N"], c["K"])).bfloat16())
        if own:                                                     # a program lays its weights out once
            from combine_top_route_moe_amd import ops
            s["handle"] = ops.linear_weights_from_codes(s["w"], s["w_scales"])
            need = ops.moe_linear_fp8_workspace_bytes(c["M"], c["N"], c["K"])
            s["ws"] = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
        return s
    T, E, K = c["T"], c["E"], c["K"]
    logits = randn(T, E) + 0.5 * randn(E)                           # some experts are liked better
    s["logits"], s["valid"] = logits, None
    if c["pad"]:
        s["valid"] = torch.ones(T, dtype=torch.uint8, device=DEV)
        s["valid"][torch.randperm(T, generator=gen, device=DEV)[: c["pad"]]] = 0
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    real = torch.ones(T, 1, dtype=torch.bool, device=DEV) if s["valid"] is None else s["valid"].bool()[:, None]
    s["idx"] = torch.where(real, idx[:, :K], -1).int()
    if c["op"] == "route_grad":
        over = top[:, :K] if c["renorm"] else top
        w = torch.exp(top[:, :K] - top[:, :1]) / torch.exp(over - top[:, :1]).sum(1, keepdim=True)
        s["w"] = torch.where(real, w, 0.0)
        s["dw"] = randn(T, K)
        ids = s["idx"][s["idx"] >= 0].long()
        s["counts"] = torch.bincount(ids, minlength=E).int()
        s["tokens"] = real.sum().int().reshape(1)
        s["d_loss"] = torch.tensor([0.01, 0.001], device=DEV) * T   # the losses' weights beside a sum over tokens
    return s


# ---------------------------------------------------------------- the plain forms
def _norm_plain(s):
    h = s["x"] if s["stream"] is None else (s["x"].float() + s["stream"].float()).bfloat16()
    f = h.float()
    rstd = 1 / torch.sqrt((f * f).mean(1) + EPS)
    v = f * rstd[:, None] * s["weight"].float()
    out = {"rstd": rstd}
    if s["stream"] is not None:
        out["h"] = h
    if s["y"]:
        out["y"] = v.bfloat16()
    if s["codes"]:
        out["codes"], out["scales"] = _rows8(v)
    return out


def _norm_grad_plain(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    hat = s["h"].float() * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.bfloat16(), (dy * hat).sum(0)


def _linear_plain(s):
    x = (s["x"].float().reshape(s["M"], -1, 128) * s["x_scales"].t()[:, :, None]).reshape(s["M"], -1)
    sw = s["w_scales"].repeat_interleave(128, 0)[: s["N"]].repeat_interleave(128, 1)
    return (x @ (s["w"].float() * sw).t()).bfloat16()


def _softmax(s):
    real = 1.0 if s["valid"] is None else s["valid"].float()[:, None]
    top = s["logits"].amax(1, keepdim=True)
    e = torch.exp(s["logits"] - top)
    z = e.sum(1, keepdim=True)
    return e / z * real, (top + torch.log(z)) * real


def _balance_plain(s):
    T, E, K = s["T"], s["E"], s["K"]
    p, lse = _softmax(s)
    n = torch.full((1,), T, device=DEV) if s["valid"] is None else s["valid"].long().sum().reshape(1)
    ids = torch.where(s["idx"] >= 0, s["idx"], E).flatten().long()
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add_(0, ids, torch.ones_like(ids))[:E]
    mean = p.double().sum(0) / n.clamp(min=1)
    loss = E * (counts.double() / (n * K).clamp(min=1) * mean).sum()
    z = lse.double().square().sum() / n.clamp(min=1)
    return torch.cat([loss.reshape(1), z.reshape(1)]).float(), counts.int(), mean.float(), n.int()


def _route_grad_plain(s):
    E, K, d, n = s["E"], s["K"], s["d_loss"], s["tokens"].clamp(min=1)
    p, lse = _softmax(s)
    f = E * s["counts"].double() / (n * K) - 1                      # its own mean under p is taken off below
    f = f.float()
    g = d[0] / n * p * (f - (p * f).sum(1, keepdim=True)) + 2 * d[1] / n * lse * p
    on = s["idx"] >= 0
    wd = torch.where(on, s["w"] * s["dw"], 0.0)
    dot = wd.sum(1, keepdim=True)
    if s["renorm"]:
        wd = wd - torch.where(on, s["w"], 0.0) * dot
    else:
        g = g - p * dot
    return g.scatter_add_(1, torch.where(on, s["idx"], 0).long(), wd)


def run(state):
    s = state
    if own:
        return _own(s)
    return {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "linear": _linear_plain, "balance": _balance_plain,
            "route_grad": _route_grad_plain}[s["op"]](s)


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from combine_top_route_moe_amd import ops
    if s["op"] == "norm":
        r = ops.moe_rmsnorm(s["x"], s["weight"], EPS, residual=s["stream"], y=bool(s["y"]), codes=bool(s["codes"]), rstd=True)
        out = {"rstd": r.rstd}
        if s["stream"] is not None:
            out["h"] = r.h
        if s["y"]:
            out["y"] = r.y
        if s["codes"]:
            out["codes"], out["scales"] = r.codes.view(torch.float8_e4m3fn), r.scales
        return out
    if s["op"] == "norm_grad":
        return ops.moe_rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["weight"], d_residual=s["dh"])
    if s["op"] == "linear":
        return ops.moe_linear_fp8(s["x"], s["x_scales"], s["handle"], workspace=s["ws"])
    if s["op"] == "balance":
        r = ops.moe_balance_loss(s["logits"], s["idx"], row_valid=s["valid"])
        return r.loss, r.counts, r.probs, r.num_tokens
    return ops.moe_route_backward(s["logits"], s["idx"], s["w"], s["dw"], row_valid=s["valid"], renormalize=bool(s["renorm"]),
                                  d_loss=s["d_loss"], counts=s["counts"], num_tokens=s["tokens"])


# ---------------------------------------------------------------- in 64 bits
def _codes64(v):
    """E4M3 codes and scales of rows in 64 bits: nearest by the grid of each binade."""
    T, H = v.shape
    t = v.reshape(T, H // 128, 128)
    s = t.abs().amax(2) / 448
    r = (t / torch.where(s > 0, s, 1.0)[:, :, None]).clamp(-448, 448)
    step = torch.exp2((torch.frexp(r.abs()).exponent - 4).clamp(min=-9).double())
    return (torch.round(r / step) * step).reshape(T, H), s.t()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        if s["stream"] is not None:
            h = (h + s["stream"].double()).float().bfloat16().double()
        rstd = torch.rsqrt(h.square().sum(1) / c["H"] + EPS)
        v = h * s["weight"].double() * rstd[:, None]
        out = {"rstd": rstd}
        if s["stream"] is not None:
            out["h"] = h
        if c["y"]:
            out["y"] = v
        if c["codes"]:
            out["codes"], out["scales"] = _codes64(v)
        return out
    if c["op"] == "norm_grad":
        # row by row the Jacobian of h * r(h) * w: r (w - h (h.w) r^2 / H), applied to dy
        h, r = s["h"].double(), s["rstd"].double()[:, None]
        g = s["dy"].double() * s["weight"].double()
        dx = r * g - h * r ** 3 * (h * g).sum(1, keepdim=True) / c["H"]
        if s["dh"] is not None:
            dx += s["dh"].double()
        return dx, torch.einsum("th,th->h", s["dy"].double(), h * r)
    if c["op"] == "linear":
        y = torch.zeros(c["M"], c["N"], dtype=torch.float64, device=DEV)
        row = torch.arange(c["N"], device=DEV) // 128
        for b in range(c["K"] // 128):
            k = slice(128 * b, 128 * b + 128)
            part = s["x"][:, k].double() @ s["w"][:, k].double().t().contiguous()
            y += part * s["x_scales"][b].double()[:, None] * s["w_scales"][row, b].double()
        return y
    real = torch.ones(c["T"], device=DEV, dtype=torch.bool) if s["valid"] is None else s["valid"] != 0
    l, idx, n = s["logits"].double()[real], s["idx"][real].long(), max(1, int(real.sum()))
    p, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)
    if c["op"] == "balance":
        counts = torch.bincount(idx.flatten(), minlength=c["E"])
        mean = p.sum(0) / n
        loss = c["E"] * torch.dot(counts.double(), mean) / (n * c["K"])
        return torch.stack([loss, lse.square().sum() / n]), counts.int(), mean, real.sum().int().reshape(1)
    # by the chain rule through a function in 64 bits
    l.requires_grad_(True)
    p = torch.softmax(l, 1)
    over = torch.logsumexp(l.gather(1, idx) if c["renorm"] else l, 1, keepdim=True)
    w = torch.exp(l.gather(1, idx) - over)
    d = s["d_loss"].double()
    total = (w * s["dw"].double()[real]).sum() + d[1] * torch.logsumexp(l, 1).square().sum() / n
    total = total + d[0] * c["E"] * torch.dot(s["counts"].double(), p.sum(0)) / (n * c["K"]) / n
    out = torch.zeros(c["T"], c["E"], dtype=torch.float64, device=DEV)
    out[real] = torch.autograd.grad(total, l)[0]
    return out
