"""The few-token MoE layer and the grouped expert FFN on 4-bit weights: cases,
inputs, plain forms and the framework's calls.

  decode  the whole layer for a few tokens: route each token to its top-k
          experts, run those experts' SwiGLU FFNs, weight and add the rows,
          add the shared expert where there is one.  Expert weights in bf16,
          FP8 (E4M3, one float32 scale per 128 x 128 tile), MXFP4 (E2M1, one
          power-of-two scale per 32 weights of a row) or NVFP4 (E2M1, one E4M3
          scale per 16 weights of a row under a float32 scale per expert).
  ffn     y = row_scale * W2_g (silu(W1_g x) * (W3_g x)) for every row x of
          every group g's segment, MXFP4 or NVFP4 weights.

A quantized weight is the bf16 value that its code and scale stand for.
"""

import math

import torch

own = False

DEV = "cuda"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------- the cases
def listed():
    d = lambda name, fmt, T, H, E, K, I, shared=0, pad=0, local=0: {  # noqa: E731
        "name": name, "op": "decode", "fmt": fmt, "T": T, "H": H, "E": E, "K": K, "I": I,
        "shared": shared, "pad": pad, "local": local or E}
    f = lambda name, fmt, rows, G, H, I, skew: {  # noqa: E731
        "name": name, "op": "ffn", "fmt": fmt, "rows": rows, "G": G, "H": H, "I": I, "skew": skew}
    return [
        # one token through the smallest layer: launch latency
        d("decode tiny bf16 1", "bf16", 1, 256, 8, 2, 128),
        # one user's next token, a small mixture (2048 hidden, 64 experts)
        d("decode small bf16 1", "bf16", 1, 2048, 64, 8, 1024),
        # a ragged batch with padding rows (a captured batch size filled in part)
        d("decode small fp8 13", "fp8", 13, 2048, 64, 8, 1024, pad=2),
        # a full decode batch of the same mixture
        d("decode small mxfp4 64", "mxfp4", 64, 2048, 64, 8, 1024),
        # one user's next token, a large mixture with a shared expert
        d("decode large bf16 1", "bf16", 1, 7168, 256, 8, 2048, shared=2048),
        d("decode large mxfp4 1", "mxfp4", 1, 7168, 256, 8, 2048, shared=2048),
        # a decode batch on one of four expert-parallel ranks of the large mixture
        d("decode large fp8 48 rank", "fp8", 48, 7168, 256, 8, 2048, shared=2048, local=64),
        # a decode batch of a middle-sized mixture
        d("decode middle nvfp4 24", "nvfp4", 24, 4096, 128, 8, 1536),
        # one row through one expert: the matrix-vector product
        f("ffn small mxfp4 1 row", "mxfp4", 1, 1, 2048, 1024, 0),
        # a short ragged batch over many experts, some of them empty
        f("ffn small nvfp4 333 rows", "nvfp4", 333, 64, 2048, 1024, 1),
        # a batch of 512 tokens, top-8: 64 rows an expert
        f("ffn small mxfp4 4096 rows", "mxfp4", 4096, 64, 2048, 1024, 0),
        # a prompt of 4096 tokens, top-8, on 64 experts
        f("ffn middle mxfp4 32768 rows", "mxfp4", 32768, 64, 4096, 1536, 1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        H, I = 128 * _log(rng, 2, 56), 128 * _log(rng, 1, 16)
        if rng.random() < 0.6:
            E = _log(rng, 4, 256)
            K = rng.randint(1, min(E, 10))
            T = _log(rng, 1, 64)
            c = {"op": "decode", "fmt": rng.choice(["bf16", "fp8", "mxfp4", "nvfp4"]), "T": T, "H": H,
                 "E": E, "K": K, "I": I, "shared": rng.choice([0, 128 * _log(rng, 1, 16)]),
                 "pad": rng.randint(0, T // 4), "local": rng.choice([E, E, max(1, E // 2)])}
            if c["local"] * I * H <= 6e8:
                return c
        else:
            G, rows = _log(rng, 1, 96), _log(rng, 1, 16384)
            c = {"op": "ffn", "fmt": rng.choice(["mxfp4", "nvfp4"]), "rows": rows, "G": G, "H": H, "I": I,
                 "skew": rng.randint(0, 1)}
            if G * I * H <= 4e8 and rows * I * H <= 1e11:
                return c


def _begin(c):
    """First local expert: the second share where there is more than one."""
    return c["local"] if 2 * c["local"] <= c["E"] else 0


BITS = {"bf16": 16.0, "fp8": 8.0 + 32 / 128 ** 2, "mxfp4": 4.0 + 8 / 32, "nvfp4": 4.0 + 8 / 16}


def work(case):
    c, per = case, 3 * case["H"] * case["I"]
    if c["op"] == "ffn":
        active = c["G"] if not c["skew"] else c["G"] * (1 - 0.8 ** max(1.0, c["rows"] / c["G"]))
        active = max(1.0, min(active, c["rows"]))
        return {"bytes": active * per * BITS[c["fmt"]] / 8 + 4 * c["rows"] * c["H"], "flops": 2 * c["rows"] * per}
    T, real = c["T"], c["T"] - c["pad"]
    active = c["local"] * (1 - (1 - c["K"] / c["E"]) ** real)      # expected, routes being uniform
    shared = 3 * c["H"] * c["shared"]
    return {"bytes": (active * per + shared) * BITS[c["fmt"]] / 8 + 4 * T * c["H"] + 4 * T * c["E"] + 8 * T * c["K"],
            "flops": 2 * per * real * c["K"] * c["local"] / c["E"] + 2 * shared * T}


# ---------------------------------------------------------------- the inputs
def _e2m1_code(r):
    """E2M1 codes of r, |r| <= 6: nearest, halfway values to the even code."""
    a = r.abs()
    q = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return q.to(torch.uint8) | (torch.signbit(r).to(torch.uint8) << 3)


def _pow2(e):
    """2^e as float32, exactly, for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _nibbles(q):
    return q[..., 0::2] | (q[..., 1::2] << 4)                       # the even element in the low half


def _quantize(w, fmt):
    """One expert's bf16 matrix [N, Kd] -> what a checkpoint holds of it."""
    if fmt == "bf16":
        return {"w": w}
    x = w.float()
    N, Kd = x.shape
    if fmt == "fp8":
        t = x.reshape(N // 128, 128, Kd // 128, 128)
        s = t.abs().amax((1, 3)) / 448.0
        q = torch.where(s[:, None, :, None] > 0, t / s[:, None, :, None], torch.zeros_like(t)).clamp(-448, 448)
        return {"w": q.reshape(N, Kd).to(torch.float8_e4m3fn), "s": s}
    n = 32 if fmt == "mxfp4" else 16
    t = x.reshape(N, Kd // n, n)
    amax = t.abs().amax(2)
    if fmt == "mxfp4":
        e = (torch.frexp(amax).exponent - 3).clamp(-126, 126)       # 2^(floor(log2 amax) - 2)
        q = _e2m1_code((t * _pow2(-e)[..., None]).clamp(-6, 6))
        return {"w": _nibbles(q.reshape(N, Kd)), "s": (e + 127).to(torch.uint8)}
    g = x.abs().max() / 2688.0                                      # 6 * 448
    b = (amax / (6.0 * g)).clamp(max=448).to(torch.float8_e4m3fn)
    S = (b.float() * g)[..., None]
    q = _e2m1_code(torch.where(S > 0, t / S, torch.zeros_like(t)).clamp(-6, 6))
    return {"w": _nibbles(q.reshape(N, Kd)), "s": b, "g": g}


def _expert_weights(gen, fmt, G, H, I):
    """G experts' (w13, w2) drawn at a checkpoint's scale, as stacked checkpoint
    tensors; the framework's packed form of the same weights beside them."""
    plain, w13, w2 = None, None, None
    for g in range(G):
        a = (torch.randn(2 * I, H, generator=gen, device=DEV) * 0.02).bfloat16()
        b = (torch.randn(H, I, generator=gen, device=DEV) * 0.02).bfloat16()
        parts = {"13" + k: v for k, v in _quantize(a, fmt).items()}
        parts |= {"2" + k: v for k, v in _quantize(b, fmt).items()}
        if plain is None:
            plain = {k: torch.empty((G,) + tuple(v.shape), dtype=v.dtype, device=DEV) for k, v in parts.items()}
            if own:
                w13, w2 = plain.get("13w"), plain.get("2w")
                if fmt != "bf16":
                    w13 = torch.empty(G, 2 * I, H, dtype=torch.bfloat16, device=DEV)
                    w2 = torch.empty(G, H, I, dtype=torch.bfloat16, device=DEV)
        for k, v in parts.items():
            plain[k][g] = v
        if own and fmt != "bf16":
            w13[g], w2[g] = a, b
    handle = None
    if own:
        from combine_top_route_moe_amd import ops
        if fmt == "fp8":                                            # the checkpoint's codes, as they are
            return plain, ops.ffn_weights_from_codes(fmt, plain["13w"], plain["13s"], plain["2w"], plain["2s"])
        handle = ops.ffn_weights(w13, w2, fmt, w13_tensor_scale=plain.get("13g"), w2_tensor_scale=plain.get("2g"))
    return plain, handle


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(c)
    if c["op"] == "decode":
        T, E, H, K = c["T"], c["E"], c["H"], c["K"]
        s["logits"] = torch.randn(T, E, generator=gen, device=DEV)
        s["hidden"] = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
        s["valid"] = None
        if c["pad"]:
            s["valid"] = torch.ones(T, dtype=torch.uint8, device=DEV)
            s["valid"][torch.randperm(T, generator=gen, device=DEV)[: c["pad"]]] = 0
        s["plain"], s["handle"] = _expert_weights(gen, c["fmt"], c["local"], H, c["I"])
        s["shared_plain"] = s["shared_handle"] = None
        if c["shared"]:
            s["shared_plain"], s["shared_handle"] = _expert_weights(gen, c["fmt"], 1, H, c["shared"])
        if own:
            from combine_top_route_moe_amd import ops
            s["topk_idx"] = torch.empty(T, K, dtype=torch.int32, device=DEV)
            s["topk_w"] = torch.empty(T, K, device=DEV)
            s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
            need = ops.moe_decode_workspace_bytes(T, H, c["I"], K, c["local"], c["shared"])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        return s
    G, H, rows = c["G"], c["H"], c["rows"]
    p = torch.ones(G, device=DEV)
    if c["skew"]:                                                   # a few busy experts, many idle ones
        p = torch.exp(1.5 * torch.randn(G, generator=gen, device=DEV))
    if c["skew"]:
        pick = torch.multinomial(p, rows, replacement=True, generator=gen)
    else:
        pick = torch.arange(rows, device=DEV) % G
    counts = torch.bincount(pick, minlength=G)
    s["longest"] = int(counts.max())
    s["counts"] = counts.to(torch.int32)
    s["cu"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["x"] = torch.randn(rows, H, generator=gen, device=DEV).bfloat16()
    s["row_scale"] = torch.rand(rows, generator=gen, device=DEV)
    s["plain"], s["handle"] = _expert_weights(gen, c["fmt"], G, H, c["I"])
    if own:
        from combine_top_route_moe_amd import ops
        s["y"] = torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.empty(ops.moe_grouped_ffn_fp4_workspace_bytes(rows, G, H, c["I"]), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- the plain forms
def _dense(plain, which, fmt, pick=None):
    """float32 weights [n, N, Kd] of the experts `pick` (all: None)."""
    take = (lambda t: t) if pick is None else (lambda t: t[pick])
    w = take(plain[which + "w"])
    if fmt == "bf16":
        return w.float()
    s = take(plain[which + "s"])
    if fmt == "fp8":
        n, N, Kd = w.shape
        v = w.float().reshape(n, N // 128, 128, Kd // 128, 128) * s[:, :, None, :, None]
        return v.reshape(n, N, Kd).bfloat16().float()
    n, N, half = w.shape
    lut = torch.tensor(E2M1 + [-v for v in E2M1], device=w.device)
    v = torch.stack([lut[(w & 15).int()], lut[(w >> 4).int()]], -1)
    if fmt == "mxfp4":
        v = v.reshape(n, N, -1, 32)
        return (v * _pow2(s.int() - 127)[..., None]).reshape(n, N, 2 * half)
    S = s.float() * take(plain[which + "g"])[:, None, None]
    return (v.reshape(n, N, -1, 16) * S[..., None]).reshape(n, N, 2 * half).bfloat16().float()


def _swiglu(h):
    g, u = h.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def _decode_plain(s):
    T, K, E, fmt = s["T"], s["K"], s["E"], s["fmt"]
    first, local = _begin(s), s["local"]
    logits, x = s["logits"], s["hidden"].float()
    idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :K]
    top = logits.gather(1, idx)
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    if s["valid"] is not None:
        keep = s["valid"].bool()[:, None]
        idx, w = torch.where(keep, idx, -1), torch.where(keep, w, 0.0)
    here = (idx >= first) & (idx < first + local)
    e = torch.where(here, idx - first, 0)
    wl = torch.where(here, w, 0.0)
    if T * K < local:                                               # the chosen experts, slot by slot
        p = e.reshape(-1)
        xs = x.repeat_interleave(K, 0)[:, :, None]
        a = _swiglu(torch.bmm(_dense(s["plain"], "13", fmt, p), xs)[:, :, 0])
        rows = torch.bmm(_dense(s["plain"], "2", fmt, p), a[:, :, None])[:, :, 0]
        out = (rows.reshape(T, K, -1) * wl[:, :, None]).sum(1)
    else:                                                           # every expert, weight 0 where not chosen
        dense = torch.zeros(T, local, device=x.device).scatter_add_(1, e, wl)
        w13 = _dense(s["plain"], "13", fmt)
        a = _swiglu((x @ w13.flatten(0, 1).t()).reshape(T, local, -1))
        w2 = _dense(s["plain"], "2", fmt).permute(0, 2, 1).flatten(0, 1)
        out = (a * dense[:, :, None]).flatten(1) @ w2
    if s["shared"]:
        a = _swiglu(x @ _dense(s["shared_plain"], "13", fmt)[0].t())
        out = out + a @ _dense(s["shared_plain"], "2", fmt)[0].t()
    return out.bfloat16(), idx.int(), w


def _ffn_plain(s):
    rows, fmt, counts, cu = s["rows"], s["fmt"], s["counts"], s["cu"]
    i = torch.arange(s["longest"], device=counts.device)
    real = i < counts[:, None]
    at = torch.where(real, cu[:-1, None] + i, rows).long()          # [G, longest], padding at row `rows`
    near = at.clamp(max=rows - 1)
    a = _swiglu(torch.bmm(s["x"][near].float(), _dense(s["plain"], "13", fmt).transpose(1, 2)))
    y = torch.bmm(a, _dense(s["plain"], "2", fmt).transpose(1, 2)) * s["row_scale"][near][:, :, None]
    out = torch.empty(rows + 1, s["H"], dtype=torch.bfloat16, device=y.device)
    return out.index_copy_(0, at.flatten(), y.flatten(0, 1).bfloat16())[:rows]


def run(state):
    s = state
    if own:
        from combine_top_route_moe_amd import ops
        if s["op"] == "decode":
            return ops.moe_decode(s["logits"], s["hidden"], s["K"], s["handle"], row_valid=s["valid"],
                                  expert_begin=_begin(s), shared=s["shared_handle"], topk_idx=s["topk_idx"],
                                  topk_w=s["topk_w"], out=s["out"], workspace=s["ws"])
        return ops.moe_grouped_ffn_fp4(s["x"], s["cu"], s["counts"], s["handle"], s["row_scale"], y=s["y"],
                                       workspace=s["ws"])
    return _decode_plain(s) if s["op"] == "decode" else _ffn_plain(s)


# ---------------------------------------------------------------- in 64 bits
def _matrix64(plain, which, fmt, g):
    """One expert's weights in 64 bits, decoded from the bits of its codes."""
    w = plain[which + "w"][g]
    if fmt == "bf16":
        return w.double()
    s = plain[which + "s"][g]
    if fmt == "fp8":
        scale = s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return (w.double() * scale).float().bfloat16().double()
    q = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.int32, device=w.device)
    q[:, 0::2], q[:, 1::2] = w.int() % 16, w.int() // 16
    sign, e, m = 1 - 2 * (q // 8), (q % 8) // 2, (q % 2).double()
    v = sign * torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    if fmt == "mxfp4":
        return v * torch.exp2(s.double() - 127).repeat_interleave(32, 1)
    S = (s.double() * plain[which + "g"][g].double()).float().double().repeat_interleave(16, 1)
    return (v * S).float().bfloat16().double()


def _expert64(plain, fmt, g, x):
    h = x @ _matrix64(plain, "13", fmt, g).t()
    n = h.shape[1] // 2
    return (h[:, :n] * torch.sigmoid(h[:, :n]) * h[:, n:]) @ _matrix64(plain, "2", fmt, g).t()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "ffn":
        y = torch.zeros(c["rows"], c["H"], dtype=torch.float64, device=DEV)
        at = s["cu"].tolist()
        for g in range(c["G"]):
            if at[g + 1] > at[g]:
                y[at[g]:at[g + 1]] = _expert64(s["plain"], c["fmt"], g, s["x"][at[g]:at[g + 1]].double())
        return y * s["row_scale"].double()[:, None]
    T, K = c["T"], c["K"]
    rows = s["logits"].double().tolist()
    ids = torch.full((T, K), -1, dtype=torch.int64)
    wts = torch.zeros(T, K, dtype=torch.float64)
    for t in range(T):
        if s["valid"] is not None and not int(s["valid"][t]):
            continue
        order = sorted(range(c["E"]), key=lambda e: (-rows[t][e], e))[:K]
        terms = [math.exp(rows[t][e] - rows[t][order[0]]) for e in order]
        ids[t] = torch.tensor(order)
        wts[t] = torch.tensor([v / math.fsum(terms) for v in terms], dtype=torch.float64)
    x = s["hidden"].double()
    out = torch.zeros(T, c["H"], dtype=torch.float64, device=DEV)
    for e in range(c["local"]):
        t, k = torch.nonzero(ids == e + _begin(c), as_tuple=True)
        if len(t):
            t, wt = t.to(DEV), wts[t, k].to(DEV)
            out[t] += wt[:, None] * _expert64(s["plain"], c["fmt"], e, x[t])
    if c["shared"]:
        out += _expert64(s["shared_plain"], c["fmt"], 0, x)
    return out, ids.int().to(DEV), wts.to(DEV)
