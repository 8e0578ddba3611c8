"""The operators around the expert layer: cases, inputs, plain forms and 64-bit values.

  router     the load-balance loss of a top-k router with its per-expert counts, and the
             gradient of the router's logits (from the loss and from the chosen probabilities)
  ln_fwd     layer norm of the block's input
  ln_bwd     its backward pass, with the reduction of the weight's and bias's gradients
  clip       global gradient norm over a list of tensors, and clipping
  fp8_infer  a dense layer (a shared expert's projection) in E4M3 with a scale for each block
             of 128: the activations quantised in the call, the weights kept quantised
  fp8_train  the same layer's training step: weights quantised from their bf16 masters, forward,
             input gradient and weight gradient

`own` selects the framework's kernels; otherwise run() is the plain form in 32 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "fp32": F32}
CLIP_EPS = 1e-6      # added to the norm before the division
LN_EPS = 1e-5
FP8_MAX = 448.0      # largest E4M3 value
FP8_TINY = 2.0 ** -100  # floor of a block's amax: keeps both factors finite and normal


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a small router: the repository's smoke shape, where the launches are what counts
        {"name": "router_tiny", "kind": "router", "T": 512, "E": 4, "k": 2, "mask": False},
        # Mixtral's router on its training batch, some tokens of it padding
        {"name": "router_mixtral", "kind": "router", "T": 8192, "E": 8, "k": 2, "mask": True},
        # DeepSeek-V3's router over sixteen micro-batches of 4096 tokens
        {"name": "router_dsv3", "kind": "router", "T": 65536, "E": 256, "k": 8, "mask": False},
        # one decoded token at DeepSeek-V3's hidden size
        {"name": "ln_fwd_token", "kind": "ln_fwd", "M": 1, "N": 7168, "x": "bf16", "w": "bf16"},
        # the GPT-OSS-shaped batch, norm weights kept in fp32; 2880 is no power of two
        {"name": "ln_fwd_gptoss", "kind": "ln_fwd", "M": 16384, "N": 2880, "x": "bf16",
         "w": "fp32"},
        # Mixtral's training batch, backward
        {"name": "ln_bwd_mixtral", "kind": "ln_bwd", "M": 8192, "N": 4096, "x": "bf16",
         "w": "bf16"},
        # the small tensors of a block (router, norms, biases), fp32, in place, not clipped:
        # what most steps do
        {"name": "clip_small", "kind": "clip", "tensors": 12, "numel": 60_001, "types": "fp32",
         "bite": False},
        # a Mixtral-size expert layer's weight gradients with the small tensors beside them,
        # clipped into the optimiser's buffers
        {"name": "clip_layer", "kind": "clip", "tensors": 10, "numel": 1_409_286_144,
         "types": "mixed", "bite": True},
        # one token through a DeepSeek-V3 shared expert's gate and linear projection
        {"name": "fp8_infer_token", "kind": "fp8_infer", "M": 1, "N": 4096, "K": 7168},
        # the same projection on a batch of 4096 tokens
        {"name": "fp8_infer_batch", "kind": "fp8_infer", "M": 4096, "N": 4096, "K": 7168},
        # a GPT-OSS-shaped square layer, an odd number of tokens; 2880 ends inside a block
        {"name": "fp8_train_ragged", "kind": "fp8_train", "M": 1999, "N": 2880, "K": 2880},
        # a dense layer of Mixtral's FC1 shape: the largest
        {"name": "fp8_train_mixtral", "kind": "fp8_train", "M": 8192, "N": 14336, "K": 4096},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]; one in three made odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v if rng.random() < 0.67 else max(lo, v | 1 if v < hi else v)


def draw(rng):
    kind = rng.choice(["router", "ln_fwd", "ln_bwd", "clip", "fp8_infer", "fp8_train"])
    if kind == "router":
        E = _log(rng, 2, 256)
        return {"kind": kind, "T": _log(rng, 1, 65536), "E": E, "k": rng.randint(1, min(8, E)),
                "mask": rng.random() < 0.5}
    if kind in ("ln_fwd", "ln_bwd"):
        N = _log(rng, 33, 16384)
        x, w = rng.choice([("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
        return {"kind": kind, "M": _log(rng, 1, max(1, min(32768, 33_000_000 // N))), "N": N,
                "x": x, "w": w}
    if kind == "clip":
        return {"kind": kind, "tensors": rng.randint(1, 48), "numel": _log(rng, 1000, 200_000_000),
                "types": rng.choice(["bf16", "fp32", "mixed"]), "bite": rng.random() < 0.5}
    if kind == "fp8_infer":
        return {"kind": kind, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 8192),
                "K": _log(rng, 64, 8192)}
    return {"kind": kind, "M": _log(rng, 16, 8192), "N": _log(rng, 128, 8192),
            "K": _log(rng, 128, 4096)}


def _clip_sizes(case):
    """Element counts of the tensors: a few large ones and a tail of small ones, the total
    about case["numel"]; shares fall by half, so that sizes spread over the logarithm."""
    n, total = case["tensors"], case["numel"]
    share = np.array([0.5 ** min(i, 12) for i in range(n)])
    return [max(1, int(total * s / share.sum())) | 1 for s in share]


def _clip_types(case):
    n = case["tensors"]
    if case["types"] != "mixed":
        return [TYPES[case["types"]]] * n
    return [BF16 if i % 5 < 3 else F32 for i in range(n)]  # experts' bf16, routers' and norms' fp32


# ------------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kind = case["kind"]
    st = {"kind": kind, "case": case}
    if own:
        import grouped_gemm_device_gb300 as lib
        st["lib"] = lib

    def normal(*shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    if kind == "router":
        T, E, k = case["T"], case["E"], case["k"]
        rank = torch.randperm(E, generator=g, device=DEV) + 1
        logits = normal(T, E) - 1.1 * torch.log(rank.float())  # some experts are more popular
        top, ids = torch.topk(logits, k, dim=1)
        st.update(logits=logits, ids=ids.to(torch.int32), probs=torch.softmax(top, dim=1),
                  d_probs=normal(T, k, scale=1e-3), coef=0.01,
                  mask=(torch.rand(T, generator=g, device=DEV) < 0.9) if case["mask"] else None,
                  d_loss=torch.rand(1, generator=g, device=DEV) + 0.5)
        if own:  # the plan: the loss's buffers for up to T tokens
            st["plan"] = st["lib"].RouterLoss(E, k, T, coef=st["coef"])
    elif kind in ("ln_fwd", "ln_bwd"):
        M, N = case["M"], case["N"]
        xt, wt = TYPES[case["x"]], TYPES[case["w"]]
        # a residual stream: a mean beside its spread, rows of different size
        x = (normal(M, N) * (0.5 + torch.rand(M, 1, generator=g, device=DEV)) + 0.5).to(xt)
        st.update(x=x, gamma=(1 + normal(N, scale=0.1)).to(wt), beta=normal(N, scale=0.1).to(wt))
        if kind == "ln_bwd":
            mean = x.float().mean(1)
            rstd = torch.rsqrt((x.float() - mean[:, None]).square().mean(1) + LN_EPS)
            st.update(dy=normal(M, N, dtype=xt), mean=mean, rstd=rstd)  # saved by the forward
        if own:
            st["plan"] = st["lib"].LayerNorm(N, M, dtype=xt, weight_dtype=wt, eps=LN_EPS)
    elif kind == "clip":
        grads = [normal(n, dtype=t, scale=1e-2 * 2.0 ** -(i % 4))
                 for i, (n, t) in enumerate(zip(_clip_sizes(case), _clip_types(case)))]
        norm = math.sqrt(sum(t.numel() * (1e-2 * 2.0 ** -(i % 4)) ** 2
                             for i, t in enumerate(grads)))
        st.update(grads=grads, max_norm=norm * (0.37 if case["bite"] else 3.0))
        # clipped gradients go to buffers of their own; where the norm is within the limit the
        # gradients stay in place, so that a pass can be repeated on the same state
        st["outs"] = [torch.empty_like(t) for t in grads] if case["bite"] else grads
        if own:
            st["plan"] = st["lib"].GradClip(grads, st["outs"])
    else:
        M, N, K = case["M"], case["N"], case["K"]
        st["x"] = normal(M, K, dtype=BF16)
        w = normal(N, K, dtype=BF16, scale=0.02)
        if kind == "fp8_train":
            st.update(w=w, dy=normal(M, N, dtype=BF16, scale=1e-2))
            if own:
                st["plan"] = st["lib"].Fp8Linear(N, K, M)
        elif own:  # serving keeps the quantised weights
            st["plan"] = st["lib"].Fp8Linear(N, K, M, train=False)
            st["plan"].set_weight(w)
        else:
            st["wq"] = _quant_2d(w)
    return st


# ------------------------------------------------------------------------------- one pass
def run(st):
    return (_own if own else _plain)(st)


def _own(st):
    kind, plan = st["kind"], st["plan"]
    if kind == "router":
        loss, counts, mean_prob = plan.forward(st["logits"], st["ids"], st["mask"])
        d_logits = plan.backward(st["logits"], st["ids"], st["probs"], st["d_probs"],
                                 st["mask"], d_loss=st["d_loss"])
        return {"loss": loss, "counts": counts, "mean_prob": mean_prob, "d_logits": d_logits}
    if kind == "ln_fwd":
        y, mean, rstd = plan.forward(st["x"], st["gamma"], st["beta"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "ln_bwd":
        dx, dgamma, dbeta = plan.backward(st["dy"], st["x"], st["gamma"], st["mean"], st["rstd"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if kind == "clip":
        return {"norm": plan.clip(st["max_norm"]), "grads": st["outs"]}
    if kind == "fp8_infer":
        return {"y": plan.forward(st["x"])}
    plan.set_weight(st["w"])
    y = plan.forward(st["x"])
    dx, dw = plan.backward(st["dy"])
    return {"y": y, "dx": dx, "dw": dw}


def _plain(st):
    kind = st["kind"]
    if kind == "router":
        return _router_plain(st)
    if kind == "ln_fwd":
        x = st["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = torch.rsqrt((c * c).mean(1) + LN_EPS)
        y = c * rstd[:, None] * st["gamma"].float() + st["beta"].float()
        return {"y": y.to(st["x"].dtype), "mean": mean, "rstd": rstd}
    if kind == "ln_bwd":
        dy, wt = st["dy"].float(), st["gamma"].dtype
        xhat = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
        dyg = dy * st["gamma"].float()
        dx = st["rstd"][:, None] * (dyg - dyg.mean(1, keepdim=True)
                                    - xhat * (dyg * xhat).mean(1, keepdim=True))
        return {"dx": dx.to(st["x"].dtype), "dgamma": (dy * xhat).sum(0).to(wt),
                "dbeta": dy.sum(0).to(wt)}
    if kind == "clip":
        sums = torch.stack([t.float().square().sum() for t in st["grads"]])
        norm = sums.sum().sqrt()
        coef = torch.clamp(st["max_norm"] / (norm + CLIP_EPS), max=1.0)
        return {"norm": norm.reshape(1),
                "grads": [(t.float() * coef).to(t.dtype) for t in st["grads"]]}
    if kind == "fp8_infer":
        return {"y": (_quant_row(st["x"]) @ st["wq"].t()).to(BF16)}
    wq, x, dy = _quant_2d(st["w"]), st["x"], st["dy"]
    y = (_quant_row(x) @ wq.t()).to(BF16)
    dx = (_quant_row(dy) @ wq).to(BF16)
    dw = (_quant_row(dy.t()) @ _quant_row(x.t()).t()).to(BF16)  # blocks along the tokens
    return {"y": y, "dx": dx, "dw": dw}


def _router_plain(st):
    logits, ids, c = st["logits"], st["ids"].long(), st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    m = torch.ones(T, device=DEV) if st["mask"] is None else st["mask"].float()
    nv = m.sum()
    ex = torch.exp(logits - logits.amax(1, keepdim=True))
    p = ex / ex.sum(1, keepdim=True)
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    counts.index_add_(0, ids.reshape(-1), m.to(torch.int32).repeat_interleave(k))
    inv = 1.0 / torch.clamp(nv, min=1.0)
    mean_prob = (p * m[:, None]).sum(0) * inv
    f = counts.float() * (E / k) * inv
    loss = st["coef"] * (f * mean_prob).sum()
    d = (st["d_loss"] * st["coef"] * inv) * m[:, None] * p * (f - (p * f).sum(1, keepdim=True))
    w, dw = st["probs"], st["d_probs"]
    d.scatter_add_(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    return {"loss": loss.reshape(1), "counts": counts, "mean_prob": mean_prob, "d_logits": d}


def _blocks(x, rows):
    """x in blocks of rows x 128, zeros to fill them: [blocks of rows, rows, blocks, 128]."""
    M, N = x.shape
    Mp, Np = -(-M // rows) * rows, -(-N // 128) * 128
    v = torch.nn.functional.pad(x.float(), (0, Np - N, 0, Mp - M))
    return v.view(Mp // rows, rows, Np // 128, 128)


def _quant(x, rows):
    """The values that E4M3 codes with one scale for each block of rows x 128 stand for:
    scale amax / 448, codes the nearest E4M3 of v * (448 / amax), each step in 32 bits."""
    M, N = x.shape
    v = _blocks(x, rows)
    amax = v.abs().amax(dim=(1, 3), keepdim=True).clamp(min=FP8_TINY)
    top = torch.full_like(amax, FP8_MAX)  # a tensor: one IEEE division, not a reciprocal
    q = (v * (top / amax)).to(torch.float8_e4m3fn).float() * (amax / top)
    return q.reshape(v.shape[0] * rows, -1)[:M, :N]


def _quant_row(x):
    return _quant(x, 1)


def _quant_2d(w):
    return _quant(w, 128)


# ------------------------------------------------------------------------------- cost
def work(case):
    kind = case["kind"]
    if kind == "router":
        T, E, k = case["T"], case["E"], case["k"]
        # logits read, their gradient written; ids, probabilities and their gradient; the mask
        return {"bytes": T * (8 * E + 12 * k + (1 if case["mask"] else 0)) + 12 * E,
                "flops": 12 * T * E}
    if kind in ("ln_fwd", "ln_bwd"):
        M, N = case["M"], case["N"]
        xb, wb = (2 if case["x"] == "bf16" else 4), (2 if case["w"] == "bf16" else 4)
        if kind == "ln_fwd":
            return {"bytes": 2 * M * N * xb + 2 * N * wb + 8 * M, "flops": 8 * M * N}
        return {"bytes": 3 * M * N * xb + 3 * N * wb + 8 * M, "flops": 14 * M * N}
    if kind == "clip":
        by = sum(n * (2 if t is BF16 else 4)
                 for n, t in zip(_clip_sizes(case), _clip_types(case)))
        n = sum(_clip_sizes(case))
        return {"bytes": by * (2 if case["bite"] else 1) + 4, "flops": n * (3 if case["bite"] else 2)}
    M, N, K = case["M"], case["N"], case["K"]
    nb = -(-N // 128) * -(-K // 128)
    if kind == "fp8_infer":
        return {"bytes": 2 * M * K + N * K + 4 * nb + 2 * M * N, "flops": 2 * M * N * K}
    # masters, x and dy read; y, dx and dw written
    return {"bytes": 2 * N * K + 2 * M * K + 2 * M * N + 2 * M * N + 2 * M * K + 2 * N * K,
            "flops": 6 * M * N * K}


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    kept, own = own, False  # the inputs alone
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    kind = case["kind"]
    if kind == "router":
        return _exact_router(st, case)
    if kind in ("ln_fwd", "ln_bwd"):
        x = st["x"].to(F64)
        gamma = st["gamma"].to(F64)
        if kind == "ln_fwd":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            sd = torch.sqrt(var + LN_EPS)
            y = (x - mean.unsqueeze(1)).div_(sd.unsqueeze(1)).mul_(gamma).add_(st["beta"].to(F64))
            return {"y": y, "mean": mean, "rstd": sd.reciprocal()}
        N = case["N"]
        r = st["rstd"].to(F64).unsqueeze(1)
        h = (x - st["mean"].to(F64).unsqueeze(1)).mul_(r)
        dy = st["dy"].to(F64)
        a = torch.einsum("mn,n->m", dy, gamma) / N
        b = torch.einsum("mn,mn,n->m", dy, h, gamma) / N
        dx = (dy * gamma - a.unsqueeze(1) - h * b.unsqueeze(1)) * r
        return {"dx": dx, "dgamma": torch.einsum("mn,mn->n", dy, h), "dbeta": dy.sum(dim=0)}
    if kind == "clip":
        total = 0.0
        for t in st["grads"]:
            for part in t.split(1 << 26):
                total += float(torch.dot(part.to(F64), part.to(F64)))
        norm = math.sqrt(total)
        c = min(1.0, st["max_norm"] / (norm + CLIP_EPS))
        return {"norm": torch.tensor([norm], dtype=F64, device=DEV),
                "grads": [t.to(F64) * c for t in st["grads"]]}
    x = _codes64(st["x"], False)
    if kind == "fp8_infer":
        return {"y": x @ st["wq"].to(F64).t()}
    w = _codes64(st["w"], True)
    dy, dyt = _codes64(st["dy"], False), _codes64(st["dy"].t(), False)
    xt = _codes64(st["x"].t(), False)
    return {"y": x @ w.t(), "dx": dy @ w, "dw": dyt @ xt.t()}


def _codes64(x, square):
    """Dequantised values in 64 bits. Which code a value gets is decided by the definition's two
    32-bit roundings (the factor 448 / amax, and the product with it); a column block at a time."""
    x = x.to(F32)
    M, N = x.shape
    out = torch.empty(M, N, dtype=F64, device=DEV)
    for c0 in range(0, N, 128):
        blk = x[:, c0:c0 + 128]
        amax = blk.abs().max(dim=1).values
        if square:
            pad = (-M) % 128
            amax = torch.cat([amax, amax.new_zeros(pad)]).view(-1, 128).max(dim=1).values
            amax = amax.repeat_interleave(128)[:M]
        amax = torch.where(amax < FP8_TINY, torch.full_like(amax, FP8_TINY), amax)
        top = torch.full_like(amax, FP8_MAX)
        code = torch.mul(blk, torch.div(top, amax).unsqueeze(1))
        scale = torch.div(amax, top).to(F64).unsqueeze(1)
        out[:, c0:c0 + 128] = _nearest_e4m3(code.to(F64)) * scale
    return out


def _nearest_e4m3(v):
    """The E4M3 value nearest to each v, ties to even mantissas, at most 448 in magnitude."""
    a = v.abs()
    _, e = torch.frexp(a)                       # a = m * 2^e, m in [0.5, 1)
    step = torch.ldexp(torch.ones_like(a), torch.clamp(e, min=-5) - 4)  # 3 mantissa bits
    return torch.sign(v) * torch.clamp(torch.round(a / step) * step, max=FP8_MAX)


def _exact_router(st, case):
    T, E, k = case["T"], case["E"], case["k"]
    p = torch.softmax(st["logits"].to(F64), dim=1)
    valid = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"]
    n = max(int(valid.sum()), 1)
    ids = st["ids"].long()
    counts = torch.bincount(ids[valid].flatten(), minlength=E)
    f = counts.to(F64) * E / (k * n)
    mean_prob = p[valid].sum(dim=0) / n
    loss = st["coef"] * torch.dot(f, mean_prob)
    g = float(st["d_loss"]) * st["coef"] / n
    d = p * (f.unsqueeze(0) - (p @ f).unsqueeze(1)) * g
    d[~valid] = 0.0
    w, dw = st["probs"].to(F64), st["d_probs"].to(F64)
    d.scatter_add_(1, ids, w * dw - w * torch.einsum("tk,tk->t", w, dw).unsqueeze(1))
    return {"loss": loss.reshape(1), "counts": counts.to(torch.int32), "mean_prob": mean_prob,
            "d_logits": d}
