"""More operators of an expert block's step: cases, inputs, plain forms and 64-bit values.

  route       the choice of experts: softmax or sigmoid scores, a bias for balance, groups of
              experts, top-k, renormalised weights, tokens per expert
  route_grad  the gradient of the router's logits, on its own or added to the balance loss's
  norm_fwd    the residual stream and the branch that joins it: a norm and a gate of the branch, the
              sum, and the norm before the next block
  norm_bwd    its backward pass, with the gradients of both norms' weights and of the gate
  adamw       an AdamW step over a list of tensors, states in 32 or in 8 bits

`own` selects the framework's kernels; otherwise run() is the plain form in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64, I32, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64
TYPES = {"bf16": BF16, "fp32": F32}
NORM_EPS = 1e-6
WEIGHT_EPS = 1e-20                  # added to the sum that sigmoid scores are divided by
SCALE = 0.5                         # of the branch in the residual stream
LR, BETA1, BETA2, ADAM_EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.1
STEPS = 100                         # steps done before the measured one
CLIP_EPS = 1e-6                     # added to the norm before the division
BLOCK = 256                         # values that share a scale in an 8-bit state
NAN_SCALE, LOW_SCALE = 255, 32      # scale of a block that is not finite; the smallest one
SEED = 20240607


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token through DeepSeek-V3's router
        {"name": "route_token", "kind": "route", "T": 1, "E": 256, "k": 8, "logits": "fp32",
         "score": "sigmoid", "bias": True, "groups": 8, "of_groups": 4, "group_top": 2,
         "renorm": True, "scale": 2.5, "mask": False},
        # a GPT-OSS-shaped router on its training batch, logits as its bf16 projection leaves them,
        # some tokens padding
        {"name": "route_gptoss", "kind": "route", "T": 16384, "E": 128, "k": 4, "logits": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "of_groups": 1, "group_top": 1,
         "renorm": True, "scale": 1.0, "mask": True},
        # DeepSeek-V3's router over sixteen micro-batches of 4096 tokens
        {"name": "route_dsv3", "kind": "route", "T": 65536, "E": 256, "k": 8, "logits": "fp32",
         "score": "sigmoid", "bias": True, "groups": 8, "of_groups": 4, "group_top": 2,
         "renorm": True, "scale": 2.5, "mask": False},
        # a small router whose weights are the probabilities themselves
        {"name": "route_grad_tiny", "kind": "route_grad", "T": 512, "E": 4, "k": 2,
         "logits": "fp32", "score": "softmax", "renorm": False, "scale": 1.0, "mask": False,
         "add": False},
        # DeepSeek-V3's again, added to what the balance loss has left
        {"name": "route_grad_dsv3", "kind": "route_grad", "T": 65536, "E": 256, "k": 8,
         "logits": "fp32", "score": "sigmoid", "renorm": True, "scale": 2.5, "mask": True,
         "add": True},
        # one decoded token at DeepSeek-V3's hidden size
        {"name": "norm_fwd_token", "kind": "norm_fwd", "M": 1, "N": 7168, "x": "bf16",
         "o": "bf16", "w": "bf16", "post": False, "gate": False},
        # the GPT-OSS-shaped batch on an fp32 residual stream, norms on both sides of the block and
        # a gate for each token
        {"name": "norm_fwd_gptoss", "kind": "norm_fwd", "M": 16384, "N": 2880, "x": "fp32",
         "o": "bf16", "w": "fp32", "post": True, "gate": True},
        # Mixtral's training batch, backward
        {"name": "norm_bwd_mixtral", "kind": "norm_bwd", "M": 8192, "N": 4096, "x": "bf16",
         "o": "bf16", "w": "bf16", "post": False, "gate": False},
        # an odd width and an odd number of tokens, norms on both sides and a gate, backward
        {"name": "norm_bwd_odd", "kind": "norm_bwd", "M": 3001, "N": 4095, "x": "bf16",
         "o": "bf16", "w": "bf16", "post": True, "gate": True},
        # the small tensors of a block (router, norms, biases)
        {"name": "adamw_small", "kind": "adamw", "tensors": 12, "numel": 60_001, "types": "fp32",
         "grads": "same", "bits": 32, "clip": "idle"},
        # an expert layer's weights in bf16 with fp32 masters, the small tensors beside them; states
        # in 32 bits, gradients clipped: the largest
        {"name": "adamw_layer", "kind": "adamw", "tensors": 10, "numel": 402_653_184,
         "types": "mixed", "grads": "same", "bits": 32, "clip": "bite"},
        # a quarter of it with states in 8 bits
        {"name": "adamw_layer_8bit", "kind": "adamw", "tensors": 10, "numel": 100_663_296,
         "types": "mixed", "grads": "same", "bits": 8, "clip": "bite"},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]; one in three made odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v if rng.random() < 0.67 else max(lo, v | 1 if v < hi else v)


def draw(rng):
    kind = rng.choice(["route", "route", "route_grad", "norm_fwd", "norm_bwd", "adamw", "adamw"])
    if kind in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8]) if kind == "route" else 1
        E = _log(rng, 2, 256) if groups == 1 else groups * _log(rng, 2, 256 // groups)
        k = rng.randint(1, min(8, E))
        of = max(rng.randint(1, groups), -(-k * groups // E))
        c = {"kind": kind, "T": _log(rng, 1, 65536), "E": E, "k": k,
             "logits": rng.choice(["fp32", "bf16"]), "score": rng.choice(["softmax", "sigmoid"])}
        if kind == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, of_groups=of,
                     group_top=rng.choice([1, 2]) if groups > 1 else 1)
        c.update(renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                 mask=rng.random() < 0.5)
        if kind == "route_grad":
            c["add"] = rng.random() < 0.5
        return c
    if kind in ("norm_fwd", "norm_bwd"):
        N = _log(rng, 33, 16384)
        x, o, w = rng.choice([("bf16", "bf16", "bf16"), ("bf16", "bf16", "fp32"),
                              ("fp32", "bf16", "fp32"), ("fp32", "fp32", "fp32")])
        return {"kind": kind, "M": _log(rng, 1, max(1, min(32768, 33_000_000 // N))), "N": N,
                "x": x, "o": o, "w": w, "post": rng.random() < 0.5, "gate": rng.random() < 0.5}
    bits = rng.choice([32, 8])
    return {"kind": kind, "tensors": rng.randint(1, 12),
            "numel": _log(rng, 1000, 100_000_000 if bits == 32 else 50_000_000),
            "types": rng.choice(["bf16", "fp32", "mixed"]), "grads": rng.choice(["same", "fp32"]),
            "bits": bits, "clip": rng.choice(["none", "idle", "bite"])}


def _sizes(case):
    """Element counts of the tensors: a few large ones and a tail of small ones, the total about
    case["numel"]; shares fall by half, so that sizes spread over the logarithm."""
    n, total = case["tensors"], case["numel"]
    share = [0.5 ** min(i, 12) for i in range(n)]
    return [max(1, int(total * s / sum(share))) | 1 for s in share]


def _param_types(case):
    n = case["tensors"]
    if case["types"] != "mixed":
        return [TYPES[case["types"]]] * n
    return [BF16 if i % 5 < 3 else F32 for i in range(n)]  # experts' bf16, routers' and norms' fp32


def _grad_types(case):
    return [F32 if case["grads"] == "fp32" else t for t in _param_types(case)]


def _decays(case):
    return [DECAY if i % 5 < 3 else 0.0 for i in range(case["tensors"])]  # none for norms


# ------------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"kind": case["kind"], "case": case}
    if own:
        import grouped_gemm_device_gb300 as lib
        st["lib"] = lib

    def normal(*shape, dtype=F32, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    fill = {"route": _fill_route, "route_grad": _fill_route, "norm_fwd": _fill_norm,
            "norm_bwd": _fill_norm, "adamw": _fill_adamw}[case["kind"]]
    fill(st, case, normal, uniform, g)
    return st


def _fill_route(st, case, normal, uniform, g):
    T, E, k = case["T"], case["E"], case["k"]
    rank = torch.randperm(E, generator=g, device=DEV) + 1
    logits = (normal(T, E) - 1.1 * torch.log(rank.float())).to(TYPES[case["logits"]])
    mask = uniform(T) < 0.9 if case["mask"] else None
    st.update(logits=logits, mask=mask)
    if case["kind"] == "route":
        # what the balance has learnt: unpopular experts are preferred
        st["bias"] = 0.1 * torch.log(rank.float()) + normal(E, scale=0.01) if case["bias"] else None
    else:
        ids = torch.topk(logits.float() + uniform(T, E), k, dim=1).indices.to(I32)
        if mask is not None:
            ids[~mask] = -1
        st.update(ids=ids, d_weights=normal(T, k, scale=1e-3),
                  d_logits=normal(T, E, scale=1e-4) if case["add"] else None)
    if own:  # the plan: the choice's buffers for up to T tokens
        more = {} if case["kind"] == "route_grad" else {
            "n_group": case["groups"], "topk_group": case["of_groups"],
            "group_top": case["group_top"]}
        st["plan"] = st["lib"].RouterTopK(E, k, T, score=case["score"], renorm=case["renorm"],
                                          scale=case["scale"], dtype=logits.dtype, **more)


def _fill_norm(st, case, normal, uniform, g):
    M, N, post = case["M"], case["N"], case["post"]
    xt, ot, wt = TYPES[case["x"]], TYPES[case["o"]], TYPES[case["w"]]
    # a residual stream: rows of different size, a few large features
    x = (normal(M, N) * (0.5 + uniform(M, 1)) * (1 + 4 * (uniform(N) < 0.01))).to(xt)
    st.update(x=x, o=normal(M, N, dtype=ot, scale=0.7), w=(1 + normal(N, scale=0.1)).to(wt),
              wp=(1 + normal(N, scale=0.1)).to(wt) if post else None,
              gate=torch.sigmoid(normal(M)) if case["gate"] else None)
    if case["kind"] == "norm_bwd":  # x is what the forward has left
        st.update(dh=normal(M, N, dtype=ot, scale=1e-2), dx=normal(M, N, dtype=xt, scale=1e-2),
                  rstd=torch.rsqrt(x.float().square().mean(1) + NORM_EPS),
                  rstd_post=torch.rsqrt(st["o"].float().square().mean(1) + NORM_EPS) if post
                  else None)
    if own:
        st["plan"] = st["lib"].ResidualNorm(N, M, dtype=xt, branch_dtype=ot, weight_dtype=wt,
                                            post_norm=post, scale=SCALE, eps=NORM_EPS)


def _fill_adamw(st, case, normal, uniform, g):
    sizes, bits = _sizes(case), case["bits"]
    types = list(zip(_param_types(case), _grad_types(case)))
    masters = [normal(n, scale=0.02) for n in sizes]
    grads = [normal(n, dtype=t, scale=1e-3 * 2.0 ** -(i % 4))
             for i, (n, (_, t)) in enumerate(zip(sizes, types))]
    params = [p.to(t) if t is BF16 else p for p, (t, _) in zip(masters, types)]
    masters = [p if t is BF16 else None for p, (t, _) in zip(masters, types)]

    def codes(n, signed):  # magnitudes fall off by a few powers of two from a block's largest
        top, per = (127, 12) if signed else (255, 6)
        mag = (top - normal(n).abs_().mul_(per).to(I32)).clamp_(min=0).to(torch.uint8)
        if signed:
            mag |= (uniform(n) < 0.5).to(torch.uint8) << 7
        return mag

    def scales(n):
        return (115 + 3 * uniform(-(-n // BLOCK))).to(torch.uint8)

    if bits == 32:
        m = [normal(n, scale=5e-4 * 2.0 ** -(i % 4)) for i, n in enumerate(sizes)]
        v = [(normal(n, scale=5e-4 * 2.0 ** -(i % 4))).square_() for i, n in enumerate(sizes)]
        st.update(m=m, v=v)
    else:
        st.update(m=[codes(n, True) for n in sizes], v=[codes(n, False) for n in sizes],
                  m_exp=[scales(n) for n in sizes], v_exp=[scales(n) + 1 for n in sizes])
    norm = math.sqrt(sum(n * (1e-3 * 2.0 ** -(i % 4)) ** 2 for i, n in enumerate(sizes)))
    st.update(params=params, masters=masters, grads=grads,
              steps=torch.full((1,), STEPS, dtype=I64, device=DEV),
              norm=None if case["clip"] == "none" else torch.full((1,), norm, device=DEV),
              max_norm={"none": math.inf, "idle": 3.0 * norm, "bite": 0.37 * norm}[case["clip"]])
    if own:
        plan = st["plan"] = st["lib"].AdamW(
            params, grads, lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=_decays(case),
            state_bits=bits, masters=masters, seed=SEED)
        for name in ("m", "v") if bits == 32 else ("m", "v", "m_exp", "v_exp"):
            for mine, given in zip(getattr(plan, name), st.pop(name)):
                mine.copy_(given)
        plan.steps.copy_(st["steps"])


# ------------------------------------------------------------------------------- one pass
def run(st):
    return (_own if own else _plain)(st)


def _own(st):
    kind, plan = st["kind"], st["plan"]
    if kind == "route":
        ids, weights, counts = plan.forward(st["logits"], st["bias"], st["mask"])
        return {"ids": ids, "weights": weights, "counts": counts}
    if kind == "route_grad":
        return {"d_logits": plan.backward(st["logits"], st["d_weights"], st["ids"],
                                          add_to=st["d_logits"])}
    if kind == "norm_fwd":
        x, h = plan.forward(st["x"], st["o"], st["w"], st["wp"], st["gate"])
        return {"x": x, "h": h}
    if kind == "norm_bwd":
        dx, do, dw, dwp, d_gate = plan.backward(
            st["dh"], st["x"], st["o"], st["w"], st["wp"], st["gate"], dx_new=st["dx"],
            rstd=st["rstd"], rstd_post=st["rstd_post"])
        return {"dx": dx, "do": do, "dw": dw, "dwp": dwp, "d_gate": d_gate}
    plan.step(norm=st["norm"], max_norm=st["max_norm"])
    # 8-bit states come back as the values that the codes stand for, the second as its square root
    m, v = (plan.m, plan.v) if st["case"]["bits"] == 32 else plan.moments()
    return {"params": plan.params, "masters": st["masters"], "m": m, "v": v, "steps": plan.steps}


def _plain(st):
    return {"route": _route_plain, "route_grad": _route_grad_plain, "norm_fwd": _norm_plain,
            "norm_bwd": _norm_grad_plain, "adamw": _adamw_plain}[st["kind"]](st, st["case"])


def _pair_sum(x):
    """Row sums, neighbours in pairs and then pairs of pairs: an order that is part of the
    definition, as a choice between near scores goes by it."""
    E = x.shape[1]
    if E == 1:
        return x
    half = 1 << (E - 1).bit_length() - 1
    x = torch.nn.functional.pad(x, (0, 2 * half - E)).view(-1, half, 2)
    return _pair_sum(x[:, :, 0] + x[:, :, 1])


def _scores(x, score):
    """fp32 scores, each step one fp32 operation."""
    if score == "sigmoid":
        return torch.reciprocal(1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e * torch.reciprocal(_pair_sum(e))


def _route_plain(st, c):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = st["logits"].float()
    s = _scores(x, c["score"])
    value = s if st["bias"] is None else s + st["bias"]
    choice = x if st["bias"] is None else value  # the logits have the order of their scores
    if G > 1:
        by = choice if c["group_top"] == 1 else value
        best = by.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        chosen = best.sum(2).sort(dim=1, descending=True, stable=True).indices[:, :c["of_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, chosen, True)
        choice = choice.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if c["renorm"] and c["score"] == "sigmoid":
        w = w / (w.sum(1, keepdim=True) + WEIGHT_EPS)
    elif c["renorm"]:
        l = x.gather(1, ids)
        w = torch.exp(l - l.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    live = torch.ones(T, dtype=I32, device=DEV) if st["mask"] is None else st["mask"].to(I32)
    counts = torch.zeros(E, dtype=I32, device=DEV)
    counts.index_add_(0, ids.reshape(-1), live.repeat_interleave(k))
    on = live[:, None] > 0
    return {"ids": torch.where(on, ids, -1).to(I32), "weights": torch.where(on, w, 0.0),
            "counts": counts}


def _route_grad_plain(st, c):
    x, ids = st["logits"].float(), st["ids"].long()
    on, at = ids >= 0, ids.clamp(min=0)
    dw = torch.where(on, st["d_weights"], 0.0) * c["scale"]
    if c["score"] == "softmax" and c["renorm"]:
        l = x.gather(1, at).masked_fill(~on, -math.inf)
        top = l.amax(1, keepdim=True).clamp(min=-3e38)
        w = torch.exp(l - top)
        w = w / w.sum(1, keepdim=True).clamp(min=1e-38)
        d = torch.zeros_like(x).scatter_add_(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    elif c["score"] == "softmax":
        p = _scores(x, "softmax")
        ds = torch.zeros_like(x).scatter_add_(1, at, dw)
        d = p * (ds - (p * ds).sum(1, keepdim=True))
    else:
        s = torch.where(on, torch.reciprocal(1.0 + torch.exp(-x.gather(1, at))), 0.0)
        if c["renorm"]:
            total = s.sum(1, keepdim=True) + WEIGHT_EPS
            dw = (dw - (dw * s).sum(1, keepdim=True) / total) / total
        d = torch.zeros_like(x).scatter_add_(1, at, dw * s * (1.0 - s))
    return {"d_logits": d if st["d_logits"] is None else st["d_logits"] + d}


def _norm_plain(st, c):
    x, o, w = st["x"].float(), st["o"].float(), st["w"].float()
    if st["wp"] is not None:
        o = o * torch.rsqrt(o.square().mean(1, keepdim=True) + NORM_EPS) * st["wp"].float()
    q = SCALE if st["gate"] is None else SCALE * st["gate"][:, None]
    new = (x + q * o).to(st["x"].dtype)
    y = new.float()                          # the next norm is of the stream as it is kept
    h = y * torch.rsqrt(y.square().mean(1, keepdim=True) + NORM_EPS) * w
    return {"x": new, "h": h.to(st["o"].dtype)}


def _norm_grad_plain(st, c):
    wt = st["w"].dtype
    dh, o, r = st["dh"].float(), st["o"].float(), st["rstd"][:, None]
    y = st["x"].float() * r
    u = dh * st["w"].float()
    dx = st["dx"].float() + r * (u - y * (u * y).mean(1, keepdim=True))
    q = SCALE if st["gate"] is None else SCALE * st["gate"][:, None]
    e, dwp, rp = dx, None, 1.0
    if st["wp"] is not None:
        rp = st["rstd_post"][:, None]
        o = o * rp
        e = dx * st["wp"].float()
        dwp = (q * dx * o).sum(0).to(wt)
    dot = (e * o).sum(1, keepdim=True)
    do = q * e if st["wp"] is None else q * rp * (e - o * (dot / c["N"]))
    return {"dx": dx.to(st["x"].dtype), "do": do.to(st["o"].dtype), "dw": (dh * y).sum(0).to(wt),
            "dwp": dwp, "d_gate": None if st["gate"] is None else SCALE * dot[:, 0]}


def _mix(x):
    """32-bit hash of the low 32 bits of x (int64): shifts, exclusive ors and odd multipliers."""
    x = x & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0xF75341D5) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x99D5D0A1) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _stream(steps, tensor, n):
    """The 32 random bits of each of a tensor's first n elements in the step after `steps`."""
    lo, hi = torch.full_like(steps, SEED & 0xFFFFFFFF), torch.full_like(steps, SEED >> 32)
    key = _mix(_mix(_mix(lo ^ _mix(hi)) ^ (steps + 1)) + tensor)
    e = torch.arange(n, device=DEV)
    return _mix((e & 0xFFFFFFFF) ^ _mix(key ^ (e >> 32)))


def _decode(codes, exps, signed):
    """The fp32 values of 8-bit codes: the top bits of an fp32 number, less a base that the block's
    scale sets; code 0 is 0, a block of scale 255 is NaN."""
    top = 127 if signed else 255
    mag = (codes & top).to(I32)
    scale = exps.to(I32).repeat_interleave(BLOCK)[:codes.numel()]
    x = ((mag + (scale * 8 + 7 - top)) << 20).view(F32)
    x = torch.where(mag == 0, 0.0, x)
    if signed:
        x = torch.where(codes > 127, -x, x)
    return torch.where(scale == NAN_SCALE, math.nan, x)


def _encode(x, bits, signed):
    """Codes and scales of fp32 values; `bits`: 16 random ones for each, as whole numbers."""
    top, n = 127 if signed else 255, x.numel()
    mag = x.abs().view(I32)
    blocks = torch.nn.functional.pad(mag, (0, -n % BLOCK)).view(-1, BLOCK)
    exps = ((blocks.amax(1) + 0xFFFFF) >> 23).clamp(min=LOW_SCALE)
    base = (exps * 8 + 7 - top).repeat_interleave(BLOCK)[:n]
    least = ((base + 1) << 20).view(F32)
    up = ((mag + (bits << 4).to(I32)) >> 20) - base
    low = (bits.float() * (least * 2.0 ** -16) < x.abs()).to(I32)
    code = torch.where(x.abs() < least, low, up)
    if signed:
        code = code | ((x < 0) & (code > 0)).to(I32) << 7
    code = torch.where(exps.repeat_interleave(BLOCK)[:n] == NAN_SCALE, 0, code)
    return code.to(torch.uint8), exps.to(torch.uint8)


def _adamw_plain(st, c):
    t = st["steps"].to(F64) + 1
    a = (LR / -torch.expm1(t * math.log(BETA1))).float()
    rb = torch.rsqrt(-torch.expm1(t * math.log(BETA2))).float()
    factor = None
    if st["norm"] is not None:
        limit = torch.full_like(st["norm"], st["max_norm"])
        factor = torch.clamp(limit / (st["norm"] + CLIP_EPS), max=1.0)
    new = [_adamw_tensor(st, i, a, rb, factor, d) for i, d in enumerate(_decays(c))]
    st["steps"] += 1
    m, v = zip(*new)
    return {"params": st["params"], "masters": st["masters"], "m": list(m), "v": list(v),
            "steps": st["steps"]}


def _adamw_tensor(st, i, a, rb, factor, decay):
    g = st["grads"][i].float()
    if factor is not None:
        g = g * factor
    bits = None
    if st["case"]["bits"] == 32:
        m, v = st["m"][i], st["v"][i]
    else:
        bits = _stream(st["steps"], i, g.numel())
        m = _decode(st["m"][i], st["m_exp"][i], True)
        v = _decode(st["v"][i], st["v_exp"][i], False).square()
    m = m * BETA1 + g * (1 - BETA1)         # each product and the sum rounded to fp32
    v = v * BETA2 + (g * (1 - BETA2)) * g
    r = torch.sqrt(v)
    p = st["params"][i] if st["masters"][i] is None else st["masters"][i]
    p.copy_((p - p * (LR * decay)) - a * (m / (r * rb + ADAM_EPS)))
    if st["masters"][i] is not None:
        st["params"][i].copy_(p)            # rounded to bf16
    if bits is None:
        st["m"][i].copy_(m)
        st["v"][i].copy_(v)
        return st["m"][i], st["v"][i]
    st["m"][i], st["m_exp"][i] = _encode(m, bits & 0xFFFF, True)
    st["v"][i], st["v_exp"][i] = _encode(r, bits >> 16, False)
    # four significant bits: exact in bf16
    return (_decode(st["m"][i], st["m_exp"][i], True).to(BF16),
            _decode(st["v"][i], st["v_exp"][i], False).to(BF16))


# ------------------------------------------------------------------------------- cost
def work(case):
    kind = case["kind"]
    if kind in ("route", "route_grad"):
        T, E, k, mask = case["T"], case["E"], case["k"], case["mask"]
        lb = 2 if case["logits"] == "bf16" else 4
        if kind == "route":  # logits and mask read; ids and weights written; bias and counts
            return {"bytes": T * (lb * E + 8 * k + (1 if mask else 0)) + 8 * E,
                    "flops": 4 * T * E}
        # the chosen logits alone unless every probability has a gradient
        whole = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * (lb * (E if whole else k) + 8 * k + 4 * E * (2 if case["add"] else 1)),
                "flops": 2 * T * E}
    if kind in ("norm_fwd", "norm_bwd"):
        M, N, post, gate = case["M"], case["N"], case["post"], case["gate"]
        xb, ob, wb = (2 if case[t] == "bf16" else 4 for t in ("x", "o", "w"))
        rows = (4 + 4 * post + 4 * gate) * M
        weights = N * wb * (2 if post else 1)
        if kind == "norm_fwd":
            return {"bytes": M * N * 2 * (xb + ob) + weights + rows, "flops": 10 * M * N}
        return {"bytes": M * N * 3 * (xb + ob) + 2 * weights + rows + 4 * gate * M,
                "flops": 20 * M * N}
    total = 0
    for n, p, t in zip(_sizes(case), _param_types(case), _grad_types(case)):
        total += n * ((4 if t is F32 else 2) + 8 + (2 if p is BF16 else 0))  # gradient, fp32 value
        # states read and written; 8-bit ones also returned as bf16 values
        total += 16 * n if case["bits"] == 32 else 8 * n + 4 * -(-n // BLOCK)
    return {"bytes": total, "flops": 16 * sum(_sizes(case))}


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    kept, own = own, False  # the inputs alone
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    return {"route": _route_exact, "route_grad": _route_grad_exact, "norm_fwd": _norm_exact,
            "norm_bwd": _norm_grad_exact, "adamw": _adamw_exact}[case["kind"]](st, case)


def _route_exact(st, case):
    """Weights of the experts that the definition's fp32 steps choose; those steps taken in 64 bits
    and rounded after each (53 bits hold twice 24 and two more, so the second rounding is
    harmless)."""
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    x = st["logits"].to(F64)
    if case["score"] == "sigmoid":
        s32 = (1 / (1 + torch.exp(-x.to(F32)).to(F64)).to(F32).to(F64)).to(F32).to(F64)
        s = torch.sigmoid(x)
    else:
        e = torch.exp((x - x.max(dim=1, keepdim=True).values).to(F32)).to(F64)
        total = e
        while total.shape[1] > 1:
            odd = total.shape[1] % 2
            total = torch.cat([total, total.new_zeros(T, odd)], 1)
            total = (total[:, 0::2] + total[:, 1::2]).to(F32).to(F64)
        s32 = (e * (1 / total).to(F32).to(F64)).to(F32).to(F64)
        s = torch.softmax(x, dim=1)
    value, choice = s32, x
    if st["bias"] is not None:
        value = choice = (s32 + st["bias"].to(F64)).to(F32).to(F64)
    if G > 1:
        score = torch.full((T, G), -math.inf, dtype=F64, device=DEV)
        for j in range(G):
            part = slice(j * (E // G), (j + 1) * (E // G))
            if case["group_top"] == 1:
                score[:, j] = choice[:, part].max(dim=1).values
            else:
                two = torch.topk(value[:, part], 2, dim=1).values
                score[:, j] = (two[:, 0] + two[:, 1]).to(F32).to(F64)
        left = torch.full_like(choice, -math.inf)
        for _ in range(case["of_groups"]):
            j = _first_max(score)
            score[torch.arange(T, device=DEV), j] = -math.inf
            inside = torch.arange(E, device=DEV)[None, :] // (E // G) == j[:, None]
            left = torch.where(inside, choice, left)
        choice = left
    choice = choice.clone()
    ids = torch.empty(T, k, dtype=I64, device=DEV)
    for j in range(k):
        ids[:, j] = _first_max(choice)
        choice[torch.arange(T, device=DEV), ids[:, j]] = -math.inf
    w = s.gather(1, ids)
    if case["renorm"] and case["score"] == "sigmoid":
        w = w / (w.sum(dim=1, keepdim=True) + WEIGHT_EPS)
    elif case["renorm"]:
        w = torch.softmax(x.gather(1, ids), dim=1)
    on = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"]
    w = w * case["scale"] * on[:, None]
    counts = torch.bincount(ids[on].flatten(), minlength=E).to(I32)
    ids[~on] = -1
    return {"ids": ids.to(I32), "weights": w, "counts": counts}


def _first_max(x):
    """The lowest index of each row's maximum."""
    at = torch.arange(x.shape[1], device=DEV)
    return torch.where(x == x.max(dim=1, keepdim=True).values, at, x.shape[1]).min(dim=1).values


def _route_grad_exact(st, case):
    """The weights' product with their gradients, differentiated in 64 bits."""
    x = st["logits"].to(F64).requires_grad_()
    ids = st["ids"].to(I64)
    on, at = ids >= 0, ids.clamp(min=0)
    if case["score"] == "sigmoid":
        s = torch.sigmoid(x).gather(1, at) * on
        w = s / (s.sum(dim=1, keepdim=True) + WEIGHT_EPS) if case["renorm"] else s
    elif case["renorm"]:
        w = torch.softmax(x.gather(1, at), dim=1) * on  # a token's slots are dropped together
    else:
        w = torch.softmax(x, dim=1).gather(1, at) * on
    (d,) = torch.autograd.grad((w * st["d_weights"].to(F64)).sum() * case["scale"], x)
    return {"d_logits": d if st["d_logits"] is None else d + st["d_logits"].to(F64)}


def _norm_exact(st, case):
    N = case["N"]
    o = st["o"].to(F64)
    if case["post"]:
        o = o / torch.sqrt(torch.einsum("mn,mn->m", o, o) / N + NORM_EPS).unsqueeze(1)
        o = o * st["wp"].to(F64)
    q = torch.full((case["M"],), SCALE, dtype=F64, device=DEV)
    if case["gate"]:
        q = q * st["gate"].to(F64)
    new = torch.addcmul(st["x"].to(F64), o, q.unsqueeze(1))
    kept = new.to(st["x"].dtype).to(F64)
    root = torch.sqrt(torch.einsum("mn,mn->m", kept, kept) / N + NORM_EPS)
    return {"x": new, "h": kept * st["w"].to(F64) / root.unsqueeze(1)}


def _norm_grad_exact(st, case):
    N = case["N"]
    r = st["rstd"].to(F64).unsqueeze(1)
    y = st["x"].to(F64).mul_(r)
    dh, w = st["dh"].to(F64), st["w"].to(F64)
    dw = torch.einsum("mn,mn->n", dh, y)
    c = torch.einsum("mn,mn,n->m", dh, y, w).unsqueeze(1) / N
    dx = st["dx"].to(F64) + (dh * w - y * c) * r
    del dh, y
    o = st["o"].to(F64)
    q = torch.full((case["M"], 1), SCALE, dtype=F64, device=DEV)
    if case["gate"]:
        q = q * st["gate"].to(F64).unsqueeze(1)
    if not case["post"]:
        gate = SCALE * torch.einsum("mn,mn->m", dx, o) if case["gate"] else None
        return {"dx": dx, "do": dx * q, "dw": dw, "dwp": None, "d_gate": gate}
    rp, wp = st["rstd_post"].to(F64).unsqueeze(1), st["wp"].to(F64)
    o = o * rp
    dot = torch.einsum("mn,mn,n->m", dx, o, wp)
    do = (dx * wp - o * (dot / N).unsqueeze(1)) * (q * rp)
    return {"dx": dx, "do": do, "dw": dw, "dwp": torch.einsum("mn,mn,mo->n", dx, o, q),
            "d_gate": SCALE * dot if case["gate"] else None}


def _adamw_exact(st, case):
    t = STEPS + 1
    c = 1.0 if st["norm"] is None else min(1.0, st["max_norm"] / (float(st["norm"]) + CLIP_EPS))
    c1, c2 = 1 - BETA1 ** t, 1 - BETA2 ** t
    out = {"params": [], "masters": [], "m": [], "v": [], "steps": st["steps"] + 1}
    for i, decay in enumerate(_decays(case)):
        m, v, p = [], [], []
        value = st["params"][i] if st["masters"][i] is None else st["masters"][i]
        for lo in range(0, value.numel(), 1 << 26):  # whole blocks at a time
            part = slice(lo, min(lo + (1 << 26), value.numel()))
            g = st["grads"][i][part].to(F64) * c
            if case["bits"] == 32:
                m0, v0 = st["m"][i][part].to(F64), st["v"][i][part].to(F64)
            else:
                blocks = slice(part.start // BLOCK, -(-part.stop // BLOCK))
                m0 = _value64(st["m"][i][part], st["m_exp"][i][blocks], True)
                v0 = _value64(st["v"][i][part], st["v_exp"][i][blocks], False) ** 2
            m1, v1 = BETA1 * m0 + (1 - BETA1) * g, BETA2 * v0 + (1 - BETA2) * g * g
            x = value[part].to(F64)
            p.append(x * (1 - LR * decay) - LR * (m1 / c1) / (torch.sqrt(v1 / c2) + ADAM_EPS))
            if case["bits"] == 8:
                m1, v1 = _held64(st, i, part, m0, v0)
            m.append(m1)
            v.append(v1)
        p = torch.cat(p)
        out["params"].append(p)
        out["masters"].append(None if st["masters"][i] is None else p)
        out["m"].append(torch.cat(m))
        out["v"].append(torch.cat(v))
    return out


def _value64(codes, exps, signed):
    """(1 + fraction / 8) 2^exponent: the largest code's exponent is the scale's, each 8 codes below
    it are one less."""
    top = 127 if signed else 255
    mag = (codes & top).to(F64)
    scale = exps.to(F64).repeat_interleave(BLOCK)[:codes.numel()] - 127
    down = torch.floor((top - mag) / 8)
    x = (1 + (mag - (top - 7 - 8 * down)) / 8) * torch.exp2(scale - down) * (mag > 0)
    return torch.where(codes > 127, -x, x) if signed else x


def _held64(st, i, part, m0, v0):
    """The values that the new codes stand for. Which code a value gets is decided by the
    definition's fp32 steps, taken in 64 bits and rounded after each."""
    def r32(x):
        return x.to(F32).to(F64)

    def f32(x):
        return float(torch.tensor(x, dtype=F32))

    g = st["grads"][i][part].to(F64)
    if st["norm"] is not None:
        g = r32(g * min(1.0, f32(f32(st["max_norm"]) / f32(float(st["norm"]) + f32(CLIP_EPS)))))
    m = r32(r32(m0 * f32(BETA1)) + r32(g * f32(1 - BETA1)))
    v = r32(r32(r32(v0) * f32(BETA2)) + r32(r32(g * f32(1 - BETA2)) * g))
    n = g.numel()
    word = _stream(st["steps"], i, part.stop)[part.start:]
    held = []
    for x, u, binades in ((m, word % 65536, 127 / 8), (r32(torch.sqrt(v)), word // 65536, 255 / 8)):
        a = x.abs()
        _, e = torch.frexp(a)                              # a in [2^(e-1), 2^e)
        step = torch.exp2(e.to(F64) - 4)                   # eight values a power of two
        pad = torch.nn.functional.pad(torch.ceil(a / step) * step, (0, -n % BLOCK))
        top = torch.floor(torch.log2(pad.view(-1, BLOCK).max(dim=1).values.clamp(min=2.0 ** -95)))
        # the least value: eighths of a power of two, counted down from the largest code
        count = int(binades * 8) - 1
        low = (1 + (7 - count % 8) / 8) * torch.exp2(top - count // 8)
        low = low.repeat_interleave(BLOCK)[:n]
        down = torch.floor(a / step)
        # 16 of the 20 bits below a code's last one are compared
        frac = torch.floor((a / step - down) * 2.0 ** 20)
        near = (down + (frac + 16 * u.to(F64) >= 2.0 ** 20)) * step
        y = torch.where(a < low, (u.to(F64) * low < a * 65536) * low, near)
        held.append(torch.sign(x) * y)
    return held
