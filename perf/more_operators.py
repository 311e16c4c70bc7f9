"""Measured cases of the norms and encodes in front of 8-bit products, of the 8-bit product, and of the router of an expert layer.

Operators
  norm      root-mean-square norm of x (plus a residual) with its gradients, as a training step runs it
  norm8     the same norm as a serving step runs it: 8-bit codes with one scale per row, read back as the values they stand for
  quantise  rows -> 8-bit codes with one scale per row (activations between two products, weights once)
  product   Y = X W^T of two 8-bit matrices, a scale per token and per channel
  route     router logits -> each token's experts and their weights, for training with the gradient of the logits

A case is a dict of plain values; `prepare` makes its inputs from a seed, `run` is one pass (plain torch where `own` is
false, this package's kernels where it is true), `exact` the same outputs from the definitions in 64 bits.

Definitions. Norm: t = x + residual, rounded to x's type; r = 1 / sqrt(mean(t^2) + eps); y = t r w.
Codes: p = fp32(t w) (of an encode without a norm: p = x), scale = max |p| r / 127 (r = 1), code = the whole number nearest to
127 p / max |p|, ties to even: the norm's factor r is in the scale alone. A row of zeros has the scale 0 and the codes 0.
Product: y = (sum of the codes' products) x_scale w_scale, the sum exact.
Router: s = softmax(logits) or 1 / (1 + exp(-logits)); c = s + bias. With groups (equal runs of experts), a group's score is the
sum of its `best` largest c, and the `top_groups` best groups stay. The chosen experts are the k largest c of what stays,
in that order; ties go to the lowest index. Their weights are s, over their sum where renormalised, times `scale`."""
import math

import torch

own = False

FLOATS = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
SOFTMAX, SIGMOID = 0, 1
EPS = 1e-6
DEVICE = "cuda"


def listed():
    return [
        # one decoded token between two blocks of a 5120-wide model: the latency of a call
        {"name": "norm8 token", "op": "norm8", "rows": 1, "D": 5120, "x": "bf16", "w": "bf16", "residual": True},
        # a prefill of 8192 tokens: the bytes
        {"name": "norm8 prefill", "op": "norm8", "rows": 8192, "D": 5120, "x": "bf16", "w": "bf16", "residual": True},
        # a training step's norm with the gradients of x, residual and weight
        {"name": "norm train", "op": "norm", "rows": 16384, "D": 2048, "x": "bf16", "w": "fp32", "residual": True},
        # a few odd-sized fp32 rows, no residual
        {"name": "norm ragged", "op": "norm", "rows": 333, "D": 1999, "x": "fp32", "w": "fp32", "residual": False},
        # what a gated layer leaves for a small batch, cut out of the wider rows of gate and up
        {"name": "quantise batch", "op": "quantise", "rows": 13, "K": 17408, "stride": 34816, "x": "bf16"},
        # a projection's weights, once, when they are loaded: a scale per channel
        {"name": "quantise weights", "op": "quantise", "rows": 17408, "K": 5120, "stride": 5120, "x": "fp32"},
        # one decoded token through the 17408-wide projection: the weights' bytes
        {"name": "product token", "op": "product", "M": 1, "N": 17408, "K": 5120, "pad": True, "out": "bf16"},
        # a small batch through the projection back, the long sum
        {"name": "product batch", "op": "product", "M": 33, "N": 5120, "K": 17408, "pad": True, "out": "fp32"},
        # odd sizes on every axis
        {"name": "product ragged", "op": "product", "M": 333, "N": 1001, "K": 2063, "pad": True, "out": "bf16"},
        # a prefill of 8192 tokens: the arithmetic
        {"name": "product prefill", "op": "product", "M": 8192, "N": 17408, "K": 5120, "pad": True, "out": "bf16"},
        # a decode step of a few sequences, softmax scores
        {"name": "route decode", "op": "route", "T": 12, "E": 128, "k": 8, "score": SOFTMAX, "bias": False, "groups": 1, "top_groups": 1,
         "best": 1, "renormalise": True, "scale": 1.0, "x": "bf16", "train": False},
        # a training step: sigmoid scores, a bias for balance, groups, and the gradient of the logits
        {"name": "route train", "op": "route", "T": 16384, "E": 256, "k": 8, "score": SIGMOID, "bias": True, "groups": 8, "top_groups": 4,
         "best": 2, "renormalise": True, "scale": 2.5, "x": "fp32", "train": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("norm", "norm8", "quantise", "product", "product", "route", "route"))
    if op in ("norm", "norm8"):
        D = _log(rng, 16, 17408)
        return {"op": op, "rows": min(_log(rng, 1, 16384), 33_000_000 // D), "D": D, "x": rng.choice(("bf16", "fp32")),
                "w": rng.choice(("bf16", "fp32")), "residual": rng.choice((True, False))}
    if op == "quantise":
        K = _log(rng, 16, 17408)
        return {"op": op, "rows": min(_log(rng, 1, 17408), 80_000_000 // K), "K": K, "stride": K + rng.choice((0, 0, 1, 8, K)),
                "x": rng.choice(("bf16", "fp32"))}
    if op == "product":
        M, N, K = _log(rng, 1, 8192), _log(rng, 1, 17408), _log(rng, 16, 17408)
        if rng.random() < 0.7:
            K = -(-K // 16) * 16
        while M * N * K > 8192 * 17408 * 5120 // 2:
            M, N = max(1, M * 2 // 3), max(1, N * 4 // 5)
        return {"op": op, "M": M, "N": N, "K": K, "pad": rng.random() < 0.7, "out": rng.choice(("bf16", "fp32"))}
    groups = rng.choice((1, 1, 2, 4, 8))
    E = groups * max(2, _log(rng, 8, 512) // groups)
    top = rng.randint(max(1, groups // 2), groups)
    return {"op": op, "T": min(_log(rng, 1, 16384), 4_000_000 // E), "E": E, "k": rng.randint(1, min(8, E // groups * top)),
            "score": rng.choice((SOFTMAX, SIGMOID)), "bias": rng.choice((True, False)), "groups": groups, "top_groups": top,
            "best": rng.choice((1, 2)), "renormalise": rng.choice((True, False)), "scale": rng.choice((1.0, 2.5)),
            "x": rng.choice(("bf16", "fp32")), "train": rng.choice((True, False))}


# ---- inputs --------------------------------------------------------------------------------------

def _activations(gen, rows, K):
    """Activations as a residual stream has them: unit noise, a tenth of the channels several times louder."""
    loud = 1.0 + 6.0 * (torch.rand(K, generator=gen, device=DEVICE) < 0.1)
    return torch.randn(rows, K, generator=gen, device=DEVICE) * loud


def _codes(gen, rows, K, pad):
    """8-bit codes of normal values, each row's largest at the top of the range; rows padded to 16 bytes (the padding is not the operand's) or not."""
    x = torch.randn(rows, K, generator=gen, device=DEVICE)
    codes = torch.round(x * (127.0 / x.abs().amax(1, keepdim=True))).to(torch.int8)
    wide = torch.full((rows, -(-K // 16) * 16 if pad else K), 77, dtype=torch.int8, device=DEVICE)
    wide[:, :K] = codes
    return wide[:, :K]


def prepare(case, seed):
    gen, op = torch.Generator(device=DEVICE).manual_seed(int(seed)), case["op"]
    state = {"case": case}
    if op in ("norm", "norm8"):
        rows, D, kind = case["rows"], case["D"], FLOATS[case["x"]]
        state["x"] = _activations(gen, rows, D).to(kind)
        state["weight"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device=DEVICE)).to(FLOATS[case["w"]])
        state["residual"] = _activations(gen, rows, D).to(kind) if case["residual"] else None
        if op == "norm":
            state["dy"] = torch.randn(rows, D, generator=gen, device=DEVICE).to(kind)
            state["dtotal"] = torch.randn(rows, D, generator=gen, device=DEVICE).to(kind) if case["residual"] else None
        return state
    if op == "quantise":
        return state | {"x": _activations(gen, case["rows"], case["stride"]).to(FLOATS[case["x"]])[:, :case["K"]]}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        state["x"], state["w"] = _codes(gen, M, K, case["pad"]), _codes(gen, N, K, case["pad"])
        state["x_scales"] = 0.01 + 0.05 * torch.rand(M, generator=gen, device=DEVICE)
        state["w_scales"] = 0.0002 + 0.001 * torch.rand(N, generator=gen, device=DEVICE)
        return state
    T, E = case["T"], case["E"]
    logits = torch.randn(T, E, generator=gen, device=DEVICE) + 0.5 * torch.randn(E, generator=gen, device=DEVICE)
    state["logits"] = logits.to(FLOATS[case["x"]])
    state["bias"] = 0.1 * torch.randn(E, generator=gen, device=DEVICE) if case["bias"] else None
    state["dweights"] = torch.randn(T, case["k"], generator=gen, device=DEVICE) if case["train"] else None
    return state


# ---- one pass --------------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import block_quantized_weight_pn3t_gb300 as pnq

    c = state["case"]
    op = c["op"]
    if op == "norm":
        y, total, rstd = pnq.rms_norm(state["x"], state["weight"], EPS, state["residual"])
        dx, dweight = pnq.rms_norm_backward(state["dy"], total, state["weight"], rstd, state["dtotal"])
        return {"y": y, "total": total, "dx": dx, "dweight": dweight}
    if op == "norm8":
        codes, scales, total = pnq.rms_norm_int8(state["x"], state["weight"], EPS, state["residual"])
        return {"values": pnq.int8_dequantize(codes, scales), "scales": scales, "total": total}
    if op == "quantise":
        codes, scales = pnq.int8_quantize(state["x"])
        return {"values": pnq.int8_dequantize(codes, scales), "scales": scales}
    if op == "product":
        return pnq.int8_gemm(state["x"], state["x_scales"], state["w"], state["w_scales"], dtype=FLOATS[c["out"]])
    ids, weights = pnq.expert_route(state["logits"], c["k"], score=c["score"], bias=state["bias"], groups=c["groups"],
                                    top_groups=c["top_groups"], best=c["best"], renormalize=c["renormalise"], scale=c["scale"])
    if not c["train"]:
        return {"ids": ids, "weights": weights}
    dlogits = pnq.expert_route_backward(state["dweights"], state["logits"], ids, score=c["score"], renormalize=c["renormalise"],
                                        scale=c["scale"])
    return {"ids": ids, "weights": weights, "dlogits": dlogits}


# ---- the plain forms ---------------------------------------------------------------------------------

def _encode(p):
    """p fp32 -> (whole codes as fp32, max |p|). In 64 bits next to the border between two codes."""
    top = p.abs().amax(1, keepdim=True)
    t = p.to(torch.float64) * 127.0 / top.to(torch.float64)
    return torch.where(top > 0, torch.round(t), 0.0).to(torch.float32), top


def _run_plain(state):
    c = state["case"]
    op = c["op"]
    if op in ("norm", "norm8"):
        kind, weight = state["x"].dtype, state["weight"].to(torch.float32)
        total = state["x"] if state["residual"] is None else (state["x"].to(torch.float32) + state["residual"].to(torch.float32)).to(kind)
        t = total.to(torch.float32)
        rstd = 1.0 / torch.sqrt((t * t).mean(1, keepdim=True) + EPS)
        if op == "norm8":
            codes, top = _encode(t * weight)
            scales = top * rstd / 127.0
            return {"values": codes * scales, "scales": scales[:, 0], "total": total}
        dy = state["dy"].to(torch.float32)
        n = t * rstd
        g = dy * weight
        dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
        if state["dtotal"] is not None:
            dx = dx + state["dtotal"].to(torch.float32)
        return {"y": (n * weight).to(kind), "total": total, "dx": dx.to(kind), "dweight": (dy * n).sum(0)}
    if op == "quantise":
        codes, top = _encode(state["x"].to(torch.float32))
        scales = top / 127.0
        return {"values": codes * scales, "scales": scales[:, 0]}
    if op == "product":
        y = state["x"].to(torch.float32) @ state["w"].to(torch.float32).T
        return (y * state["x_scales"][:, None] * state["w_scales"]).to(FLOATS[c["out"]])
    # scores in 64 bits: which of two near ones is larger must not hang on a rounding
    T, E, k = c["T"], c["E"], c["k"]
    logits = state["logits"].to(torch.float64)
    if c["score"] == SOFTMAX:
        s = torch.exp(logits - logits.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-logits))
    choice = s if state["bias"] is None else s + state["bias"].to(torch.float64)
    if c["groups"] > 1:
        each = choice.view(T, c["groups"], -1)
        score = torch.sort(each, dim=2, descending=True)[0][:, :, :c["best"]].sum(2)
        kept = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        out = torch.ones_like(score, dtype=torch.bool).scatter_(1, kept, False)
        choice = each.masked_fill(out[:, :, None], -math.inf).view(T, E)
    ids = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    chosen = s.gather(1, ids)
    norm = chosen.sum(1, keepdim=True) if c["renormalise"] else 1.0
    weights = c["scale"] * chosen / norm
    found = {"ids": ids.to(torch.int32), "weights": weights.to(torch.float32)}
    if not c["train"]:
        return found
    s, weights = s.to(torch.float32), weights.to(torch.float32)
    dw = state["dweights"]
    d = c["scale"] * dw
    if c["renormalise"]:
        d = (d - (dw * weights).sum(1, keepdim=True)) / norm.to(torch.float32)
    ds = torch.zeros_like(s).scatter_(1, ids, d)
    dlogits = s * (ds - (ds * s).sum(1, keepdim=True)) if c["score"] == SOFTMAX else ds * s * (1.0 - s)
    return found | {"dlogits": dlogits.to(state["logits"].dtype)}


# ---- what a pass cannot do without -----------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm8"):
        n, b = case["rows"] * case["D"], SIZE[case["x"]]
        small = case["D"] * SIZE[case["w"]]
        added = 2 * n * b if case["residual"] else 0  # residual read, total written
        if op == "norm8":  # x -> codes and scales, and the values that the codes stand for in fp32
            return {"bytes": n * (b + 1) + added + n * (1 + 4) + small + 8 * case["rows"], "flops": 8 * n}
        # x -> y; dy, total -> dx (and the residual's gradient on the way), dweight
        return {"bytes": n * 2 * b + added + n * 3 * b + added // 2 + small * 2 + case["D"] * 4, "flops": 16 * n}
    if op == "quantise":
        n = case["rows"] * case["K"]
        return {"bytes": n * (SIZE[case["x"]] + 1) + n * (1 + 4) + 8 * case["rows"], "flops": 4 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K + 4) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    n = case["T"] * case["E"] * SIZE[case["x"]]
    chosen = case["T"] * case["k"]
    back = 2 * n + 8 * chosen if case["train"] else 0
    return {"bytes": n + 8 * chosen + back + (4 * case["E"] if case["bias"] else 0), "flops": 8 * case["T"] * case["E"] * (2 if case["train"] else 1)}


# ---- the same from the definitions, in 64 bits -------------------------------------------------------

def _exact_codes(p):
    """Codes of p (fp32 values in 64 bits): the whole number below and whether the rest is over a half of a step."""
    top = p.abs().amax(1, keepdim=True)
    twice = 254.0 * p.abs()
    low = torch.floor(torch.where(top > 0, 127.0 * p.abs() / top, 0.0))
    middle = (2.0 * low + 1.0) * top
    up = (twice > middle) | ((twice == middle) & (low % 2 == 1))
    return torch.sign(p) * torch.where(top > 0, low + up, 0.0), top[:, 0]


def exact(case, seed):
    state = prepare(case, seed)
    op, wide = case["op"], torch.float64
    if op in ("norm", "norm8"):
        total = state["x"]
        if state["residual"] is not None:
            total = (total.to(wide) + state["residual"].to(wide)).to(torch.float32).to(total.dtype)
        t, weight = total.to(wide), state["weight"].to(wide)
        D = case["D"]
        root = torch.sqrt(torch.einsum("rd,rd->r", t, t) / D + EPS)
        if op == "norm8":
            codes, top = _exact_codes((t * weight).to(torch.float32).to(wide))
            scales = top / (127.0 * root)
            return {"values": codes * scales[:, None], "scales": scales, "total": t}
        dy = state["dy"].to(wide)
        along = torch.einsum("rd,rd,d->r", dy, t, weight)  # how the row's length enters: d root = t dt / (D root)
        dx = dy * weight / root[:, None] - t * (along / (D * root ** 3))[:, None]
        if state["dtotal"] is not None:
            dx += state["dtotal"].to(wide)
        return {"y": t * weight / root[:, None], "total": t, "dx": dx, "dweight": torch.einsum("rd,rd,r->d", dy, t, 1.0 / root)}
    if op == "quantise":
        codes, top = _exact_codes(state["x"].to(wide))
        return {"values": codes * (top / 127.0)[:, None], "scales": top / 127.0}
    if op == "product":
        if case["M"] * case["N"] * case["K"] > 4_000_000_000_000:
            return None
        return (state["x"].to(wide) @ state["w"].to(wide).T) * torch.outer(state["x_scales"].to(wide), state["w_scales"].to(wide))
    T, k, G = case["T"], case["k"], case["groups"]
    logits = state["logits"].to(wide)
    if case["score"] == SOFTMAX:
        s = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True))
    else:
        s = torch.sigmoid(logits)
    choice = s.clone() if state["bias"] is None else s + state["bias"].to(wide)
    at = torch.arange(T, device=logits.device)
    if G > 1:
        each = choice.view(T, G, -1).clone()
        score = torch.zeros(T, G, dtype=wide, device=logits.device)
        for _ in range(min(case["best"], each.shape[2])):
            best = each.max(2)
            score += best.values
            each.scatter_(2, best.indices[:, :, None], -math.inf)
        stays = torch.zeros(T, G, dtype=torch.bool, device=logits.device)
        for _ in range(case["top_groups"]):
            best = score.argmax(1)
            stays[at, best], score[at, best] = True, -math.inf
        choice[~stays.repeat_interleave(choice.shape[1] // G, 1)] = -math.inf
    ids = torch.empty(T, k, dtype=torch.int64, device=logits.device)
    for j in range(k):
        ids[:, j] = choice.argmax(1)
        choice[at, ids[:, j]] = -math.inf
    weights = s.gather(1, ids)
    if case["renormalise"]:
        weights = weights / weights.sum(1, keepdim=True)
    if not case["train"]:
        return {"ids": None, "weights": case["scale"] * weights}
    # by the logarithm: d s_i / d logit_j = s_i (i == j) - s_i s_j, or s_i (1 - s_i) (i == j)
    pull = state["dweights"].to(wide) * case["scale"] * weights
    if case["renormalise"]:
        pull = pull - weights * pull.sum(1, keepdim=True)
    if case["score"] == SOFTMAX:
        dlogits = -s * pull.sum(1, keepdim=True)
    else:
        dlogits = torch.zeros_like(s)
        pull = pull * (1.0 - s.gather(1, ids))
    dlogits.scatter_add_(1, ids, pull)
    return {"ids": None, "weights": case["scale"] * weights, "dlogits": dlogits}
