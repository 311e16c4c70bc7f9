"""Measured cases of the 4-bit microscaled product and of the expert layer around it.

Operators
  quantise  x (bf16 or fp32, rows possibly strided) -> 4-bit codes with one scale per group of 16 (NVFP4, E4M3 scales) or
            32 (MXFP4, power-of-two scales), read back as the values they stand for
  product   Y = X W^T of two such matrices (tokens x weights)
  experts   the same product for an expert layer: tokens sorted by expert, quantised on the way, multiplied by their expert
  dispatch  tokens sorted by expert and gathered, with the gradient of the gather
  combine   expert rows back to their tokens with the router's weights applied, with both gradients

A case is a dict of plain values; `prepare` makes its inputs from a seed, `run` is one pass (plain torch where `own` is
false, this package's kernels where it is true), `exact` the same outputs from the definitions in 64 bits.

Formats. y = fp32(x r), r = fp32(1 / g) for the matrix's global scale g. A group's scale is e4m3(fp32(amax |y| / 6)),
nearest, ties to the even word, at most 448 (NVFP4), or 2^(floor(log2 amax) - 2) (MXFP4). Each code is the nearest E2M1
value of y / s, ties to the even word, saturating at 6; a zero scale has zero codes. A value is fp32(e2m1 s g).
Codes are packed two a byte along K, low nibble first, rows padded to 16 bytes. Scales are kept in blocks of 128 rows by
four groups, 512 bytes each: row r, group j of a block at byte 16 (r % 32) + 4 (r / 32) + j; blocks of one row range
follow each other along K; every matrix (expert) starts a new row range.

A plan of an expert layer (tokens T, k slots each, E experts; n = T k) is one int32 buffer: offsets [E + 1] (first sorted row
of each expert), block_start [E + 1] (first 128-row scale block), order [n] (slot of each sorted row, -1 past the end),
position [n] (sorted row of each slot, -1 for a dropped slot), scale_row [n] (row of each sorted row in the tiled scales)."""
import math

import numpy as np
import torch

own = False

NVFP4, MXFP4 = 1004, 1006
GROUP = {NVFP4: 16, MXFP4: 32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
FLOATS = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEVICE = "cuda"


def listed():
    return [
        # one token's activations on their way into a 5120-wide projection: the latency of a call
        {"name": "quantise token", "op": "quantise", "type": NVFP4, "rows": 1, "K": 5120, "stride": 5120, "x": "bf16"},
        # a prefill's rows cut out of a wider fp32 buffer: an odd row count and a stride of its own
        {"name": "quantise strided rows", "op": "quantise", "type": MXFP4, "rows": 8191, "K": 5152, "stride": 6144, "x": "fp32"},
        # one decoded token through the 17408-wide projection: the weights' bytes
        {"name": "product token", "op": "product", "type": NVFP4, "M": 1, "N": 17408, "K": 5120, "out": "fp32"},
        # a small batch through the projection back, the long sum
        {"name": "product batch", "op": "product", "type": MXFP4, "M": 13, "N": 5120, "K": 17408, "out": "fp32"},
        # odd sizes on every axis, rows of codes that need padding
        {"name": "product ragged", "op": "product", "type": NVFP4, "M": 333, "N": 1001, "K": 2064, "out": "bf16"},
        # a prefill of 8192 tokens: the arithmetic
        {"name": "product prefill", "op": "product", "type": NVFP4, "M": 8192, "N": 17408, "K": 5120, "out": "bf16"},
        # a decode step of a few sequences over many experts, most of them with one or two rows
        {"name": "experts decode", "op": "experts", "type": NVFP4, "T": 12, "k": 8, "E": 128, "N": 1536, "K": 2048, "skew": 0.5, "drop": 0.0, "out": "bf16"},
        # a prefill's tokens over experts of uneven load, some slots dropped at capacity
        {"name": "experts prefill", "op": "experts", "type": MXFP4, "T": 4096, "k": 8, "E": 64, "N": 1408, "K": 2048, "skew": 1.0, "drop": 0.02, "out": "bf16"},
        # a small step's routing
        {"name": "dispatch decode", "op": "dispatch", "T": 33, "k": 8, "E": 256, "D": 2048, "skew": 0.5, "drop": 0.0, "x": "bf16"},
        # a training step's routing with its gradient
        {"name": "dispatch train", "op": "dispatch", "T": 16384, "k": 8, "E": 128, "D": 2048, "skew": 1.0, "drop": 0.02, "x": "bf16"},
        # the way back of a few odd-sized fp32 rows
        {"name": "combine decode", "op": "combine", "T": 7, "k": 6, "E": 60, "D": 1999, "skew": 0.5, "drop": 0.1, "x": "fp32"},
        # the way back of a training step with the gradients of the rows and of the router's weights
        {"name": "combine train", "op": "combine", "T": 16384, "k": 8, "E": 128, "D": 2048, "skew": 1.0, "drop": 0.02, "x": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("quantise", "product", "product", "experts", "dispatch", "combine"))
    kind = rng.choice((NVFP4, MXFP4))
    g = GROUP[kind]
    if op == "quantise":
        K = g * max(1, _log(rng, 64, 17408) // g)
        return {"op": op, "type": kind, "rows": min(_log(rng, 1, 8192), 42_000_000 // K), "K": K,
                "stride": K + rng.choice((0, 0, 1, 8, 1000)), "x": rng.choice(("bf16", "fp32"))}
    if op == "product":
        M, N, K = _log(rng, 1, 8192), _log(rng, 1, 17408), g * max(1, _log(rng, 64, 17408) // g)
        while M * N * K > 8192 * 17408 * 5120 // 2:
            M, N = max(1, M * 2 // 3), max(1, N * 4 // 5)
        return {"op": op, "type": kind, "M": M, "N": N, "K": K, "out": rng.choice(("fp32", "bf16"))}
    case = {"op": op, "T": 0, "k": rng.randint(1, 8), "E": _log(rng, 8, 256), "skew": rng.choice((0.0, 0.5, 1.0)),
            "drop": rng.choice((0.0, 0.0, 0.05))}
    if op == "experts":
        case["E"] = min(case["E"], 128)
        N, K = _log(rng, 32, 2048), g * max(1, _log(rng, 64, 4096) // g)
        T = min(_log(rng, 1, 4096), max(1, 4096 * 8 * 1408 * 2048 // (case["k"] * N * K)))
        return case | {"type": kind, "T": T, "N": N, "K": K, "out": rng.choice(("fp32", "bf16"))}
    D = _log(rng, 16, 6144)
    return case | {"T": min(_log(rng, 1, 16384), 16384 * 2048 // D), "D": D, "x": rng.choice(("bf16", "fp32"))}


# ---- the layouts ------------------------------------------------------------------------------

def _up(a, b):
    return -(-a // b) * b


def _blocks(rows, K, kind):
    """(128-row blocks, four-group chunks) of the tiled scales of one matrix."""
    return -(-rows // 128), -(-K // (4 * GROUP[kind]))


def _tile(scales):
    """Scale words [matrices][rows][groups] -> the tiled bytes, padding zero."""
    E, R, G = scales.shape
    full = scales.new_zeros((E, _up(R, 128), _up(G, 4)))
    full[:, :R, :G] = scales
    return full.view(E, -1, 4, 32, full.shape[2] // 4, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(-1)


def _untile(tiled, rows, groups, matrices=1):
    """The tiled bytes -> scale words [matrices][rows][groups]."""
    rb, c = -(-rows // 128), -(-groups // 4)
    return tiled.view(matrices, rb, c, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(matrices, rb * 128, c * 4)[:, :rows, :groups]


def _pack(codes):
    """4-bit codes [rows][K] -> bytes [rows][pitch]."""
    R, K = codes.shape
    out = codes.new_zeros((R, _up(K // 2, 16)))
    out[:, :K // 2] = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return out


def _unpack(codes, K):
    return torch.stack((codes & 15, codes >> 4), -1).view(codes.shape[0], -1)[:, :K]


# ---- the plain forms, in 32 bits ----------------------------------------------------------------

def _scale_value(words, kind):
    """fp32 values of scale words."""
    if kind == NVFP4:
        return words.view(torch.float8_e4m3fn).to(torch.float32)
    return torch.where(words == 255, math.nan, torch.exp2(words.to(torch.float32) - 127.0))


def _quantise(x, kind, g):
    """x [rows][K] -> (codes [rows][K], scale words [rows][K / group])."""
    R, K = x.shape
    y = (x.to(torch.float32) * float(np.float32(1.0) / np.float32(g))).reshape(R, -1, GROUP[kind])
    amax = y.abs().amax(-1)
    if kind == NVFP4:
        scale = torch.clamp(amax / torch.full_like(amax, 6.0), max=448.0).to(torch.float8_e4m3fn)
        words, s = scale.view(torch.uint8), scale.to(torch.float32)
    else:
        words = torch.where(amax > 0, torch.frexp(amax)[1] + 124, 0).clamp(0, 254).to(torch.uint8)
        s = _scale_value(words, kind)
    s = s[..., None]
    t = torch.where(s > 0, y.abs() / s, 0.0)
    code = (t > 0.25).to(torch.uint8)
    code += t >= 0.75
    code += t > 1.25
    code += t >= 1.75
    code += t > 2.5
    code += t >= 3.5
    code += t > 5.0
    code += (torch.signbit(y) & (s > 0)).to(torch.uint8) * 8
    return code.reshape(R, K), words


def _values(codes, words, kind, g):
    """fp32 values of codes [rows][K] and scale words [rows][groups]."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    s = _scale_value(words, kind).repeat_interleave(GROUP[kind], 1)
    return grid[codes.to(torch.int32)] * s * g


def _operand_values(codes, scales, rows, K, kind, g, matrices=1):
    words = _untile(scales, rows, K // GROUP[kind], matrices).reshape(matrices * rows, -1)
    return _values(_unpack(codes, K), words, kind, g)


def _plan(ids, E):
    """The plan buffer of ids [T][k] (torch operations; ids outside 0 .. E - 1 are dropped)."""
    n = ids.numel()
    flat = ids.reshape(-1).to(torch.int64)
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(flat, stable=True)
    count = (flat[:, None] == torch.arange(E, device=flat.device)[None, :]).sum(0)
    zero = count.new_zeros(1)
    offsets = torch.cat((zero, count.cumsum(0)))
    blocks = torch.cat((zero, ((count + 127) // 128).cumsum(0)))
    rows = torch.arange(n, device=flat.device)
    kept = rows < offsets[E]
    expert = flat[order].clamp(max=E - 1)
    scale_row = torch.where(kept, rows - offsets[expert] + 128 * blocks[expert], -1)
    position = torch.empty_like(order)
    position[order] = torch.where(kept, rows, -1)
    return torch.cat((offsets, blocks, torch.where(kept, order, -1), position, scale_row)).to(torch.int32)


def _parts(plan, n, E):
    return torch.split(plan, (E + 1, E + 1, n, n, n))


# ---- inputs --------------------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _activations(gen, rows, K, stride=None):
    """Activations as a normalised layer gives them: unit noise, a tenth of the channels several times louder."""
    loud = 1.0 + 6.0 * (torch.rand(stride or K, generator=gen, device=DEVICE) < 0.1)
    return (torch.randn(rows, stride or K, generator=gen, device=DEVICE) * loud)[:, :K]


def _route(gen, T, k, E, skew, drop):
    """k different experts for each token (fewer than k where there are fewer experts), loads uneven by `skew`; dropped slots are -1."""
    logits = torch.randn(T, E, generator=gen, device=DEVICE) + skew * torch.randn(E, generator=gen, device=DEVICE)
    ids = torch.full((T, k), -1, dtype=torch.int32, device=DEVICE)
    ids[:, :min(k, E)] = logits.topk(min(k, E), -1).indices.to(torch.int32)
    ids[torch.rand(T, k, generator=gen, device=DEVICE) < drop] = -1
    return ids


def _global(x, kind):
    """The global scale a calibration gives: the largest value at the top of both formats (none for MXFP4)."""
    return float(x.abs().max()) / (6.0 * 448.0) if kind == NVFP4 else 1.0


def _matrix(x, kind, matrices=1):
    """x [matrices * rows][K] as a quantised operand: (codes, tiled scales, global scale)."""
    g = _global(x, kind)
    codes, words = _quantise(x, kind, g)
    return _pack(codes), _tile(words.view(matrices, x.shape[0] // matrices, -1)), g


def prepare(case, seed):
    gen, op = _generator(seed), case["op"]
    state = {"case": case}
    if op == "quantise":
        x = _activations(gen, case["rows"], case["K"], case["stride"])
        return state | {"g": _global(x, case["type"]), "x": x.to(FLOATS[case["x"]])}
    if op == "product":
        state["x"] = _matrix(_activations(gen, case["M"], case["K"]), case["type"])
        state["w"] = _matrix(0.02 * torch.randn(case["N"], case["K"], generator=gen, device=DEVICE), case["type"])
        return state
    T, k, E = case["T"], case["k"], case["E"]
    ids = _route(gen, T, k, E, case["skew"], case["drop"])
    if op == "experts":
        x = _activations(gen, T, case["K"])
        w = 0.02 * torch.randn(E * case["N"], case["K"], generator=gen, device=DEVICE)
        return state | {"ids": ids, "g": _global(x, case["type"]), "x": x.to(torch.bfloat16), "w": _matrix(w, case["type"], E)}
    kind = FLOATS[case["x"]]
    rows = torch.randn(T * k, case["D"], generator=gen, device=DEVICE).to(kind)
    token = torch.randn(T, case["D"], generator=gen, device=DEVICE).to(kind)
    if op == "dispatch":
        return state | {"ids": ids, "x": token, "dxs": rows}
    weights = torch.rand(T, k, generator=gen, device=DEVICE)
    return state | {"plan": _plan(ids, E), "ys": rows, "dy": token, "weights": weights / weights.sum(-1, keepdim=True)}


# ---- one pass --------------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import block_quantized_weight_pn3t_gb300 as pnq

    c = state["case"]
    op = c["op"]
    if op == "quantise":
        return pnq.fp4_dequantize(pnq.fp4_quantize(c["type"], state["x"], state["g"]))
    if op == "product":
        x = pnq.Fp4Matrix(c["type"], c["M"], c["K"], *state["x"])
        w = pnq.Fp4Matrix(c["type"], c["N"], c["K"], *state["w"])
        return pnq.fp4_gemm(x, w, dtype=FLOATS[c["out"]])
    if op == "experts":
        plan = pnq.expert_sort(state["ids"], c["E"])
        x = pnq.fp4_quantize(c["type"], state["x"], state["g"], plan=plan)
        w = pnq.Fp4Matrix(c["type"], c["N"], c["K"], *state["w"], matrices=c["E"])
        return {"offsets": plan.offsets, "y": pnq.fp4_gemm_experts(x, w, plan, dtype=FLOATS[c["out"]])}
    if op == "dispatch":
        plan = pnq.expert_sort(state["ids"], c["E"])
        xs = pnq.expert_gather(state["x"], plan)
        dx = pnq.expert_gather_backward(state["dxs"], plan)
        return {"offsets": plan.offsets, "order": plan.order, "position": plan.position, "xs": xs, "dx": dx}
    plan = pnq.ExpertPlan(c["T"], c["k"], c["E"], state["plan"])
    y = pnq.expert_combine(state["ys"], plan, state["weights"])
    dys, dweights = pnq.expert_combine_backward(state["dy"], state["ys"], plan, state["weights"])
    return {"y": y, "dys": dys, "dweights": dweights}


def _run_plain(state):
    c = state["case"]
    op, kind = c["op"], c.get("type")
    if op == "quantise":
        return _values(*_quantise(state["x"], kind, state["g"]), kind, state["g"])
    if op == "product":
        x = _operand_values(*state["x"][:2], c["M"], c["K"], kind, state["x"][2])
        w = _operand_values(*state["w"][:2], c["N"], c["K"], kind, state["w"][2])
        return (x @ w.T).to(FLOATS[c["out"]])
    T, k, E = c["T"], c["k"], c["E"]
    n = T * k
    if op == "combine":
        _, _, order, position, _ = _parts(state["plan"], n, E)
        kept = (position >= 0)[:, None]
        rows = torch.where(kept, state["ys"][position.clamp(min=0)].to(torch.float32), 0.0).view(T, k, -1)
        dy = state["dy"].to(torch.float32)
        y = (rows * state["weights"][..., None]).sum(1)
        dweights = (rows * dy[:, None, :]).sum(-1)
        slot = order.clamp(min=0)
        dys = torch.where((order >= 0)[:, None], dy[slot // k] * state["weights"].view(-1)[slot][:, None], 0.0)
        return {"y": y.to(state["ys"].dtype), "dys": dys.to(state["ys"].dtype), "dweights": dweights}
    plan = _plan(state["ids"], E)
    offsets, _, order, position, _ = _parts(plan, n, E)
    token = order.clamp(min=0) // k
    if op == "dispatch":
        xs = torch.where((order >= 0)[:, None], state["x"][token], 0.0).to(state["x"].dtype)
        rows = torch.where((position >= 0)[:, None], state["dxs"][position.clamp(min=0)].to(torch.float32), 0.0)
        return {"offsets": offsets, "order": order, "position": position, "xs": xs, "dx": rows.view(T, k, -1).sum(1).to(state["x"].dtype)}
    x = _values(*_quantise(state["x"], kind, state["g"]), kind, state["g"])
    w = _operand_values(*state["w"][:2], c["N"], c["K"], kind, state["w"][2], E).view(E, c["N"], c["K"])
    # each expert's rows, padded to the largest expert's, in one batched product
    offsets = offsets.to(torch.int64)
    rows = torch.arange(n, device=x.device)
    expert = torch.searchsorted(offsets[1:], rows, right=True).clamp(max=E - 1)
    within = rows - offsets[expert]
    kept = order >= 0
    padded = x.new_zeros((E, max(1, int((offsets[1:] - offsets[:-1]).max())), c["K"]))
    padded[expert[kept], within[kept]] = x[token[kept]]
    y = x.new_zeros((n, c["N"]))
    y[kept] = torch.bmm(padded, w.transpose(1, 2))[expert[kept], within[kept]]
    return {"offsets": offsets.to(torch.int32), "y": y.to(FLOATS[c["out"]])}


# ---- what a pass cannot do without -----------------------------------------------------------------

def _operand_bytes(rows, K, kind):
    return rows * (K // 2 + K // GROUP[kind])


def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "quantise":
        each = case["rows"] * case["K"]
        # read x, write the codes and scales, read them back, write the values
        return {"bytes": each * (size[case["x"]] + 4) + 2 * _operand_bytes(case["rows"], case["K"], case["type"]), "flops": 4 * each}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _operand_bytes(M + N, K, case["type"]) + M * N * size[case["out"]], "flops": 2 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    n = T * k
    plan = 4 * (2 * (E + 1) + 3 * n)
    if op == "experts":
        N, K = case["N"], case["K"]
        # experts that a token reaches, were the choices even
        used = E * (1.0 - (1.0 - min(k, E) / E) ** T)
        return {"bytes": 4 * n + plan + T * K * 2 + 2 * _operand_bytes(n, K, case["type"]) + used * _operand_bytes(N, K, case["type"])
                + n * N * size[case["out"]], "flops": 2 * n * N * K}
    each = size[case["x"]] * case["D"]
    if op == "dispatch":
        return {"bytes": 4 * n + plan + 2 * (T + n) * each, "flops": n * case["D"]}
    # forward: rows, weights -> y; backward: dy, rows, weights -> dys, dweights
    return {"bytes": plan + 12 * n + (3 * n + 2 * T) * each, "flops": 5 * n * case["D"]}


# ---- the same from the definitions, in 64 bits -------------------------------------------------------

def _nearest(v, table):
    """The nearest of the rising `table`'s values to each v >= 0, ties to the even place, past the end the last: its place."""
    table = torch.tensor(table, dtype=torch.float64, device=v.device)
    at = torch.searchsorted(table, v).clamp(max=len(table) - 1)
    low = (at - 1).clamp(min=0)
    down, up = v - table[low], table[at] - v
    return torch.where((down < up) | ((down == up) & (low % 2 == 0)), low, at)


_E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _exact_quantised(x, kind, g):
    """The values in 64 bits that quantised x stands for."""
    step = GROUP[kind]
    y = (x.to(torch.float64) * float(np.float32(1.0) / np.float32(g))).to(torch.float32).to(torch.float64).unflatten(1, (-1, step))
    top = y.abs().max(-1, keepdim=True).values
    if kind == NVFP4:
        table = torch.tensor(_E4M3, dtype=torch.float64, device=x.device)
        s = table[_nearest((top / 6.0).to(torch.float32).to(torch.float64), _E4M3)]
    else:
        s = torch.where(top > 0, torch.ldexp(torch.ones_like(top), (torch.frexp(top)[1] - 3).clamp(min=-127)), 2.0 ** -127)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    v = torch.where(s > 0, grid[_nearest(torch.where(s > 0, y.abs() / s, 0.0), E2M1)], 0.0)
    return (torch.sign(y) * v * s * g).flatten(1)


def _exact_operand(codes, scales, g, rows, K, kind, matrices=1):
    """The values in 64 bits of an operand, read place by place."""
    r = torch.arange(matrices * rows, device=codes.device)
    r = (r // rows) * _up(rows, 128) + r % rows
    j = torch.arange(K // GROUP[kind], device=codes.device)
    chunks = _blocks(rows, K, kind)[1]
    at = ((r // 128)[:, None] * chunks + (j // 4)[None, :]) * 512 + ((r % 32) * 16 + (r // 32 % 4) * 4)[:, None] + (j % 4)[None, :]
    word = scales[at].to(torch.int64)
    if kind == NVFP4:
        s = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device=codes.device)[word]
    else:
        s = torch.ldexp(torch.ones(word.shape, dtype=torch.float64, device=codes.device), word - 127)
    kk = torch.arange(K, device=codes.device)
    code = (codes[:, kk // 2] >> (4 * (kk % 2)).to(torch.uint8)) & 15
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    return grid[code.to(torch.int64)].unflatten(1, (-1, GROUP[kind])).mul_(s[..., None]).flatten(1).mul_(g)


def exact(case, seed):
    state = prepare(case, seed)
    op, kind = case["op"], case.get("type")
    if op == "quantise":
        return _exact_quantised(state["x"], kind, state["g"])
    if op == "product":
        x = _exact_operand(*state["x"], case["M"], case["K"], kind)
        return torch.matmul(x, _exact_operand(*state["w"], case["N"], case["K"], kind).T)
    T, k, E = case["T"], case["k"], case["E"]
    n = T * k
    if op == "combine":
        position = _parts(state["plan"], n, E)[3].view(T, k).to(torch.int64)
        y = torch.zeros((T, case["D"]), dtype=torch.float64, device=DEVICE)
        dys = torch.zeros((n, case["D"]), dtype=torch.float64, device=DEVICE)
        dweights = torch.zeros((T, k), dtype=torch.float64, device=DEVICE)
        dy, weights = state["dy"].to(torch.float64), state["weights"].to(torch.float64)
        for j in range(k):
            at = (position[:, j] >= 0).nonzero()[:, 0]
            rows = state["ys"][position[at, j]].to(torch.float64)
            y[at] += weights[at, j, None] * rows
            dweights[at, j] = (dy[at] * rows).sum(-1)
            dys[position[at, j]] = weights[at, j, None] * dy[at]
        return {"y": y, "dys": dys, "dweights": dweights}
    # tokens of each expert in the order of their slots
    ids = state["ids"].reshape(-1).cpu().numpy()
    lists = [np.nonzero(ids == e)[0] for e in range(E)]
    order = torch.from_numpy(np.concatenate(lists)).to(DEVICE)
    if op == "dispatch":
        xs = torch.zeros((n, case["D"]), dtype=torch.float64, device=DEVICE)
        xs[:order.numel()] = state["x"][order // k].to(torch.float64)
        dx = torch.zeros((T, case["D"]), dtype=torch.float64, device=DEVICE)
        dx.index_add_(0, order // k, state["dxs"][:order.numel()].to(torch.float64))
        return {"offsets": None, "order": None, "position": None, "xs": xs, "dx": dx}
    x = _exact_quantised(state["x"], kind, state["g"])
    codes, scales, g = state["w"]
    codes, scales = codes.view(E, case["N"], -1), scales.view(E, -1)
    y, at = torch.zeros((n, case["N"]), dtype=torch.float64, device=DEVICE), 0
    for e in range(E):
        if len(lists[e]):
            w = _exact_operand(codes[e], scales[e], g, case["N"], case["K"], kind)
            y[at:at + len(lists[e])] = x[torch.from_numpy(lists[e]).to(DEVICE) // k] @ w.T
            at += len(lists[e])
    return {"offsets": None, "y": y}
