"""A gated expert layer on 4-bit weights and activations: the residual stream normalised, tokens routed by an 8-bit router, sorted by
expert, encoded once, multiplied by their experts' matrices, gated, encoded again, multiplied back, and combined with the
router's weights. Then, at the same sizes, the gradients that a trained router and what lies before the layer need: of the combine,
the routing, the gather and the norm.

    python examples/expert_layer.py [--tokens 64] [--experts 32] [--slots 4] [--hidden 1024] [--inner 768] [--mx]

Random weights; the result is compared with the same layer on the values the codes stand for."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_weight_pn3t_gb300 as pnq  # noqa: E402


class ExpertLayer:
    """Weights [experts][out][in] encoded once; a call takes tokens, router choices and weights."""

    def __init__(self, kind, gate_up, down, x_scale, h_scale):
        self.kind, self.x_scale, self.h_scale = kind, x_scale, h_scale
        scale = lambda w: float(w.abs().max()) / (6 * 448) if kind == pnq.NVFP4 else 1.0  # noqa: E731
        self.gate_up = pnq.fp4_quantize(kind, gate_up, scale(gate_up))
        self.down = pnq.fp4_quantize(kind, down, scale(down))
        self.experts, self.inner = gate_up.shape[0], down.shape[2]

    def rows(self, x, plan):
        """The experts' outputs, sorted rows: [tokens * slots][hidden] bf16."""
        q = pnq.fp4_quantize(self.kind, x, self.x_scale, plan=plan)
        h = pnq.fp4_gemm_experts(q, self.gate_up, plan, dtype=torch.bfloat16)
        h = torch.nn.functional.silu(h[:, :self.inner]) * h[:, self.inner:]
        q = pnq.fp4_quantize(self.kind, h, self.h_scale, plan=plan, sorted=True)  # the rows are in expert order already
        return pnq.fp4_gemm_experts(q, self.down, plan, dtype=torch.bfloat16)

    def __call__(self, x, ids, weights):
        plan = pnq.expert_sort(ids, self.experts)
        return pnq.expert_combine(self.rows(x, plan), plan, weights), plan


def reference(layer, x, plan, weights):
    """The layer in fp64 on the decoded values (activations encoded and decoded by the same calls)."""
    kind = layer.kind
    decode = lambda m: pnq.fp4_dequantize(m).double()  # noqa: E731
    gate_up = decode(layer.gate_up).view(layer.experts, -1, x.shape[1])
    down = decode(layer.down).view(layer.experts, x.shape[1], -1)
    xv = decode(pnq.fp4_quantize(kind, x, layer.x_scale))
    off = plan.offsets.tolist()
    order = plan.order[:off[-1]].long()
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(layer.experts):
        slot = order[off[e]:off[e + 1]]
        if not len(slot):
            continue
        h = (xv[slot // plan.slots] @ gate_up[e].T).to(torch.bfloat16)
        h = torch.nn.functional.silu(h[:, :layer.inner]) * h[:, layer.inner:]
        hv = decode(pnq.fp4_quantize(kind, h.contiguous(), layer.h_scale))
        out = (hv @ down[e].T) * weights.view(-1)[slot, None].double()
        y.index_add_(0, slot // plan.slots, out)
    return y


def run(tokens=64, experts=32, slots=4, hidden=1024, inner=768, kind=None, seed=0):
    kind = pnq.NVFP4 if kind is None else kind
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    layer = ExpertLayer(kind, r(experts, 2 * inner, hidden) * hidden ** -0.5, r(experts, hidden, inner) * inner ** -0.5,
                        6.0 / (6 * 448) if kind == pnq.NVFP4 else 1.0, 8.0 / (6 * 448) if kind == pnq.NVFP4 else 1.0)
    # what comes in and the residual stream, added and normalised: as they are for the experts, in 8 bits for the router
    norm, router = 1 + 0.1 * r(hidden), pnq.int8_quantize(r(experts, hidden) * hidden ** -0.5)
    x, stream = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda"), r(tokens, hidden).to(torch.bfloat16)
    codes, scales, total = pnq.rms_norm_int8(r(tokens, hidden).to(torch.bfloat16), norm, residual=stream, y=x)
    logits = pnq.int8_gemm(codes, scales, *router)
    ids, weights = pnq.expert_route(logits, slots, renormalize=True)
    y, plan = layer(x, ids, weights)
    want = reference(layer, x, plan, weights)
    err = float((y.double() - want).norm() / want.norm())

    # training around frozen experts: the gradient of the combine reaches the experts' rows and the router's logits, that of
    # the gather the tokens (here through experts that pass their rows on), and that of the norm the residual stream
    xs = pnq.expert_gather(x, plan)
    dy = r(tokens, hidden).to(torch.bfloat16)
    dys, dweights = pnq.expert_combine_backward(dy, xs, plan, weights)
    dx = pnq.expert_gather_backward(dys, plan)
    dlogits = pnq.expert_route_backward(dweights, logits, ids, renormalize=True)
    _, _, rstd = pnq.rms_norm(total, norm)
    dstream, dnorm = pnq.rms_norm_backward(dx, total, norm, rstd, dtotal=dy)
    assert all(bool(g.isfinite().all()) for g in (dlogits, dstream, dnorm))
    whole = float((dx.double() - dy.double() * weights.sum(-1, keepdim=True).double()).norm() / dx.double().norm())
    assert pnq.device_error() == 0
    return err, whole, dweights


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 64), ("experts", 32), ("slots", 4), ("hidden", 1024), ("inner", 768)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--mx", action="store_true", help="MXFP4 instead of NVFP4")
    a = ap.parse_args()
    err, whole, dweights = run(a.tokens, a.experts, a.slots, a.hidden, a.inner, pnq.MXFP4 if a.mx else pnq.NVFP4)
    print(f"layer against fp64 on the decoded values: {err:.2e} of its norm (bf16 rows and sums)")
    print(f"gradient through gather and combine: {whole:.2e}; router gradients {tuple(dweights.shape)}")


if __name__ == "__main__":
    main()
