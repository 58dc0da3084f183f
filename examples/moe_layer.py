"""One training step of a mixture-of-experts layer on this package's operators:

    out = x + sum_k w_k * expert_k(rmsnorm(x)),   expert(v) = (silu(v W1g) * (v W1u)) W2

The norm and the SwiGLU keep their inputs in 8 bits for the backward pass; tokens are packed by
expert and summed back with the router's weights. The rows that enter each of the experts' products
are quantized to NVFP4 with the amax that the dispatch and the SwiGLU already found: the operands of
block-scaled GEMMs. The experts' products below are plain torch products over each expert's BF16 rows,
and main() shows how far the operands are from those; moe_nvfp4_step.py multiplies the operands.

    python examples/moe_layer.py [--tokens 512 --hidden 1024 --width 512 --experts 8 --topk 2]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_block_scaled_quantize_gb300 import api  # noqa: E402


def expert_products(rows, weights, ends):
    """rows[e's range] @ weights[e] for every expert, zeros past the last range."""
    out = rows.new_zeros(rows.shape[0], weights.shape[2])
    begin = 0
    for e, end in enumerate(ends):
        torch.mm(rows[begin:end], weights[e], out=out[begin:end])
        begin = end
    return out


def expert_weight_gradients(rows, grads, ends):
    """rows[e's range]^T @ grads[e's range] in float32."""
    out, begin = [], 0
    for end in ends:
        out.append(rows[begin:end].float().t() @ grads[begin:end].float())
        begin = end
    return torch.stack(out)


def operand_values(operands, ends):
    """What the NVFP4 operands of packed rows stand for: float32, the last expert's end rows."""
    out, begin = [], 0
    for e, end in enumerate(ends):
        if end > begin:
            out.append(api.nvfp4_dequantize(operands["row_codes"][begin:end],
                                            operands["row_scales"][begin:end],
                                            operands["row_gscale"][e]))
        begin = end
    return torch.cat(out)


class MoELayer:
    def __init__(self, hidden, width, experts, topk, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        draw = lambda *s: torch.randn(*s, generator=g, device=device)
        self.topk, self.experts = topk, experts
        self.norm = (1 + 0.1 * draw(hidden)).to(torch.bfloat16)
        self.router = draw(hidden, experts) * hidden ** -0.5
        self.w1 = (draw(experts, hidden, 2 * width) * hidden ** -0.5).to(torch.bfloat16)
        self.w2 = (draw(experts, width, hidden) * width ** -0.5).to(torch.bfloat16)

    def forward(self, x):
        n = api.nvfp4_rmsnorm_checkpoint(x, self.norm)
        logits = n["y"].float() @ self.router
        ids, weights = api.nvfp4_moe_router(logits, self.topk)
        plan = api.nvfp4_moe_plan(ids, self.experts)
        packed, amax = api.nvfp4_moe_dispatch(n["y"], plan)
        operands = api.nvfp4_quantize_grouped(packed, plan["offsets"], columnwise=False,
                                              amax_row=amax)
        ends = plan["offsets"].tolist()
        act = api.nvfp4_swiglu_checkpoint(expert_products(packed, self.w1, ends),
                                          offsets=plan["offsets"])
        act_operands = api.nvfp4_quantize_grouped(act["y"], plan["offsets"], columnwise=False,
                                                  amax_row=act["amax"])
        y = expert_products(act["y"], self.w2, ends)
        out = x + api.nvfp4_moe_combine(y, weights, plan)
        # what the backward pass needs; the norm's and the SwiGLU's inputs in 8 bits
        self.saved = dict(norm={k: n[k] for k in ("codes", "scales", "rstd")}, n=n["y"],
                          logits=logits, ids=ids.long(), weights=weights, plan=plan, ends=ends, packed=packed, y=y,
                          glu={k: act[k] for k in ("codes", "scales")}, act=act["y"],
                          operands={"packed": operands, "act": act_operands})
        return out, operands

    def backward(self, grad_out):
        s = self.saved
        plan, ends = s["plan"], s["ends"]
        grad_y, grad_w = api.nvfp4_moe_combine_backward(grad_out, s["y"], s["weights"], plan)
        grads = {"w2": expert_weight_gradients(s["act"], grad_y, ends)}
        grad_act = expert_products(grad_y, self.w2.transpose(1, 2), ends)
        grad_h = api.nvfp4_swiglu_checkpoint_backward(grad_act, **s["glu"],
                                                      offsets=plan["offsets"])
        grads["w1"] = expert_weight_gradients(s["packed"], grad_h, ends)
        grad_packed = expert_products(grad_h, self.w1.transpose(1, 2), ends)
        grad_n = api.nvfp4_moe_dispatch_backward(grad_packed, plan)
        grad_logits = api.nvfp4_moe_router_backward(grad_w, s["logits"], s["ids"].int())
        grads["router"] = s["n"].float().t() @ grad_logits
        grad_n = (grad_n.float() + grad_logits @ self.router.t()).to(torch.bfloat16)
        grads["x"], grads["norm"] = api.nvfp4_rmsnorm_checkpoint_backward(
            grad_n, **s["norm"], weight=self.norm, grad_residual=grad_out)
        return grads


def main():
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 512), ("hidden", 1024), ("width", 512), ("experts", 8),
                        ("topk", 2)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    device = torch.device("cuda")
    layer = MoELayer(a.hidden, a.width, a.experts, a.topk, device)
    x = torch.randn(a.tokens, a.hidden, device=device).to(torch.bfloat16)
    out, operands = layer.forward(x)
    grads = layer.backward(torch.ones_like(out))
    print("out", tuple(out.shape), "operands", {k: tuple(v.shape) for k, v in operands.items()})
    for k, q in layer.saved["operands"].items():
        rows = layer.saved[k][:layer.saved["ends"][-1]].float()
        off = (operand_values(q, layer.saved["ends"]) - rows).norm() / rows.norm()
        print("operands of %-6s off by %.3f" % (k, off.item()))
    for k, v in grads.items():
        print("grad %-6s %s, norm %.4g" % (k, tuple(v.shape), v.float().norm().item()))
    bits = api.nvfp4_get_status()
    print("device status", bits)


if __name__ == "__main__":
    main()
