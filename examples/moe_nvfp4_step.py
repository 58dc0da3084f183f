"""Training steps of a mixture-of-experts layer with every expert product in NVFP4:

    out = x + sum_k w_k * expert_k(rmsnorm(x)),   expert(v) = W2 (silu(W1g v) * (W1u v))

Router, routing plan, the products of the forward pass, the products of both backward passes and the
update of the weights run on this package's operators. Rows are quantized with the amax that the
operator before found; the weights with the amax that the AdamW step found, 16 x 16 blocks, so that one
quantization serves the forward products (rowwise) and the input's gradients (columnwise). The weights'
gradients take columnwise operands under the random Hadamard transform, the gradients' operands are
rounded stochastically, and the optimizer keeps its moments in 8 bits.

    python examples/moe_nvfp4_step.py [--tokens 512 --hidden 1024 --width 512 --experts 8 --topk 2 --steps 3]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_block_scaled_quantize_gb300 import api  # noqa: E402

SIGNS = 0x5A3C  # of the Hadamard transform, the same for both operands of a weight gradient


def row(q):
    return q["row_codes"], q["row_scales"], q["row_gscale"]


def col(q):
    return q["col_codes"], q["col_scales"], q["col_gscale"]


class StackedWeights:
    """E matrices [N, K] as BF16 [E, N, K] and their NVFP4 operands."""

    def __init__(self, bf16):
        self.bf16 = bf16
        E, N, K = bf16.shape
        self.ends = torch.arange(1, E + 1, dtype=torch.int32, device=bf16.device) * N

    def quantize(self, amax=None):
        E, N, K = self.bf16.shape
        self.q = api.nvfp4_quantize_grouped(self.bf16.view(E * N, K), self.ends, col_capacity=E * N,
                                            block2d=True, amax_row=amax)

    def forward_operand(self):
        E, N, K = self.bf16.shape
        codes, scales, gscale = row(self.q)
        return codes.view(E, N, K // 2), scales.view(E, N, K // 16), gscale

    def backward_operand(self):
        """The transposed matrices: expert e's columns of the columnwise outputs."""
        E, N, K = self.bf16.shape
        codes, scales, gscale = col(self.q)
        return (codes.view(K, E, N // 2).transpose(0, 1), scales.view(K, E, N // 16).transpose(0, 1), gscale)


class MoELayer:
    def __init__(self, hidden, width, experts, topk, device, seed=0, lr=1e-3, state_bits=8):
        g = torch.Generator(device=device).manual_seed(seed)
        draw = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.topk, self.experts = topk, experts
        # float32 masters of the norm, the router, and each expert's matrices
        self.masters = {"norm": 1 + 0.1 * draw(hidden), "router": draw(experts, hidden) * hidden ** -0.5,
                        "w1": draw(experts, 2 * width, hidden) * hidden ** -0.5,
                        "w2": draw(experts, hidden, width) * width ** -0.5}
        self.grads = {k: torch.zeros_like(v) for k, v in self.masters.items()}
        self.bf16 = {k: v.to(torch.bfloat16) for k, v in self.masters.items()}
        parts = lambda d: list(d["w1"]) + list(d["w2"]) + [d["norm"], d["router"]]  # noqa: E731
        self.optimizer = api.AdamW(parts(self.masters), parts(self.grads), weights=parts(self.bf16), lr=lr,
                                   betas=(0.9, 0.95), weight_decay=[0.1] * (2 * experts) + [0.0, 0.0],
                                   state_bits=state_bits)
        self.w1, self.w2 = StackedWeights(self.bf16["w1"]), StackedWeights(self.bf16["w2"])
        self.w1.quantize()
        self.w2.quantize()
        self.steps = 0

    def _rows(self, x, offsets, amax, **kw):
        return api.nvfp4_quantize_grouped(x, offsets, rht_col=True, sign_mask=SIGNS, amax_row=amax, **kw)

    def forward(self, x):
        n = api.nvfp4_rmsnorm_checkpoint(x, self.bf16["norm"])
        logits = n["y"].float() @ self.masters["router"].t()
        ids, weights = api.nvfp4_moe_router(logits, self.topk)
        plan = api.nvfp4_moe_plan(ids, self.experts)
        offsets = plan["offsets"]
        packed, amax = api.nvfp4_moe_dispatch(n["y"], plan)
        qx = self._rows(packed, offsets, amax)
        h = api.nvfp4_gemm_grouped(*row(qx), *self.w1.forward_operand(), offsets)["out"]
        act = api.nvfp4_swiglu_checkpoint(h, offsets=offsets)
        qa = self._rows(act["y"], offsets, act["amax"])
        y = api.nvfp4_gemm_grouped(*row(qa), *self.w2.forward_operand(), offsets)["out"]
        out = x + api.nvfp4_moe_combine(y, weights, plan)
        # the kept tensors: 8 bits for the norm and the SwiGLU, columnwise NVFP4 for the products
        self.saved = dict(norm={k: n[k] for k in ("codes", "scales", "rstd")}, n=n["y"], logits=logits,
                          ids=ids, weights=weights, plan=plan, y=y, qx=qx, qa=qa,
                          glu={k: act[k] for k in ("codes", "scales")})
        return out

    def backward(self, grad_out):
        """The gradient of x; those of the masters go to self.grads."""
        s, seed = self.saved, 2 * self.steps
        plan, offsets = s["plan"], s["plan"]["offsets"]
        grad_y, grad_w = api.nvfp4_moe_combine_backward(grad_out, s["y"], s["weights"], plan)
        qy = self._rows(grad_y, offsets, None, round_row="sr", round_col="sr", seed=seed)
        api.nvfp4_gemm_grouped_wgrad(*col(qy), *col(s["qa"]), offsets, out=self.grads["w2"])
        grad_a = api.nvfp4_gemm_grouped(*row(qy), *self.w2.backward_operand(), offsets)["out"]
        grad_h = api.nvfp4_swiglu_checkpoint_backward(grad_a, **s["glu"], offsets=offsets)
        qh = self._rows(grad_h, offsets, None, round_row="sr", round_col="sr", seed=seed + 1)
        api.nvfp4_gemm_grouped_wgrad(*col(qh), *col(s["qx"]), offsets, out=self.grads["w1"])
        grad_packed = api.nvfp4_gemm_grouped(*row(qh), *self.w1.backward_operand(), offsets)["out"]
        grad_n = api.nvfp4_moe_dispatch_backward(grad_packed, plan)
        grad_logits = api.nvfp4_moe_router_backward(grad_w, s["logits"], s["ids"])
        torch.mm(grad_logits.t(), s["n"].float(), out=self.grads["router"])
        grad_n = (grad_n.float() + grad_logits @ self.masters["router"]).to(torch.bfloat16)
        grad_x, _ = api.nvfp4_rmsnorm_checkpoint_backward(grad_n, **s["norm"], weight=self.bf16["norm"],
                                                          grad_residual=grad_out, grad_weight=self.grads["norm"])
        return grad_x

    def step(self):
        """AdamW on every master; the weights are quantized anew with the amax that it found."""
        self.steps += 1
        amax = self.optimizer.step(self.steps, seed=self.steps)
        E = self.experts
        self.w1.quantize(amax[:E])
        self.w2.quantize(amax[E:2 * E])
        return amax


def main():
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 512), ("hidden", 1024), ("width", 512), ("experts", 8), ("topk", 2),
                        ("steps", 3)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    device = torch.device("cuda")
    layer = MoELayer(a.hidden, a.width, a.experts, a.topk, device)
    x = torch.randn(a.tokens, a.hidden, device=device).to(torch.bfloat16)
    target = torch.randn(a.tokens, a.hidden, device=device)
    for i in range(a.steps):
        out = layer.forward(x)
        error = out.float() - target
        layer.backward((error / error.numel()).to(torch.bfloat16))
        layer.step()
        print("step %d, mean square %.5f, norm of w1's gradient %.4g" % (
            i + 1, error.square().mean().item(), layer.grads["w1"].norm().item()))
    print("device status", api.nvfp4_get_status())


if __name__ == "__main__":
    main()
