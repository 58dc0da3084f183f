"""examples/moe_nvfp4_step.py: router, experts' products, their gradients and AdamW together."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import api

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "moe_nvfp4_step.py")


def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("moe_nvfp4_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T,H,F,E,K", [(300, 256, 96, 8, 2), (1, 128, 64, 4, 4), (2000, 512, 160, 5, 3)])
def test_gradients_against_autograd(T, H, F, E, K):
    dev = torch.device("cuda")
    layer = example().MoELayer(H, F, E, K, dev, seed=T)
    g = torch.Generator(device=dev).manual_seed(5)
    x = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    grad_out = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    out = layer.forward(x)
    grad_x = layer.backward(grad_out)
    assert api.nvfp4_get_status() == (0, 0)
    leaves = {k: v.float().clone().requires_grad_() for k, v in dict(
        x=x, norm=layer.bf16["norm"], router=layer.masters["router"], w1=layer.bf16["w1"],
        w2=layer.bf16["w2"]).items()}
    v = leaves["x"]
    n = leaves["norm"] * v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)
    ids = layer.saved["ids"].long()
    w = torch.softmax((n @ leaves["router"].t()).gather(1, ids), dim=1)
    total, spread = v, 0.0
    for k in range(K):
        h = torch.einsum("th,tfh->tf", n, leaves["w1"][ids[:, k]])
        act = torch.nn.functional.silu(h[:, :F]) * h[:, F:]
        y = torch.einsum("tf,thf->th", act, leaves["w2"][ids[:, k]])
        total = total + w[:, k:k + 1] * y
        spread = spread + ((w[:, k] * y.norm(dim=1) * grad_out.float().norm(dim=1) * n.norm(dim=1)) ** 2).sum()
    total.backward(grad_out.float())

    def off(a, b):
        return float((a.float() - b).norm() / b.norm())
    # An E2M1 operand is off by 0.08 to 0.12 of itself in the mean (steps of 1/2 to 2 below 6, half of
    # one at most; stochastic rounding twice that squared), a product of two by 1.5 times that, and a
    # gradient has two or three products and the gate between them behind it.
    assert off(out - x, (total - leaves["x"]).detach()) < 0.3
    for k, got in dict(layer.grads, x=grad_x).items():
        if k != "router":
            assert off(got, leaves[k].grad) < 0.5, (k, off(got, leaves[k].grad))
    # The router's is w (g - sum w g) n with g = <dout, y>. An error of 0.3 of y in any direction moves g
    # by 0.3 |dout| |y| / sqrt(H) (one standard deviation), whatever g itself is; the difference of two
    # such by sqrt(2) times that. Three standard deviations of a few values, less of many.
    error = (layer.grads["router"] - leaves["router"].grad).norm()
    assert error < 3 * 0.3 * 2 ** 0.5 * (spread / H).sqrt()


def test_a_step_leaves_operands_of_the_new_weights():
    m = example()
    dev = torch.device("cuda")
    layer = m.MoELayer(256, 96, 6, 2, dev, seed=3)
    x = torch.randn(90, 256, device=dev).to(torch.bfloat16)
    before = {k: v.clone() for k, v in layer.masters.items()}
    for _ in range(2):
        out = layer.forward(x)
        layer.backward((out.float() * 1e-3).to(torch.bfloat16))
        amax = layer.step()
        E = layer.experts
        for i, (name, w) in enumerate((("w1", layer.w1), ("w2", layer.w2))):
            assert torch.equal(w.bf16, layer.masters[name].to(torch.bfloat16))
            assert torch.equal(amax[i * E:(i + 1) * E], w.bf16.float().abs().amax((1, 2)))
            held = {k: v.clone() for k, v in w.q.items()}
            w.quantize()  # with an amax pass of its own
            for k, v in w.q.items():
                assert torch.equal(v, held[k]), (name, k)
        for k, v in layer.masters.items():
            # the first steps move every element with a gradient by about lr, and decay by lr * 0.1
            assert torch.isfinite(v).all() and 0 < (v - before[k]).abs().max() < 3e-3, k
    assert api.nvfp4_get_status() == (0, 0)


def test_a_captured_step_repeats():
    """Forward, backward and update captured once and replayed give what eager calls give."""
    m = example()
    dev = torch.device("cuda")
    torch.manual_seed(11)
    x = torch.randn(130, 256, device=dev).to(torch.bfloat16)
    grad = torch.randn(130, 256, device=dev).to(torch.bfloat16)
    eager, held = (m.MoELayer(256, 64, 4, 2, dev, seed=8) for _ in range(2))
    want = [(eager.forward(x).clone(), eager.backward(grad).clone()) for _ in range(2)][-1]
    held.forward(x)
    held.backward(grad)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = held.forward(x), held.backward(grad)
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for k, v in eager.grads.items():
        assert torch.equal(v, held.grads[k]), k


def test_the_example_runs():
    example()
    r = subprocess.run([sys.executable, PATH, "--tokens", "40", "--hidden", "128", "--width", "64",
                        "--experts", "4"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "step 3" in r.stdout and "device status (0, 0)" in r.stdout
