"""The routing and checkpoint operators together, as examples/moe_layer.py runs them, against the
same layer differentiated by torch in float32."""
import importlib.util
import os

import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import api

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "moe_layer.py")


def _example():
    spec = importlib.util.spec_from_file_location("moe_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T,H,F,E,K", [(300, 256, 96, 8, 2), (1, 128, 64, 4, 4), (77, 512, 160, 5, 3)])
def test_layer_against_autograd(T, H, F, E, K):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda")
    layer = _example().MoELayer(H, F, E, K, dev, seed=T)
    g = torch.Generator(device=dev).manual_seed(5)
    x = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    grad_out = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    out, operands = layer.forward(x)
    grads = layer.backward(grad_out)
    assert api.nvfp4_get_status() == (0, 0)
    assert operands["row_codes"].shape == (T * K, H // 2)

    leaves = {k: v.float().requires_grad_() for k, v in
              dict(x=x, norm=layer.norm, router=layer.router, w1=layer.w1, w2=layer.w2).items()}
    v = leaves["x"]
    n = leaves["norm"] * v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)
    ids = layer.saved["ids"]
    w = torch.softmax((n @ leaves["router"]).gather(1, ids), dim=1)
    total = v
    for k in range(K):
        h = torch.einsum("th,thf->tf", n, leaves["w1"][ids[:, k]])
        act = torch.nn.functional.silu(h[:, :F]) * h[:, F:]
        total = total + w[:, k:k + 1] * torch.einsum("tf,tfh->th", act, leaves["w2"][ids[:, k]])
    total.backward(grad_out.float())

    def off(a, b):
        return float((a.float() - b).norm() / b.norm())
    # BF16 activations and products: a few half steps of 2^-8 each
    assert off(out, total.detach()) < 0.02
    # the kept inputs are off by at most 2^-4 of themselves, about a third of that in the mean
    for k, leaf in leaves.items():
        assert off(grads[k], leaf.grad) < 0.06, (k, off(grads[k], leaf.grad))
