"""What an MoE layer hands to block-scaled GEMMs: packed rows and SwiGLU outputs quantized with the
amax that their operators give, alone and in examples/moe_layer.py."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import api, workloads

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "moe_layer.py")


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


@pytest.mark.parametrize("M,F,ends", [(70, 96, [20, 20, 63]), (300, 1056, [1, 299, 300, 300]),
                                      (33, 64, [33])])
def test_amax_is_what_the_quantizers_take(M, F, ends):
    """y quantized with the operator's own amax equals y quantized from its values alone."""
    dev = _cuda()
    h = workloads.normal_with_outliers(M, 2 * F, seed=M, fraction=0.01, gain=40.0).to(dev)
    offs = torch.tensor(ends, dtype=torch.int32, device=dev)
    a = api.nvfp4_swiglu_checkpoint(h, offsets=offs)
    q = [api.nvfp4_quantize_grouped(a["y"], offs, columnwise=False, amax_row=amax)
         for amax in (a["amax"], None)]
    for k in q[0]:
        n = len(ends) if k == "row_gscale" else ends[-1]
        assert torch.equal(q[0][k][:n], q[1][k][:n]), k
    x = h[:, :F].contiguous()
    b = api.nvfp4_rmsnorm_checkpoint(x, torch.ones(F, dtype=torch.bfloat16, device=dev))
    q = [api.nvfp4_quantize(b["y"], columnwise=False, amax_row=amax) for amax in (b["amax"], None)]
    for k in q[0]:
        assert torch.equal(q[0][k], q[1][k]), k
    assert api.nvfp4_get_status() == (0, 0)


@pytest.mark.parametrize("T,H,F,E,K", [(77, 512, 160, 5, 3), (1, 128, 64, 8, 2),
                                       (300, 256, 96, 8, 2)])
def test_operands_of_the_layer(T, H, F, E, K):
    dev = _cuda()
    spec = importlib.util.spec_from_file_location("moe_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    layer = m.MoELayer(H, F, E, K, dev, seed=T)
    g = torch.Generator(device=dev).manual_seed(5)
    layer.forward(torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16))
    s = layer.saved
    for k, q in s["operands"].items():
        rows = s[k][:s["ends"][-1]].double()
        got = m.operand_values(q, s["ends"]).double()
        # E2M1 in blocks of 16: the scale (6 for the largest magnitude) is off by at most half an
        # E4M3 step, 2^-4 of itself, and the widest step is 2, from 4 to 6 of it. Below E4M3's normal
        # range half a step of the scale is 2^-10 of amax / 2688: 6 of those are below 2^-18 amax.
        block = rows.abs().view(rows.shape[0], -1, 16).amax(2).repeat_interleave(16, 1)
        lim = block * (1 / 6 + 2.0 ** -4) * (1 + 2.0 ** -4) + rows.abs().max() * 2.0 ** -16
        assert bool(((got - rows).abs() <= lim).all()), k
    assert api.nvfp4_get_status() == (0, 0)


def test_the_example_runs():
    _cuda()
    r = subprocess.run([sys.executable, PATH, "--tokens", "40", "--hidden", "128", "--width", "64",
                        "--experts", "4"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "operands of act" in r.stdout and "device status (0, 0)" in r.stdout
