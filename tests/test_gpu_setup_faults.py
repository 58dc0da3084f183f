"""Set-up failures of the routing and checkpoint kernels, injected on the host."""
import os
import subprocess
import sys

import pytest

from nvfp4_block_scaled_quantize_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# a fresh process: its first calls are the ones that set the kernels up
FIRST_CALLS = """
import sys
import torch
from nvfp4_block_scaled_quantize_gb300 import _lib, api
CAPTURE = sys.argv[1] == "capture"
dev = torch.device("cuda")
x = torch.randn(64, 64, device=dev).to(torch.bfloat16)
w = torch.ones(64, dtype=torch.bfloat16, device=dev)
ids = torch.zeros(64, 2, dtype=torch.int32, device=dev)

def plan():
    return api.nvfp4_moe_plan(ids, 4)["offsets"].tolist()

def norm():
    return api.nvfp4_rmsnorm_checkpoint(x, w)["amax"].item() > 0

def quantizers():
    a = api.nvfp4_quantize(x, columnwise=True)
    b = api.nvfp4_quantize(x, columnwise=True, fused_amax=True)
    assert all(torch.equal(a[k], b[k]) for k in a)
    api.nvfp4_mx_quantize(x, "e4m3")
    assert api.nvfp4_get_status() == (0, 0)

for _ in range(0 if CAPTURE else 2):
    api.nvfp4_debug_setup_fault(1)
    for call in (plan, norm):
        try:
            call()
        except _lib.NVFP4Error as e:
            assert "NVFP4_ERR_CUDA" in str(e)
        else:
            raise AssertionError("a call whose set-up failed returned")
    quantizers()
api.nvfp4_debug_setup_fault(0)
if CAPTURE:
    quantizers()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = api.nvfp4_moe_plan(ids, 4)["offsets"]
    graph.replay()
    assert held.tolist() == [128] * 4
assert plan() == [128] * 4 and norm()
quantizers()
print("done")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["fault", "capture"])
def test_first_calls(how):
    """The quantizers run where the routing kernels cannot be set up, whose calls report it and run
    once they can; a routing call may be captured after any first call."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS, how], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stdout + r.stderr


def test_hook_argument_checks():
    from nvfp4_block_scaled_quantize_gb300 import build
    build.build()
    L = _lib.load()
    assert L.nvfp4_debug_setup_fault(-1) == 1 and L.nvfp4_debug_setup_fault(3) == 1
    assert L.nvfp4_debug_setup_fault(0) == 0
