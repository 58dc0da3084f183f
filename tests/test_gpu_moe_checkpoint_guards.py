"""The routing and checkpoint operators write their outputs and nothing else: every output lies in a
larger buffer whose bytes on both sides must stay as they were, at ragged sizes."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import api, workloads

pytestmark = pytest.mark.gpu

PAD = 4096  # bytes on each side; keeps every alignment


class Guarded:
    def __init__(self):
        self.held = []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((PAD + n + PAD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.held.append((buf, n))
        return buf[PAD:PAD + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.held:
            assert bool((buf[:PAD] == 0xA5).all()) and bool((buf[PAD + n:] == 0xA5).all())


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


@pytest.mark.parametrize("T,K,E,H,drop", [(1, 1, 1, 8, 0.0), (5, 3, 4, 24, 0.4), (17, 8, 9, 1032, 0.2),
                                          (129, 2, 256, 264, 0.0), (2001, 3, 5, 72, 0.1)])
def test_routing(T, K, E, H, drop):
    dev = _cuda()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    rng = np.random.default_rng(T)
    ids = np.where(rng.random((T, K)) < drop, -1, rng.integers(0, E, (T, K)))
    ids = torch.tensor(ids, device=dev)
    x, y = (workloads.normal(n, H, 1.0, seed=n).to(dev) for n in (T, T * K))
    g = Guarded()
    plan = api.nvfp4_moe_plan(ids, E, out={"row_of_slot": g((T, K), i32),
                                           "slot_of_row": g((T * K,), i32), "offsets": g((E,), i32)})
    w = torch.rand(T, K, device=dev)
    api.nvfp4_moe_dispatch(x, plan, out=g((T * K, H), bf), amax=g((E,), f32))
    api.nvfp4_moe_dispatch_backward(y, plan, out=g((T, H), bf))
    api.nvfp4_moe_combine(y, w, plan, out=g((T, H), bf))
    api.nvfp4_moe_combine_backward(x, y, w, plan, grad_y=g((T * K, H), bf),
                                   grad_weights=g((T, K), f32))
    g.check()


@pytest.mark.parametrize("M,N", [(1, 32), (3, 96), (70, 544), (9, 2080), (5, 8192), (3, 8224), (2, 16416)])
def test_checkpoints(M, N):
    dev = _cuda()
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x, dy = (workloads.normal(M, N, s, seed=M + N).to(dev) for s in (1.0, 0.1))
    h = workloads.normal(M, 2 * N, 1.0, seed=N).to(dev)
    w = torch.ones(N, dtype=bf, device=dev)
    ends = torch.tensor([M // 3, M // 3, M - M // 4], dtype=torch.int32, device=dev)
    g = Guarded()
    a = api.nvfp4_rmsnorm_checkpoint(x, w, out={
        "y": g((M, N), bf), "codes": g((M, N), u8), "scales": g((M, N // 32), u8),
        "rstd": g((M,), f32), "amax": g((1,), f32)})
    api.nvfp4_rmsnorm_checkpoint_backward(
        dy, a["codes"], a["scales"], a["rstd"], w, grad_residual=x, grad_x=g((M, N), bf),
        grad_weight=g((N,), f32), workspace=g((api.nvfp4_rmsnorm_checkpoint_workspace(M, N),), u8))
    b = api.nvfp4_swiglu_checkpoint(h, offsets=ends, out={
        "y": g((M, N), bf), "codes": g((M, 2 * N), u8), "scales": g((M, N // 16), u8),
        "amax": g((3,), f32)})
    api.nvfp4_swiglu_checkpoint_backward(dy, b["codes"], b["scales"], offsets=ends,
                                         out=g((M, 2 * N), bf))
    g.check()
