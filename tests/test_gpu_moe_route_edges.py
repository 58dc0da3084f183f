"""Token routing at its edges."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import _lib, api

pytestmark = pytest.mark.gpu


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


@pytest.mark.parametrize("experts", [257, 2**32 + 9, -2**32 + 9, 0, -1])
def test_a_number_of_experts_that_does_not_fit_is_refused(experts):
    dev = _cuda()
    ids = torch.zeros(4, 2, dtype=torch.int32, device=dev)
    before = torch.cuda.max_memory_allocated(dev)
    with pytest.raises(_lib.NVFP4Error):
        api.nvfp4_moe_plan(ids, experts)
    assert torch.cuda.max_memory_allocated(dev) - before < 2**20  # nothing of that size is made


# one CTA (no cluster), a slot more, runs that are sorted before they are written and not, more
# slots than 8 CTAs sort in shared memory (212992)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["int32", "int64"])
@pytest.mark.parametrize("T,K,E,drop", [(1024, 1, 9, 0.0), (1025, 1, 9, 0.1), (4097, 1, 3, 0.02),
                                        (5003, 6, 256, 0.06), (26000, 8, 64, 0.01),
                                        (30000, 8, 20, 0.01)])
def test_plan_where_the_large_cluster_is_rejected(T, K, E, drop, dtype):
    dev = _cuda()
    rng = np.random.default_rng(T)
    ids = np.where(rng.random((T, K)) < drop, -1, rng.integers(0, E, (T, K)))
    on_device = torch.tensor(ids, dtype=dtype, device=dev)
    usual = api.nvfp4_moe_plan(on_device, E)
    api.nvfp4_debug_setup_fault(2)
    try:
        plan = api.nvfp4_moe_plan(on_device, E)
    finally:
        api.nvfp4_debug_setup_fault(0)
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    live = int((flat >= 0).sum())
    rows = np.full(flat.size, -1)
    rows[order[:live]] = np.arange(live)
    slots = np.where(np.arange(flat.size) < live, order, -1)
    ends = np.cumsum(np.bincount(flat[flat >= 0], minlength=E))
    for got in (plan, usual):
        assert np.array_equal(got["row_of_slot"].cpu().numpy().reshape(-1), rows)
        assert np.array_equal(got["slot_of_row"].cpu().numpy(), slots)
        assert np.array_equal(got["offsets"].cpu().numpy(), ends)
    # nothing of the rejection is left behind
    assert bool(torch.isfinite((on_device.float() * 2).sum()))
    assert api.nvfp4_get_status() == (0, 0)
