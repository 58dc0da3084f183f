"""Token routing at its edges."""
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
