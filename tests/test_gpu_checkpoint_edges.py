"""The checkpoint operators at their edges: offsets that are not what the header asks."""
import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import _lib, api, workloads

pytestmark = pytest.mark.gpu


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


# (ends, flagged) for 8 rows: increasing from below zero, out of order, past the rows, and what is
# allowed: empty experts at either end, fewer rows than the tensor has
ENDS = [([-1, 2, 8], True), ([-3, 4, 8], True), ([-2, -1, 3], True), ([3, 2, 8], True),
        ([2, 9, 8], True), ([2, 4, 9], True), ([2, 4, -1], True), ([-1], True), ([9], True),
        ([0, 0, 8], False), ([8, 8, 8], False), ([0, 0, 0], False), ([2, 2, 5], False), ([8], False)]


@pytest.mark.parametrize("ends,flagged", ENDS, ids=lambda v: str(v).replace(" ", ""))
def test_offsets_are_checked_in_both_directions(ends, flagged):
    dev = _cuda()
    h = workloads.normal(8, 64, 1.0, seed=1).to(dev)
    offs = torch.tensor(ends, dtype=torch.int32, device=dev)
    want = (6, _lib.DEVICE_BAD_OFFSETS) if flagged else (0, 0)
    api.nvfp4_get_status()
    kept = api.nvfp4_swiglu_checkpoint(h, offsets=offs)
    assert api.nvfp4_get_status() == want
    grad = api.nvfp4_swiglu_checkpoint_backward(kept["y"], kept["codes"], kept["scales"],
                                                offsets=offs)
    assert api.nvfp4_get_status() == want
    # rows past the last end are zeros either way, and nothing outside the tensor counts
    live = min(max(ends[-1], 0), 8)
    for t in (kept["y"], grad):
        assert bool((t[live:] == 0).all()) and bool(t.isfinite().all())
