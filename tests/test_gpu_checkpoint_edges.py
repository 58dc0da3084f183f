"""The checkpoint operators at their edges: offsets that are not what the header asks, and buffers
with no more alignment than it asks for."""
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


def _at(t, nbytes):
    """A copy of `t` that starts `nbytes` past a 512-byte boundary."""
    size = t.element_size()
    buf = torch.empty(t.numel() + nbytes // size, dtype=t.dtype, device=t.device)
    out = buf[nbytes // size:].view(t.shape)
    assert out.data_ptr() % 512 == nbytes
    return out.copy_(t)


def test_buffers_with_the_least_alignment_and_with_less():
    dev = _cuda()
    M, N = 5, 1056
    h = workloads.normal(M, 2 * N, 1.0, seed=1).to(dev)
    x, dy = (workloads.normal(M, N, 1.0, seed=s).to(dev) for s in (2, 3))
    w = torch.linspace(0.5, 1.5, N, device=dev).to(torch.bfloat16)
    offs = torch.tensor([1, 4], dtype=torch.int32, device=dev)
    aligned = dict(y=32, codes=16, scales=1, rstd=4, amax=4)
    like = lambda d: {k: _at(v, aligned[k]) for k, v in d.items()}

    a = api.nvfp4_swiglu_checkpoint(h, offsets=offs)
    b = api.nvfp4_swiglu_checkpoint(_at(h, 32), offsets=_at(offs, 4), out=like(a))
    n = api.nvfp4_rmsnorm_checkpoint(x, w)
    m = api.nvfp4_rmsnorm_checkpoint(_at(x, 32), _at(w, 32), out=like(n))
    for p, q in ((a, b), (n, m)):
        for k in p:
            assert q[k].data_ptr() % 512 == aligned[k] and torch.equal(p[k], q[k]), k
    grad = api.nvfp4_swiglu_checkpoint_backward(dy, a["codes"], a["scales"], offsets=offs)
    assert torch.equal(grad, api.nvfp4_swiglu_checkpoint_backward(
        _at(dy, 32), b["codes"], b["scales"], offsets=_at(offs, 4), out=_at(grad, 32)))
    kept = [n[k] for k in ("codes", "scales", "rstd")]
    gx, gw = api.nvfp4_rmsnorm_checkpoint_backward(dy, *kept, w, grad_residual=x)
    kept = [m[k] for k in ("codes", "scales", "rstd")]
    ws = torch.empty(api.nvfp4_rmsnorm_checkpoint_workspace(M, N), dtype=torch.uint8, device=dev)
    got = api.nvfp4_rmsnorm_checkpoint_backward(
        _at(dy, 32), *kept, _at(w, 32), grad_residual=_at(x, 32), grad_x=_at(gx, 32),
        grad_weight=_at(gw, 16), workspace=_at(ws, 16))
    assert torch.equal(got[0], gx) and torch.equal(got[1], gw)

    # half of it is refused before anything is launched
    for call in (lambda: api.nvfp4_swiglu_checkpoint(_at(h, 16)),
                 lambda: api.nvfp4_swiglu_checkpoint(h, offsets=offs,
                                                     out=dict(a, y=_at(a["y"], 16))),
                 lambda: api.nvfp4_rmsnorm_checkpoint(x, _at(w, 16)),
                 lambda: api.nvfp4_rmsnorm_checkpoint_backward(_at(dy, 16), *kept, w)):
        with pytest.raises(_lib.NVFP4Error) as e:
            call()
        assert "NVFP4_ERR_ALIGN" in str(e.value)
    assert api.nvfp4_get_status() == (0, 0)
