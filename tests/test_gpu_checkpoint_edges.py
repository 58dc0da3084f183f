"""The checkpoint operators at their edges: offsets that are not what the header asks, buffers
with no more alignment than it asks for, and gates far from zero in the gradient."""
import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import _lib, api, workloads

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24   # half a binary32 step
UBF = 2.0 ** -8    # half a BF16 step
TINY = 2.0 ** -133


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


def test_gradient_at_gates_far_from_zero():
    dev = _cuda()
    # all of them E4M3 values times a power of two; sigmoid(-88), (-96) and (-104) are binary32
    # subnormals or below, and from 17 up sigmoid rounds to 1
    gates = [0.0, -0.0, 1.25, -1.25, -1.375, 5.5, -5.5, 16.0, 18.0, -18.0, 80.0, -80.0, 88.0, -88.0,
             -96.0, -104.0, 112.0, 1.25 * 2.0 ** 13, -1.25 * 2.0 ** 13, 1.75 * 2.0 ** 127,
             -1.75 * 2.0 ** 127, 2.0 ** -126, -2.0 ** -126]
    F = 32 * len(gates)
    pairs = [(1.0, 1.0), (-0.75, 3.0), (2.0 ** -10, 2.0 ** 100), (1.0, 2.0 ** -100)]  # dy, u
    M = len(pairs)
    h = torch.zeros(M, 2 * F, dtype=torch.bfloat16)
    h[:, :F] = torch.tensor(gates).repeat_interleave(32).to(torch.bfloat16)
    dy = torch.zeros(M, F, dtype=torch.bfloat16)
    for i, (d, u) in enumerate(pairs):
        h[i, F:], dy[i] = u, d
    kept = api.nvfp4_swiglu_checkpoint(h.to(dev))
    back = api.nvfp4_mx_dequantize(kept["codes"], kept["scales"], "e4m3").cpu().double()
    assert torch.equal(back, h.double())
    got = api.nvfp4_swiglu_checkpoint_backward(dy.to(dev), kept["codes"], kept["scales"])
    g, u = h.double().split(F, 1)
    d, s = dy.double(), torch.sigmoid(g)
    slope = s * (1 + g * (1 - s))
    ref = torch.cat([d * u * slope, d * g * s], 1)
    # t = exp(-|g|) is off by 10 + 1.173 |g| steps of 2^-23 of itself and, where it is subnormal, by
    # 2^-149; past 200 it is 0 in both, and for g > 17 so is 1 - s
    near = g.abs().clamp(max=200.0)
    n = torch.where(g > 0, near.clamp(max=17.0), near)
    rel = (10 + 1.173 * n) * 2 * U32 + 8 * U32
    under = 2.0 ** -149 * (2 + near)
    off = torch.cat([(d * u).abs() * (s * (1 + n) * rel + under) + 2.0 ** -149,
                     (d * g * s).abs() * rel + d.abs() * under], 1)
    diff = (got.cpu().double() - ref).abs()
    lim = UBF * (ref.abs() + off) + off + TINY
    assert bool((diff <= lim).all()), (diff - lim).max()
