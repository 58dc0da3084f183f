"""SwiGLU and RMSNorm with their inputs kept in 8 bits, and the backward passes from them, against
plain implementations in 64 bits. The kept codes and scales equal the definition's; a BF16 output
may be off by half a BF16 step of itself plus the error of its binary32 arithmetic."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import _lib, api, workloads

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
UBF = 2.0 ** -8
TINY = 2.0 ** -133


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


# every non-negative E4M3 value, by code
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                 for c in range(127)])


def _nearest(v):
    """The codes of the nearest E4M3 values of |v| <= 448, ties to the even code."""
    a = np.abs(v)
    i = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo, hi = a - E4M3[i - 1], E4M3[i] - a
    code = np.where((lo < hi) | ((lo == hi) & ((i - 1) % 2 == 0)), i - 1, i)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def _keep_ref(x):
    """codes, scale bytes of x (a 2-D BF16 tensor) by the definition."""
    v = x.double().numpy()
    R, C = v.shape
    b = v.reshape(R, C // 32, 32)
    fine = np.isfinite(b)
    top = np.where(fine, np.abs(b), 0).max(2)
    e = np.full(top.shape, -127)
    while True:
        low = top > 448 * 2.0 ** e
        if not low.any():
            break
        e[low] += 1
    # a kept finite value is a finite binary32: what would round to 2^128 is kept one step below
    b = np.where(fine & (np.abs(b) >= 1.9375 * 2.0 ** 127), np.copysign(1.875 * 2.0 ** 127, b), b)
    codes = _nearest(np.where(fine, b, 0) / 2.0 ** e[:, :, None])
    codes[~fine] = 0x7F
    return codes.reshape(R, C), (e + 127).astype(np.uint8)


def _kept(codes, scales):
    """The values of codes and scale bytes in 64 bits."""
    c = codes.cpu().numpy()
    v = np.where((c & 127) == 127, np.nan, E4M3[np.minimum(c & 127, 126)]) * np.where(c & 128, -1, 1)
    return torch.tensor(v * np.repeat(2.0 ** (scales.cpu().numpy().astype(np.float64) - 127), 32, 1))


def _check_kept(out, x):
    codes, scales = _keep_ref(x)
    got = out["codes"].cpu().numpy()
    nan = (codes & 127) == 127
    assert np.array_equal(out["scales"].cpu().numpy(), scales)
    assert np.array_equal(got & np.where(nan, 127, 255), codes)
    # the layout is the MX one
    back = api.nvfp4_mx_dequantize(out["codes"], out["scales"], "e4m3").cpu().double()
    assert torch.equal(back.nan_to_num(nan=7.0), _kept(out["codes"], out["scales"]).nan_to_num(nan=7.0))


def _near(got, ref, off):
    d = (got.cpu().double() - ref).abs()
    lim = UBF * (ref.abs() + off) + off + TINY
    assert bool((d <= lim).all()), float((d - lim).max())


def _ends(M, E, live, seed):
    rng = np.random.default_rng(seed)
    n = int(M * live)
    return np.sort(np.concatenate([rng.integers(0, n + 1, E - 1), [n]])).astype(np.int32)


def _sigmoid_off(a):
    """What the kernel's sigmoid may be off by, relative: exp of -|a| (2 + 1.173 |a| steps of
    2^-23, by the CUDA guide's bound), the quotient and the products."""
    return (2 + 1.173 * a.abs() + 8) * 2 * U32


# rows, F, experts (0: none), live share: one block, one row, odd widths, more than one CTA
GLU = [(1, 32, 0, 1.0), (1, 4096, 1, 1.0), (5, 96, 3, 0.6), (37, 1056, 7, 0.9), (300, 288, 256, 1.0),
       (2100, 352, 64, 0.97), (9, 64, 4, 0.0), (3, 8192, 2, 1.0)]


@pytest.mark.parametrize("M,F,E,live", GLU)
def test_swiglu(M, F, E, live):
    dev = _cuda()
    h = workloads.normal_with_outliers(M, 2 * F, seed=M + F, fraction=0.01, gain=40.0)
    ends = _ends(M, E, live, seed=M) if E else None
    n = int(ends[-1]) if E else M
    h_in = h.clone()
    h_in[n:] = float("nan")  # rows past the last expert's end are not read
    offs = torch.tensor(ends, device=dev) if E else None
    out = api.nvfp4_swiglu_checkpoint(h_in.to(dev), offsets=offs)
    h[n:] = 0
    _check_kept(out, h)
    g, u = h.double().split(F, 1)
    ref = g * torch.sigmoid(g) * u
    _near(out["y"], ref, _sigmoid_off(g) * ref.abs())
    y = out["y"].cpu()
    begin = np.concatenate([[0], ends[:-1]]) if E else [0]
    want = [float(y[b:e].abs().max()) if e > b else 0.0
            for b, e in zip(begin, ends if E else [M])]
    assert out["amax"].tolist() == want
    assert api.nvfp4_get_status() == (0, 0)


def _glu_gradient(dy, g, u):
    s = torch.sigmoid(g)
    slope = s * (1 + g * (1 - s))
    off = _sigmoid_off(g) * s * (1 + g.abs() * (1 - s) + g.abs() * s) * 2
    return (torch.cat([dy * u * slope, dy * g * s], 1),
            torch.cat([(dy * u).abs() * (off + 4 * U32 * slope.abs()),
                       (dy * g * s).abs() * (_sigmoid_off(g) + 4 * U32)], 1))


@pytest.mark.parametrize("M,F,E,live", GLU)
def test_swiglu_backward(M, F, E, live):
    dev = _cuda()
    h = workloads.normal_with_outliers(M, 2 * F, seed=M + F + 1, fraction=0.01, gain=40.0)
    dy = workloads.laplace(M, F, 1e-3, seed=F)
    ends = _ends(M, E, live, seed=M) if E else None
    n = int(ends[-1]) if E else M
    offs = torch.tensor(ends, device=dev) if E else None
    kept = api.nvfp4_swiglu_checkpoint(h.to(dev), offsets=offs)
    dy_in = dy.clone()
    dy_in[n:] = float("nan")
    got = api.nvfp4_swiglu_checkpoint_backward(
        dy_in.to(dev), kept["codes"], kept["scales"], offsets=offs,
        out=torch.full((M, 2 * F), float("nan"), dtype=torch.bfloat16, device=dev))
    dy[n:] = 0
    g, u = _kept(kept["codes"], kept["scales"]).split(F, 1)
    ref, off = _glu_gradient(dy.double(), g, u)
    _near(got, ref, off)
    assert bool((got[n:] == 0).all())


def test_swiglu_gradient_against_differences():
    dev = _cuda()
    M, F, step = 6, 64, 2.0 ** -12
    h, dy = workloads.normal(M, 2 * F, 2.0, seed=1), workloads.normal(M, F, 1.0, seed=2)
    kept = api.nvfp4_swiglu_checkpoint(h.to(dev))
    got = api.nvfp4_swiglu_checkpoint_backward(dy.to(dev), kept["codes"], kept["scales"]).cpu().double()
    at = _kept(kept["codes"], kept["scales"])

    def loss(v):
        g, u = v.split(F, 1)
        return float((dy.double() * g * torch.sigmoid(g) * u).sum())
    for seed in range(4):
        d = torch.tensor(np.random.default_rng(seed).normal(size=(M, 2 * F)))
        want = (loss(at + step * d) - loss(at - step * d)) / (2 * step)
        assert abs(float((got * d).sum()) - want) <= 1.01 * UBF * float((got * d).abs().sum()) + 1e-3


def test_bad_offsets_are_flagged():
    dev = _cuda()
    h = workloads.normal(8, 64, 1.0, seed=1).to(dev)
    for ends in ([3, 2, 8], [2, 4, 9], [2, 4, -1]):
        offs = torch.tensor(ends, dtype=torch.int32, device=dev)
        api.nvfp4_get_status()
        kept = api.nvfp4_swiglu_checkpoint(h, offsets=offs)
        assert api.nvfp4_get_status() == (6, _lib.DEVICE_BAD_OFFSETS), ends
    api.nvfp4_swiglu_checkpoint_backward(h[:, :32].contiguous(), kept["codes"], kept["scales"],
                                         offsets=offs)
    assert api.nvfp4_get_status() == (6, _lib.DEVICE_BAD_OFFSETS)


def _special(seed):
    """Rows of awkward blocks: zeros, signed zeros, BF16's whole range, values at the edges
    between two scales, ties of E4M3, subnormals, infinities and NaN."""
    rng = np.random.default_rng(seed)
    rows = [np.zeros(64), np.full(64, -0.0), np.full(64, 448.0), np.full(64, 450.0),
            np.full(64, 3.3e38), rng.normal(size=64) * 2.0 ** -126, np.full(64, 2.0 ** -133),
            np.arange(64) * 2.0 ** -9, (np.arange(64) + 0.5) * 2.0, 448.0 - np.arange(64) * 8,
            np.where(np.arange(64) % 32 == 5, np.inf, rng.normal(size=64)),
            np.where(np.arange(64) % 32 == 31, np.nan, rng.normal(size=64) * 100),
            np.where(np.arange(64) < 32, -np.inf, 1.0)]
    x = torch.tensor(np.array(rows, dtype=np.float32)).to(torch.bfloat16)
    bits = workloads.random_bf16_bits((200, 64), seed).astype(np.int16)
    return torch.cat([x, torch.from_numpy(bits).view(torch.bfloat16)])


def test_kept_values_of_special_blocks():
    dev = _cuda()
    x = _special(1)
    M = x.shape[0]
    out = api.nvfp4_swiglu_checkpoint(x.to(dev))
    _check_kept(out, x)
    out = api.nvfp4_rmsnorm_checkpoint(x.to(dev), torch.ones(64, dtype=torch.bfloat16, device=dev))
    _check_kept(out, x)
    # a kept infinity or NaN reaches its own row's gradient and no other
    kept_x = _kept(out["codes"], out["scales"])
    gx, gw = api.nvfp4_rmsnorm_checkpoint_backward(
        torch.ones(M, 64, dtype=torch.bfloat16, device=dev), out["codes"], out["scales"],
        torch.ones(M, device=dev), torch.ones(64, dtype=torch.bfloat16, device=dev))
    bad = kept_x.isnan().any(1)
    assert 3 <= int(bad.sum()) < M
    assert bool(gx.cpu()[bad].isnan().all(1).all())
    assert not bool(gx.cpu()[~bad].isnan().all(1).any())


def test_large_gates_do_not_overflow():
    dev = _cuda()
    a = np.array([-3e38, -1e4, -100.0, -89.0, -88.0, -87.0, -1.28, -0.0, 0.0, 1.28, 87.0, 89.0, 1e4],
                 dtype=np.float32)
    h = torch.zeros(1, 128, dtype=torch.bfloat16)
    h[0, :len(a)] = torch.tensor(a).to(torch.bfloat16)
    h[0, 64:] = 1.0
    out = api.nvfp4_swiglu_checkpoint(h.to(dev))
    g, u = h.double().split(64, 1)
    ref = g * torch.sigmoid(g) * u
    # the smallest exponentials are binary32 subnormals: absolute steps of 2^-149
    _near(out["y"], ref, _sigmoid_off(g).clamp(max=1.0) * ref.abs() + 2.0 ** -126 * g.abs().clamp(max=200))
    got = api.nvfp4_swiglu_checkpoint_backward(
        torch.ones(1, 64, dtype=torch.bfloat16, device=dev), out["codes"], out["scales"])
    assert bool(got.isfinite().all())


# every width class and its edges, with few and many rows
RMS = [(1, 32), (3, 512), (700, 96), (40, 544), (5, 1024), (33, 1056), (17, 2048), (9, 2080),
       (1300, 4096), (7, 4128), (400, 8192), (3, 8224), (5, 16384), (2, 16416), (160, 32768)]


@pytest.mark.parametrize("M,N", RMS)
@pytest.mark.parametrize("eps,bias", [(1e-6, 0.0), (1e-5, 1.0)])
def test_rmsnorm(M, N, eps, bias):
    dev = _cuda()
    x = workloads.normal_with_outliers(M, N, seed=M + N, fraction=0.01, gain=40.0)
    w = workloads.normal(1, N, 0.3, seed=N)[0] + 1
    out = api.nvfp4_rmsnorm_checkpoint(x.to(dev), w.to(dev), eps=eps, weight_bias=bias)
    _check_kept(out, x)
    v = x.double()
    rstd = 1 / torch.sqrt(v.square().mean(1) + eps)
    # at most 64 squares in a row, then the joins of 5 shuffles and 16 warps
    rel = 96 * U32
    assert bool(((out["rstd"].cpu().double() - rstd).abs() <= rel * rstd).all())
    ref = (w.double() + bias) * v * rstd.unsqueeze(1)
    _near(out["y"], ref, (rel + 4 * U32) * ref.abs())
    assert out["amax"].item() == float(out["y"].abs().max())


@pytest.mark.parametrize("M,N", RMS)
@pytest.mark.parametrize("residual,bias", [(False, 0.0), (True, 1.0)])
def test_rmsnorm_backward(M, N, residual, bias):
    dev = _cuda()
    x = workloads.normal_with_outliers(M, N, seed=M + N + 1, fraction=0.01, gain=40.0)
    w = workloads.normal(1, N, 0.3, seed=N + 1)[0] + 1
    dy = workloads.laplace(M, N, 1e-3, seed=M)
    res = workloads.normal(M, N, 1e-3, seed=M + 1)
    kept = api.nvfp4_rmsnorm_checkpoint(x.to(dev), w.to(dev), weight_bias=bias)
    ws = torch.empty(api.nvfp4_rmsnorm_checkpoint_workspace(M, N), dtype=torch.uint8, device=dev)
    gx, gw = api.nvfp4_rmsnorm_checkpoint_backward(
        dy.to(dev), kept["codes"], kept["scales"], kept["rstd"], w.to(dev), weight_bias=bias,
        grad_residual=res.to(dev) if residual else None, workspace=ws)
    again = api.nvfp4_rmsnorm_checkpoint_backward(
        dy.to(dev), kept["codes"], kept["scales"], kept["rstd"], w.to(dev), weight_bias=bias,
        grad_residual=res.to(dev) if residual else None)
    assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])  # the same sums every time
    r = kept["rstd"].cpu().double().unsqueeze(1)
    xh = _kept(kept["codes"], kept["scales"]) * r
    d = dy.double()
    wg = d * (w.double() + bias)
    mean = (wg * xh).mean(1, keepdim=True)
    ref = r * (wg - xh * mean)
    off = r * (xh.abs() * 96 * U32 * (wg * xh).abs().mean(1, keepdim=True) +
               6 * U32 * (wg.abs() + (xh * mean).abs()))
    if residual:
        ref = ref + res.double()
        off = off + 2 * U32 * ref.abs()
    _near(gx, ref, off)
    ref_w = (d * xh).sum(0)
    off_w = (M + 64) * U32 * (d * xh).abs().sum(0)
    assert bool(((gw.cpu().double() - ref_w).abs() <= off_w).all())


@pytest.mark.parametrize("M,N", [(22000, 512), (9001, 1056), (3100, 4096), (2100, 8192), (1000, 16384)])
def test_rmsnorm_many_tiles(M, N):
    """Rows enough that every CTA goes round its ring of tiles several times: each row equals the
    same row of a call whose CTAs have one tile each."""
    dev = _cuda()
    g = torch.Generator(device=dev).manual_seed(N)
    draw = lambda *s: torch.randn(*s, generator=g, device=dev)
    x, res = draw(M, N).to(torch.bfloat16), (draw(M, N) * 1e-3).to(torch.bfloat16)
    dy, w = (draw(M, N) * 1e-3).to(torch.bfloat16), (1 + 0.3 * draw(N)).to(torch.bfloat16)
    a = api.nvfp4_rmsnorm_checkpoint(x, w)
    for r in (None, res):
        gx, gw = api.nvfp4_rmsnorm_checkpoint_backward(dy, a["codes"], a["scales"], a["rstd"], w,
                                                       grad_residual=r)
        for i in range(0, M, 140):
            s = slice(i, min(i + 140, M))
            if r is None:
                b = api.nvfp4_rmsnorm_checkpoint(x[s], w)
                for k in ("y", "codes", "scales", "rstd"):
                    assert torch.equal(a[k][s], b[k]), (k, i)
            gb, _ = api.nvfp4_rmsnorm_checkpoint_backward(
                dy[s], a["codes"][s], a["scales"][s], a["rstd"][s], w,
                grad_residual=None if r is None else r[s])
            assert torch.equal(gx[s], gb), i
        xh = (a["codes"].view(torch.float8_e4m3fn).double() *
              torch.exp2(a["scales"].double() - 127).repeat_interleave(32, 1) *
              a["rstd"].double().unsqueeze(1))
        prod = dy.double() * xh
        assert bool(((gw.double() - prod.sum(0)).abs() <=
                     (M + 64) * U32 * prod.abs().sum(0)).all())
    assert a["amax"].item() == float(a["y"].abs().max())


def test_rmsnorm_gradient_against_differences():
    dev = _cuda()
    M, N, step, eps = 5, 96, 2.0 ** -12, 1e-5
    x, dy = workloads.normal(M, N, 1.5, seed=1), workloads.normal(M, N, 1.0, seed=2)
    w = workloads.normal(1, N, 0.3, seed=3)[0] + 1
    kept = api.nvfp4_rmsnorm_checkpoint(x.to(dev), w.to(dev), eps=eps)
    at = _kept(kept["codes"], kept["scales"])
    rstd = 1 / torch.sqrt(at.square().mean(1) + eps)  # the norm of the kept values themselves
    gx, gw = api.nvfp4_rmsnorm_checkpoint_backward(dy.to(dev), kept["codes"], kept["scales"],
                                                   rstd.float().to(dev), w.to(dev))
    gx, gw = gx.cpu().double(), gw.cpu().double()

    def loss(v, ww):
        return float((dy.double() * ww * v / torch.sqrt(v.square().mean(1, keepdim=True) + eps)).sum())
    for seed in range(4):
        rng = np.random.default_rng(seed)
        d, dw = torch.tensor(rng.normal(size=(M, N))), torch.tensor(rng.normal(size=N))
        want = (loss(at + step * d, w.double()) - loss(at - step * d, w.double())) / (2 * step)
        # eps counts in the differences and is a 1e-5 part of the gradient's formula
        assert abs(float((gx * d).sum()) - want) <= (1.01 * UBF + 1e-4) * float((gx * d).abs().sum()) + 1e-3
        want = (loss(at, w.double() + step * dw) - loss(at, w.double() - step * dw)) / (2 * step)
        assert abs(float((gw * dw).sum()) - want) <= 1e-5 * float((gw * dw).abs().sum()) + 1e-5


def test_empty():
    dev = _cuda()
    w = torch.ones(64, dtype=torch.bfloat16, device=dev)
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=dev)
    out = api.nvfp4_rmsnorm_checkpoint(x, w)
    assert out["amax"].item() == 0.0 and out["y"].shape == (0, 64)
    gx, gw = api.nvfp4_rmsnorm_checkpoint_backward(x, out["codes"], out["scales"], out["rstd"], w)
    assert gx.shape == (0, 64) and gw.tolist() == [0.0] * 64
    out = api.nvfp4_swiglu_checkpoint(x, offsets=torch.zeros(3, dtype=torch.int32, device=dev))
    assert out["amax"].tolist() == [0.0] * 3
    assert api.nvfp4_swiglu_checkpoint_backward(x[:, :32].contiguous(), out["codes"],
                                                out["scales"]).shape == (0, 64)


def test_offsets_past_32_bits():
    """More than 2^31 elements: blocks of rows equal the same rows computed alone."""
    dev = _cuda()
    M, N = 70000, 32768
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    for a in range(0, M, 5000):
        x[a:a + 5000] = torch.randn(5000, N, generator=g, device=dev)
    w = torch.ones(N, dtype=torch.bfloat16, device=dev)
    last = slice(M - 40, M)
    part = x[last].contiguous()
    big, small = api.nvfp4_rmsnorm_checkpoint(x, w), api.nvfp4_rmsnorm_checkpoint(part, w)
    for k in ("y", "codes", "scales", "rstd"):
        assert torch.equal(big[k][last], small[k]), k
    gx, _ = api.nvfp4_rmsnorm_checkpoint_backward(x, big["codes"], big["scales"], big["rstd"], w)
    gs, _ = api.nvfp4_rmsnorm_checkpoint_backward(part, small["codes"], small["scales"],
                                                  small["rstd"], w)
    assert torch.equal(gx[last], gs)
    del big, gx
    big = api.nvfp4_swiglu_checkpoint(x)
    dh = api.nvfp4_swiglu_checkpoint_backward(big["y"], big["codes"], big["scales"])
    for rows in (slice(0, 40), slice(65520, 65560), last):
        small = api.nvfp4_swiglu_checkpoint(x[rows].contiguous())
        for k in ("y", "codes", "scales"):
            assert torch.equal(big[k][rows], small[k]), k
        assert torch.equal(dh[rows], api.nvfp4_swiglu_checkpoint_backward(
            small["y"], small["codes"], small["scales"]))


def test_graph_replay_and_other_streams():
    dev = _cuda()
    M, F, N = 48, 96, 192
    h, x = (workloads.normal(M, n, 1.0, seed=n).to(dev) for n in (2 * F, N))
    w = torch.ones(N, dtype=torch.bfloat16, device=dev)
    offs = torch.tensor([10, 10, 44], dtype=torch.int32, device=dev)

    def step():
        a = api.nvfp4_swiglu_checkpoint(h, offsets=offs)
        dh = api.nvfp4_swiglu_checkpoint_backward(a["y"], a["codes"], a["scales"], offsets=offs)
        b = api.nvfp4_rmsnorm_checkpoint(x, w)
        gx, gw = api.nvfp4_rmsnorm_checkpoint_backward(b["y"], b["codes"], b["scales"], b["rstd"],
                                                       w, grad_residual=x)
        return [*a.values(), dh, *b.values(), gx, gw]

    step()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (5, 6):
        h.copy_(workloads.normal(M, 2 * F, 2.0, seed=seed))
        x.copy_(workloads.normal(M, N, 3.0, seed=seed))
        offs.copy_(torch.tensor([seed, 20, 40 + seed], dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            other = step()
        torch.cuda.synchronize()
        for a, b, c in zip(held, step(), other):
            assert torch.equal(a, b) and torch.equal(b, c)


def test_binding_checks_shapes():
    dev = _cuda()
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(128, dtype=torch.bfloat16, device=dev)
    k = api.nvfp4_rmsnorm_checkpoint(x, w)
    for call in (lambda: api.nvfp4_swiglu_checkpoint(x[:, :96].contiguous()),
                 lambda: api.nvfp4_swiglu_checkpoint(x[:, ::2]),
                 lambda: api.nvfp4_swiglu_checkpoint_backward(x, k["codes"], k["scales"]),
                 lambda: api.nvfp4_rmsnorm_checkpoint(x, w[:64]),
                 lambda: api.nvfp4_rmsnorm_checkpoint(x[:, :48].contiguous(), w[:48]),
                 lambda: api.nvfp4_rmsnorm_checkpoint(x, w, out=dict(k, rstd=k["rstd"][:2])),
                 lambda: api.nvfp4_rmsnorm_checkpoint_backward(x, k["codes"][:2], k["scales"],
                                                               k["rstd"], w),
                 lambda: api.nvfp4_rmsnorm_checkpoint_backward(x, k["codes"], k["scales"],
                                                               k["rstd"], w,
                                                               grad_residual=x[:2])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(_lib.NVFP4Error):  # a workspace that is too small
        api.nvfp4_rmsnorm_checkpoint_backward(
            x, k["codes"], k["scales"], k["rstd"], w,
            workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(TypeError):
        api.nvfp4_swiglu_checkpoint(x, offsets=torch.zeros(2, device=dev))
