"""The NVFP4 matrix products and the gradient of their epilogue against plain products in binary64."""
import math

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import api, workloads

pytestmark = pytest.mark.gpu


def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def operand(rows, K, seed, dev, lead=()):
    """Random codes, scales (one block in nine is zero) and a global scale."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (*lead, rows, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(0x28, 0x48, (*lead, rows, K // 16), generator=g, dtype=torch.uint8)
    scales[torch.rand(scales.shape, generator=g) < 1 / 9] = 0
    gs = torch.rand((*lead, 2), generator=g) * 0.02 + 0.01
    return codes.to(dev), scales.to(dev), gs.to(dev)


def values(codes, scales, gs=None):
    """What an operand stands for, binary64."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    grid = torch.cat([GRID, -GRID]).to(codes.device)
    v = grid[c] * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return v if gs is None else v * gs[..., 1].double()


def act(z, name):
    if name == "relu":
        return z.clamp_min(0)
    if name == "relu2":
        return z.clamp_min(0) ** 2
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z) if name == "silu" else z


def check_product(got, a, b, bias=None, activation=None, residual=None, live=None, preact=None):
    """a [M, K], b [N, K] binary64. The sum's error: every step of 64 products rounds the running sum
    (2^-23 of the absolute sum, cut or to nearest); then one rounding each for the scale, bias and
    residual, at most 1.2 times that through the activation's slope (2 |z| for relu2) and 8 units for
    its exponential; one rounding to the output's type."""
    z = a @ b.t()
    size = a.abs() @ b.abs().t()
    err = (a.shape[1] / 64 + 8) * 2.0 ** -23 * size
    if bias is not None:
        z = z + bias.double()
        err = err + 2.0 ** -23 * (z.abs() + bias.double().abs())
    half = 2.0 ** -8 if got.dtype is torch.bfloat16 else 2.0 ** -24
    if preact is not None:
        assert ((preact.double() - z).abs() <= err + 2.0 ** -8 * (z.abs() + err)).all()
    o = act(z, activation)
    slope = 2 * (z.abs() + err) if activation == "relu2" else 1.2
    tol = err * slope + (0 if activation in (None, "none", "relu") else 24 * 2.0 ** -23 * (1 + z.abs()) * o.abs())
    if residual is not None:
        o = o + residual.double()
        tol = tol + 2.0 ** -23 * o.abs()
    tol = tol + half * (o.abs() + tol) + 1e-37
    assert got.shape == o.shape
    bad = (got.double() - o).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                           ((got.double() - o).abs() / tol).max().item())


SHAPES = [(1, 1, 32), (1, 128, 64), (2, 33, 96), (1, 300, 4096), (17, 64, 256), (16, 130, 288),
          (33, 520, 512), (64, 96, 1024), (127, 129, 2080), (129, 257, 32), (256, 256, 256),
          (300, 200, 544), (257, 512, 768), (515, 1000, 320), (1024, 768, 1280)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm(M, N, K, dtype):
    dev = cuda()
    a, b = operand(M, K, 1 + M, dev), operand(N, K, 2 + N, dev)
    got = api.nvfp4_gemm(*a, *b, out_dtype=dtype)
    assert set(got) == {"out"} and got["out"].dtype == dtype
    check_product(got["out"], values(*a), values(*b))
    assert api.nvfp4_get_status() == (0, 0)


@pytest.mark.parametrize("M,N,K", [(2049, 1300, 288), (1290, 2048, 544), (2304, 2816, 32),
                                   (4000, 1016, 1312), (130, 9984, 320), (2560, 2560, 2560)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_of_many_tiles(M, N, K, dtype):
    """Out of more 256 x 256 tiles than half the SMs, partial ones among them, several to a pair of SMs."""
    dev = cuda()
    a, b = operand(M, K, 1 + M, dev), operand(N, K, 2 + N, dev)
    g = torch.Generator().manual_seed(5)
    bias = torch.randn(N, generator=g).to(dev)
    residual = torch.randn(M, N, generator=g).to(dtype).to(dev)
    got = api.nvfp4_gemm(*a, *b, bias=bias, activation="gelu", residual=residual, out_dtype=dtype,
                         keep_preact=True, with_amax=True)
    check_product(got["out"], values(*a), values(*b), bias, "gelu", residual, preact=got["preact"])
    assert got["amax"].item() == got["out"].abs().max().item()
    assert api.nvfp4_get_status() == (0, 0)


@pytest.mark.parametrize("K,offset", [(288, 0), (512, 3), (2080, 5)])
def test_large_products_without_a_workspace(K, offset):
    """Scales whose rows start anywhere are copied to a workspace or, without one, read as they are."""
    dev = cuda()
    M, N = 1300, 2056
    a, b = list(operand(M, K, 81, dev)), list(operand(N, K, 82, dev))
    for x in (a, b):
        wide = torch.full((x[1].shape[0], K // 16 + 7), 0x7F, dtype=torch.uint8, device=dev)
        wide[:, offset:offset + K // 16] = x[1]
        x[1] = wide[:, offset:offset + K // 16]
    none = torch.empty(0, dtype=torch.uint8, device=dev)
    some = torch.empty((M * K // 16 + 16 * M) // 16 * 16, dtype=torch.uint8, device=dev)  # for a alone
    want = api.nvfp4_gemm(*a, *b)["out"]
    for workspace in (none, some):
        for dtype in (torch.bfloat16, torch.float32):
            got = api.nvfp4_gemm(*a, *b, out_dtype=dtype, workspace=workspace)["out"]
            check_product(got, values(*a), values(*b))
        assert torch.equal(api.nvfp4_gemm(*a, *b, workspace=workspace)["out"], want)


@pytest.mark.parametrize("activation", ["none", "relu", "relu2", "gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(1, 160, 256), (45, 72, 96), (140, 261, 512), (700, 1028, 640)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bias_dtype", [torch.bfloat16, torch.float32])
def test_epilogue(activation, M, N, K, dtype, bias_dtype):
    dev = cuda()
    a, b = operand(M, K, 3, dev), operand(N, K, 4, dev)
    g = torch.Generator().manual_seed(5)
    bias = torch.randn(N, generator=g).to(bias_dtype).to(dev)
    residual = torch.randn(M, N, generator=g).to(dtype).to(dev)
    got = api.nvfp4_gemm(*a, *b, bias=bias, activation=activation, residual=residual, out_dtype=dtype,
                         keep_preact=True, with_amax=True)
    check_product(got["out"], values(*a), values(*b), bias, activation, residual, preact=got["preact"])
    assert got["amax"].item() == got["out"].abs().max().item()
    # each part alone
    check_product(api.nvfp4_gemm(*a, *b, bias=bias, out_dtype=dtype)["out"], values(*a), values(*b), bias)
    check_product(api.nvfp4_gemm(*a, *b, activation=activation, out_dtype=dtype)["out"], values(*a),
                  values(*b), None, activation)
    # the residual's own buffer as the output
    acc = residual.clone()
    api.nvfp4_gemm(*a, *b, residual=acc, out=acc)
    check_product(acc, values(*a), values(*b), residual=residual)


def test_activation_far_from_zero():
    """z up to 1e4 in magnitude: no overflow in the exponentials, the tails go to 0 and z."""
    dev = cuda()
    a, b = operand(64, 64, 6, dev), operand(128, 64, 7, dev)
    a[2][1], b[2][1] = 1.0, 1.0
    for activation in ("gelu", "silu", "relu2"):
        out = api.nvfp4_gemm(*a, *b, activation=activation, out_dtype=torch.float32)["out"]
        check_product(out, values(*a), values(*b), None, activation)


def test_zero_sizes():
    dev = cuda()
    a, b = operand(5, 64, 8, dev), operand(7, 64, 9, dev)
    assert api.nvfp4_gemm(*operand(0, 64, 8, dev), *b, with_amax=True)["amax"].item() == 0.0
    assert api.nvfp4_gemm(*a, *operand(0, 64, 9, dev))["out"].shape == (5, 0)
    bias = torch.arange(7.0, device=dev)
    got = api.nvfp4_gemm(*operand(5, 0, 8, dev), *operand(7, 0, 9, dev), bias=bias, activation="relu")
    assert torch.equal(got["out"], bias.to(torch.bfloat16).expand(5, 7))


@pytest.mark.parametrize("pad_codes,pad_scales", [(16, 16), (32, 1), (0, 2), (48, 4)])
@pytest.mark.parametrize("M,N", [(20, 300), (400, 390)])
def test_strided_operands(pad_codes, pad_scales, M, N):
    """Rows that are parts of longer ones; scales at odd addresses."""
    dev = cuda()
    K = 544
    tight = [operand(M, K, 10, dev), operand(N, K, 11, dev)]
    wide = []
    for codes, scales, gs in tight:
        c = torch.full((codes.shape[0], K // 2 + pad_codes), 0x77, dtype=torch.uint8, device=dev)
        s = torch.full((codes.shape[0], K // 16 + pad_scales), 0x7F, dtype=torch.uint8, device=dev)
        c[:, :K // 2], s[:, pad_scales:] = codes, scales
        wide += [c[:, :K // 2], s[:, pad_scales:], gs]
    got = api.nvfp4_gemm(*wide)["out"]
    check_product(got, values(*tight[0]), values(*tight[1]))
    assert torch.equal(got, api.nvfp4_gemm(*tight[0], *tight[1])["out"])


def test_extreme_scales_and_nan():
    """The largest finite scales, subnormal ones, and a NaN scale, which reaches its row alone."""
    dev = cuda()
    a, b = operand(40, 256, 12, dev), operand(136, 256, 13, dev)
    a[1][3], a[1][4], b[1][9], b[1][10] = 0x7E, 0x01, 0x7E, 0x01
    check_product(api.nvfp4_gemm(*a, *b, out_dtype=torch.float32)["out"], values(*a), values(*b))
    a[1][7, 2] = 0x7F
    out = api.nvfp4_gemm(*a, *b)["out"]
    assert torch.isnan(out[7]).all() and torch.isfinite(out[torch.arange(40) != 7]).all()


def test_of_the_quantizers_outputs():
    """Forward, input gradient and weight gradient of a linear layer from one quantization each of x,
    the weights (2D) and the gradient, the weight gradient's operands with the RHT."""
    dev = cuda()
    M, N, K = 256, 384, 512
    x = workloads.normal_with_outliers(M, K, seed=14).to(dev)
    w = workloads.normal(N, K, 0.05, seed=15).to(dev)
    g = workloads.laplace(M, N, 1e-3, seed=16).to(dev)
    qx = api.nvfp4_quantize(x, columnwise=True, rht_col=True, sign_mask=0x5A3C)
    qw = api.nvfp4_quantize(w, columnwise=True, block2d=True)
    qg = api.nvfp4_quantize(g, columnwise=True, rht_col=True, sign_mask=0x5A3C, round_col="sr", seed=3)
    row = lambda q: (q["row_codes"], q["row_scales"], q["row_gscale"])  # noqa: E731
    col = lambda q: (q["col_codes"], q["col_scales"], q["col_gscale"])  # noqa: E731
    for p, q in ((row(qx), row(qw)), (row(qg), col(qw)), (col(qg), col(qx))):
        for dtype in (torch.bfloat16, torch.float32):
            out = api.nvfp4_gemm(*p, *q, out_dtype=dtype)["out"]
            check_product(out, values(*p), values(*q))
    y = api.nvfp4_gemm(*row(qx), *row(qw), with_amax=True)
    q = api.nvfp4_quantize(y["out"], amax_row=y["amax"])
    for k, v in api.nvfp4_quantize(y["out"]).items():
        assert torch.equal(q[k], v)


COUNTS = [[5], [0, 3, 0], [1, 0, 129, 7], [300, 2, 0, 0, 41], [64] * 9, [0, 0, 520, 1, 255, 16],
          [1] * 40, [0] * 3, [700, 900, 400]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "x".join(map(str, c[:6])))
@pytest.mark.parametrize("N,K", [(72, 96), (264, 512), (136, 1056)])
@pytest.mark.parametrize("rest", [0, 21])
def test_grouped(counts, N, K, rest):
    dev = cuda()
    E, live = len(counts), sum(counts)
    T = live + rest
    ends = torch.tensor(np.cumsum(counts), dtype=torch.int32, device=dev)
    a = list(operand(T, K, 20, dev))
    a[2] = torch.rand(E, 2, generator=torch.Generator().manual_seed(21)).to(dev) + 0.5
    a[1][live:] = 0x7F  # NaN behind the last expert
    b = operand(N, K, 22, dev, lead=(E,))
    got = api.nvfp4_gemm_grouped(*a, *b, ends, with_amax=True)
    bias = torch.randn(E, N, generator=torch.Generator().manual_seed(23)).to(dev)
    full = api.nvfp4_gemm_grouped(*a, *b, ends, bias=bias, activation="silu", keep_preact=True,
                                  out_dtype=torch.float32)
    begin = 0
    for e, n in enumerate(counts):
        rows = slice(begin, begin + n)
        begin += n
        x, w = values(a[0][rows], a[1][rows], a[2][e]), values(b[0][e], b[1][e], b[2][e])
        check_product(got["out"][rows], x, w)
        assert got["amax"][e].item() == (got["out"][rows].abs().max().item() if n else 0.0)
        check_product(full["out"][rows], x, w, bias[e], "silu", preact=full["preact"][rows])
    assert not got["out"][live:].any() and not full["out"][live:].any() and not full["preact"][live:].any()
    assert api.nvfp4_get_status() == (0, 0)


@pytest.mark.parametrize("counts,rest", [([700, 900, 0, 400], 21), ([1500, 3, 260, 257, 511], 0)])
@pytest.mark.parametrize("N,K", [(2056, 288), (1300, 1056)])
def test_grouped_of_many_rows(counts, rest, N, K):
    dev = cuda()
    E, live = len(counts), sum(counts)
    T = live + rest
    ends = torch.tensor(np.cumsum(counts), dtype=torch.int32, device=dev)
    a, b = list(operand(T, K, 70, dev)), operand(N, K, 71, dev, lead=(E,))
    a[2] = torch.rand(E, 2, generator=torch.Generator().manual_seed(72)).to(dev) + 0.5
    a[1][live:] = 0x7F
    got = api.nvfp4_gemm_grouped(*a, *b, ends, activation="silu", with_amax=True, keep_preact=True)
    begin = 0
    for e, n in enumerate(counts):
        rows = slice(begin, begin + n)
        begin += n
        x, w = values(a[0][rows], a[1][rows], a[2][e]), values(b[0][e], b[1][e], b[2][e])
        check_product(got["out"][rows], x, w, None, "silu", preact=got["preact"][rows])
        assert got["amax"][e].item() == (got["out"][rows].abs().max().item() if n else 0.0)
    assert not got["out"][live:].any() and not got["preact"][live:].any()


@pytest.mark.parametrize("counts", [[300, 2, 0, 41], [0, 0, 520, 1, 255, 16]])
@pytest.mark.parametrize("M,N", [(1032, 776), (520, 2056)])
def test_grouped_wgrad_of_many_tiles(counts, M, N):
    dev = cuda()
    E, pads = len(counts), [(n + 15) // 16 * 16 for n in counts]
    cap = (sum(pads) + 31) // 32 * 32 + 32
    ends = torch.tensor(np.cumsum(counts), dtype=torch.int32, device=dev)
    a, b = list(operand(M, cap, 73, dev)), list(operand(N, cap, 74, dev))
    a[2], b[2] = torch.rand(E, 2).to(dev) + 0.5, torch.rand(E, 2).to(dev) + 0.5
    for x in (a, b):
        x[1][:, sum(pads) // 16:] = 0x7F
    before = torch.randn(E, M, N, generator=torch.Generator().manual_seed(75)).to(dev)
    got = api.nvfp4_gemm_grouped_wgrad(*a, *b, ends)
    added = api.nvfp4_gemm_grouped_wgrad(*a, *b, ends, out=before.clone(), accumulate=True)
    at = 0
    for e, n in enumerate(pads):
        c, s = slice(at // 2, (at + n) // 2), slice(at // 16, (at + n) // 16)
        at += n
        x, y = (values(o[0][:, c].contiguous(), o[1][:, s].contiguous(), o[2][e]) for o in (a, b))
        check_product(got[e], x, y)
        check_product(added[e], x, y, residual=before[e])


@pytest.mark.parametrize("E,most", [(24, 5), (9, 100)])
def test_grouped_of_many_small_experts(E, most):
    """More tiles of the small kernels than the GPU holds at once: several to a CTA."""
    dev = cuda()
    N, K = 128 * 80 - 8, 1312
    counts = [int(n) for n in torch.randint(0, most, (E,), generator=torch.Generator().manual_seed(76))]
    T = sum(counts)
    ends = torch.tensor(np.cumsum(counts), dtype=torch.int32, device=dev)
    a, b = list(operand(T, K, 77, dev)), operand(N, K, 78, dev, lead=(E,))
    a[2] = torch.rand(E, 2, generator=torch.Generator().manual_seed(79)).to(dev) + 0.5
    got = api.nvfp4_gemm_grouped(*a, *b, ends, with_amax=True)
    begin = 0
    for e, n in enumerate(counts):
        rows = slice(begin, begin + n)
        begin += n
        check_product(got["out"][rows], values(a[0][rows], a[1][rows], a[2][e]),
                      values(b[0][e], b[1][e], b[2][e]))
        assert got["amax"][e].item() == (got["out"][rows].abs().max().item() if n else 0.0)
    assert api.nvfp4_get_status() == (0, 0)


def test_grouped_input_gradient_from_columnwise_weights():
    """grad_in[rows of e] = grad_out[rows of e] W_e from the columnwise outputs of the stacked weights,
    a strided view of them."""
    dev = cuda()
    counts, N, K = [30, 0, 200, 65], 96, 160
    E, T = len(counts), sum(counts)
    ends = torch.tensor(np.cumsum(counts), dtype=torch.int32, device=dev)
    w = workloads.normal(E * N, K, 0.05, seed=24).to(dev)
    wends = torch.arange(1, E + 1, dtype=torch.int32, device=dev) * N
    qw = api.nvfp4_quantize_grouped(w, wends, col_capacity=E * N, block2d=True)
    g = workloads.laplace(T, N, 1e-3, seed=25).to(dev)
    qg = api.nvfp4_quantize_grouped(g, ends, columnwise=False)
    b_codes = qw["col_codes"].view(K, E, N // 2).transpose(0, 1)
    b_scales = qw["col_scales"].view(K, E, N // 16).transpose(0, 1)
    got = api.nvfp4_gemm_grouped(qg["row_codes"], qg["row_scales"], qg["row_gscale"], b_codes, b_scales,
                                 qw["col_gscale"], ends)["out"]
    assert got.shape == (T, K)
    begin = 0
    for e, n in enumerate(counts):
        rows = slice(begin, begin + n)
        begin += n
        check_product(got[rows], values(qg["row_codes"][rows], qg["row_scales"][rows], qg["row_gscale"][e]),
                      values(b_codes[e].contiguous(), b_scales[e].contiguous(), qw["col_gscale"][e]))


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "x".join(map(str, c[:6])))
@pytest.mark.parametrize("M,N", [(40, 72), (272, 136), (16, 640)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_grouped_wgrad(counts, M, N, dtype):
    dev = cuda()
    E = len(counts)
    pads = [(n + 15) // 16 * 16 for n in counts]
    cap = (sum(pads) + 31) // 32 * 32 + 64
    ends = torch.tensor(np.cumsum(counts), dtype=torch.int32, device=dev)
    a, b = list(operand(M, cap, 26, dev)), list(operand(N, cap, 27, dev))
    g = torch.Generator().manual_seed(28)
    a[2], b[2] = (torch.rand(E, 2, generator=g).to(dev) + 0.5 for _ in range(2))
    for x in (a, b):
        x[1][:, sum(pads) // 16:] = 0x7F  # NaN behind the last expert
    got = api.nvfp4_gemm_grouped_wgrad(*a, *b, ends, out_dtype=dtype)
    before = torch.randn(E, M, N, generator=g).to(dtype).to(dev)
    added = api.nvfp4_gemm_grouped_wgrad(*a, *b, ends, out=before.clone(), accumulate=True)
    at = 0
    for e, n in enumerate(pads):
        c, s = slice(at // 2, (at + n) // 2), slice(at // 16, (at + n) // 16)
        at += n
        x, y = (values(o[0][:, c].contiguous(), o[1][:, s].contiguous(), o[2][e]) for o in (a, b))
        check_product(got[e], x, y)
        check_product(added[e], x, y, residual=before[e])
        if n == 0:
            assert not got[e].any() and torch.equal(added[e], before[e])
    assert api.nvfp4_get_status() == (0, 0)


def test_grouped_wgrad_ignores_other_experts_nan():
    """Experts share 32-element units of the columnwise codes: a NaN scale stays with its expert."""
    dev = cuda()
    counts = [16, 33, 7]
    ends = torch.tensor(np.cumsum(counts), dtype=torch.int32, device=dev)
    a, b = list(operand(48, 96, 29, dev)), list(operand(64, 96, 30, dev))
    a[2], b[2] = torch.ones(3, 2, device=dev), torch.ones(3, 2, device=dev)
    a[1][5, 2] = 0x7F  # token block 2: expert 1
    out = api.nvfp4_gemm_grouped_wgrad(*a, *b, ends)
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()
    assert torch.isnan(out[1, 5]).all() and torch.isfinite(out[1, :5]).all()


def test_bad_offsets_are_flagged():
    dev = cuda()
    a, b = list(operand(64, 64, 31, dev)), operand(32, 64, 32, dev, lead=(3,))
    a[2] = torch.ones(3, 2, device=dev)
    c, d = list(operand(48, 64, 33, dev)), list(operand(32, 64, 34, dev))
    c[2] = d[2] = torch.ones(3, 2, device=dev)
    for ends in ([10, 5, 64], [-1, 3, 64], [10, 20, 65], [70, 80, 90]):
        offsets = torch.tensor(ends, dtype=torch.int32, device=dev)
        api.nvfp4_gemm_grouped(*a, *b, offsets)
        assert api.nvfp4_get_status()[1] == 1, ends
        api.nvfp4_gemm_grouped_wgrad(*c, *d, offsets)
        assert api.nvfp4_get_status()[1] == 1, ends
    api.nvfp4_gemm_grouped_wgrad(*c, *d, torch.tensor([15, 30, 33], dtype=torch.int32, device=dev))
    assert api.nvfp4_get_status() == (0, 0)  # 16 + 16 + 16 columns
    api.nvfp4_gemm_grouped_wgrad(*c, *d, torch.tensor([17, 34, 51], dtype=torch.int32, device=dev))
    assert api.nvfp4_get_status()[1] == 1    # 32 + 32 + 32


def test_captured_calls_replay_and_streams():
    """Captured products on new data, and the same calls on another stream."""
    dev = cuda()
    M, N, K, E = 70, 136, 320, 4
    a, b = operand(M, K, 35, dev), operand(N, K, 36, dev, lead=(E,))
    ag = torch.ones(E, 2, device=dev)
    ends = torch.tensor([10, 30, 30, 66], dtype=torch.int32, device=dev)
    dense = api.nvfp4_gemm(*a, b[0][0], b[1][0], b[2][0], with_amax=True)
    grouped = api.nvfp4_gemm_grouped(a[0], a[1], ag, *b, ends, with_amax=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.nvfp4_gemm(*a, b[0][0], b[1][0], b[2][0], out=dense["out"], amax=dense["amax"])
        api.nvfp4_gemm_grouped(a[0], a[1], ag, *b, ends, out=grouped["out"], amax=grouped["amax"])
    a[0].copy_(operand(M, K, 37, dev)[0])
    ends.copy_(torch.tensor([0, 50, 51, 70], device=dev))
    graph.replay()
    want = api.nvfp4_gemm(*a, b[0][0], b[1][0], b[2][0], with_amax=True)
    want2 = api.nvfp4_gemm_grouped(a[0], a[1], ag, *b, ends, with_amax=True)
    for x, y in ((dense, want), (grouped, want2)):
        assert torch.equal(x["out"], y["out"]) and torch.equal(x["amax"], y["amax"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = api.nvfp4_gemm_grouped(a[0], a[1], ag, *b, ends)
    side.synchronize()
    assert torch.equal(other["out"], want2["out"])


def test_two_streams_at_once():
    dev = cuda()
    ops = [(operand(300, 768, 40 + i, dev), operand(520, 768, 50 + i, dev)) for i in range(4)]
    want = [api.nvfp4_gemm(*a, *b)["out"] for a, b in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    got = [[] for _ in ops]
    for _ in range(5):
        for i, (s, (a, b)) in enumerate(zip(streams, ops)):
            with torch.cuda.stream(s):
                got[i].append(api.nvfp4_gemm(*a, *b)["out"])
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)


# ---- the gradient through the epilogue -------------------------------------------------------------


@pytest.mark.parametrize("activation", ["none", "relu", "relu2", "gelu", "silu"])
@pytest.mark.parametrize("M,N", [(1, 8), (3, 2048), (700, 72), (129, 4104), (1030, 1024), (1, 1), (517, 7),
                                 (90, 1001), (3, 4098), (1003, 999), (4097, 33), (32, 1000), (33, 1000), (31, 77), (34, 77)])
def test_epilogue_backward(activation, M, N):
    dev = cuda()
    g = torch.Generator().manual_seed(M + N)
    z = (2 * torch.randn(M, N, generator=g)).to(torch.bfloat16)
    z[0, :4] = torch.tensor([0.0, -0.0, 60.0, -60.0])[:N]
    dy = torch.randn(M, N, generator=g).to(torch.bfloat16)
    z, dy = z.to(dev), dy.to(dev)
    d, db, amax = api.nvfp4_gemm_epilogue_backward(dy, z, activation)
    zd = z.double().requires_grad_()
    y = act(zd, activation)
    (y if y.requires_grad and y is not zd else zd * 1.0).backward(dy.double())
    want = zd.grad
    if activation == "relu":
        want = torch.where(z == 0, 0, want)  # either is a subgradient; the operator takes 0
    # the slope's exponential, 24 units times its argument as in the forward pass; one rounding
    err = 24 * 2.0 ** -23 * (1 + z.double().abs()) * dy.double().abs() * 1.2
    assert ((d.double() - want).abs() <= err + 2.0 ** -8 * want.abs() + 1e-37).all()
    assert amax.item() == d.abs().max().item()
    # sums of M terms in binary32
    tol = err.sum(0) + (M + 8) * 2.0 ** -24 * want.abs().sum(0) + 1e-30
    assert ((db.double() - want.sum(0)).abs() <= tol).all()
    again = api.nvfp4_gemm_epilogue_backward(dy, z, activation)
    assert all(torch.equal(p, q) for p, q in zip(again, (d, db, amax)))
    inplace = dy.clone()
    api.nvfp4_gemm_epilogue_backward(inplace, z, activation, grad_preact=inplace)
    assert torch.equal(inplace, d)


def test_epilogue_backward_against_differences():
    dev = cuda()
    z = torch.linspace(-6, 6, 8 * 40, device=dev).reshape(40, 8).to(torch.bfloat16)
    one = torch.ones_like(z)
    for activation in ("gelu", "silu", "relu2"):
        d, _, _ = api.nvfp4_gemm_epilogue_backward(one, z, activation)
        h = 1e-4
        slope = (act(z.double() + h, activation) - act(z.double() - h, activation)) / (2 * h)
        assert ((d.double() - slope).abs() <= 2.0 ** -8 * slope.abs() + 2e-5).all()


def test_epilogue_backward_without_rows():
    dev = cuda()
    x = torch.empty(0, 16, dtype=torch.bfloat16, device=dev)
    d, db, amax = api.nvfp4_gemm_epilogue_backward(x, x, "gelu")
    assert d.shape == (0, 16) and not db.any() and amax.item() == 0.0


def test_a_layer_forward_and_backward():
    """out = gelu(x W1^T + b1) W2^T + x with every product in NVFP4: the gradients against the same
    graph on the dequantized operands in binary64."""
    dev = cuda()
    M, H, F = 160, 256, 512
    x = workloads.normal(M, H, 1.0, seed=60).to(dev)
    w1 = workloads.normal(F, H, H ** -0.5, seed=61).to(dev)
    w2 = workloads.normal(H, F, F ** -0.5, seed=62).to(dev)
    b1 = workloads.normal(1, F, 0.1, seed=63)[0].to(dev)
    dout = workloads.normal(M, H, 1e-2, seed=64).to(dev)
    row = lambda q: (q["row_codes"], q["row_scales"], q["row_gscale"])  # noqa: E731
    col = lambda q: (q["col_codes"], q["col_scales"], q["col_gscale"])  # noqa: E731
    both = lambda t, **k: api.nvfp4_quantize(t, columnwise=True, **k)  # noqa: E731
    qx, q1, q2 = both(x), both(w1, block2d=True), both(w2, block2d=True)
    h = api.nvfp4_gemm(*row(qx), *row(q1), bias=b1, activation="gelu", keep_preact=True, with_amax=True)
    qh = both(h["out"], amax_row=h["amax"], amax_col=h["amax"])
    out = api.nvfp4_gemm(*row(qh), *row(q2), residual=x)["out"]
    qd = both(dout)
    dh = api.nvfp4_gemm(*row(qd), *col(q2))["out"]
    dw2 = api.nvfp4_gemm(*col(qd), *col(qh), out_dtype=torch.float32)["out"]
    dz, db1, top = api.nvfp4_gemm_epilogue_backward(dh, h["preact"], "gelu")
    qz = both(dz, amax_row=top, amax_col=top)
    dx = api.nvfp4_gemm(*row(qz), *col(q1), residual=dout)["out"]
    dw1 = api.nvfp4_gemm(*col(qz), *col(qx), out_dtype=torch.float32)["out"]
    # the formulas on what each product was given
    check_product(out, values(*row(qh)), values(*row(q2)), residual=x)
    check_product(dh, values(*row(qd)), values(*col(q2)))
    check_product(dw2, values(*col(qd)), values(*col(qh)))
    check_product(dx, values(*row(qz)), values(*col(q1)), residual=dout)
    check_product(dw1, values(*col(qz)), values(*col(qx)))
    # and all of it against autograd in binary64 without quantization: E2M1 operands are off by about
    # a tenth (a step of 1/2 to 2 in up to 6), each product by that times sqrt(2)
    t = [v.double().requires_grad_() for v in (x, w1, w2, b1)]
    y = act(t[0] @ t[1].t() + t[3], "gelu") @ t[2].t() + t[0]
    y.backward(dout.double())
    for got, want in ((out, y.detach()), (dx, t[0].grad), (dw1, t[1].grad), (dw2, t[2].grad),
                      (db1, t[3].grad)):
        assert (got.double() - want).norm() / want.norm() < 0.35
