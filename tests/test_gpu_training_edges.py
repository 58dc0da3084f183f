"""The router, the NVFP4 products and AdamW where their calls are least ordinary: sizes whose offsets pass
32 bits, experts that lie closer together than a row is long, outputs that start anywhere, NaN beside the
amax, graphs that replay at once."""
import ctypes

import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import _lib, api
from test_gpu_gemm import act, check_product, cuda, operand, values
from test_gpu_router import check

pytestmark = pytest.mark.gpu


def random_bytes(dev, *shape):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device=dev)


def random_scales(dev, *shape):
    return torch.randint(0x28, 0x48, shape, dtype=torch.uint8, device=dev)


@pytest.mark.parametrize("E,N,K", [(64, 300, 32), (256, 40, 32), (40, 520, 96)])
@pytest.mark.parametrize("mean", [2, 90])
def test_experts_closer_together_than_there_are_experts(E, N, K, mean):
    """Columnwise stacked weights of few rows an expert: K / 2 bytes from an expert to the next, E of them
    in a row."""
    dev = cuda()
    torch.manual_seed(E)
    counts = torch.randint(0, 2 * mean + 1, (E,))
    T = int(counts.sum())
    ends = counts.cumsum(0).to(torch.int32).to(dev)
    a = random_bytes(dev, T, K // 2), random_scales(dev, T, K // 16), torch.rand(E, 2, device=dev)
    codes = random_bytes(dev, N, E, K // 2).transpose(0, 1)
    scales = random_scales(dev, N, E, K // 16).transpose(0, 1)
    gs = torch.rand(E, 2, device=dev)
    got = api.nvfp4_gemm_grouped(*a, codes, scales, gs, ends)["out"]
    begin = 0
    for e in range(0, E):
        end = int(ends[e])
        if end > begin and e % 5 == 0:
            check_product(got[begin:end], values(a[0][begin:end], a[1][begin:end], a[2][e]),
                          values(codes[e].contiguous(), scales[e].contiguous(), gs[e]))
        begin = end
    assert api.nvfp4_get_status() == (0, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(3, 130), (70, 264), (300, 520), (2100, 2312)])
def test_outputs_that_start_anywhere(dtype, M, N):
    """out, residual and preact inside larger buffers, a few elements off any boundary: the results are
    those of aligned ones and what lies around them stays."""
    dev = cuda()
    a, b = operand(M, 96, 1, dev), operand(N, 96, 2, dev)
    g = torch.Generator().manual_seed(3)
    residual = torch.randn(M, N, generator=g).to(dtype).to(dev)
    bias = torch.randn(N, generator=g).to(dev)
    want = api.nvfp4_gemm(*a, *b, bias=bias, activation="silu", residual=residual, out_dtype=dtype,
                          keep_preact=True, with_amax=True)

    def inside(off, t):
        flat = torch.full((M * N + 64,), 7, dtype=t, device=dev)
        return flat, flat[off:off + M * N].view(M, N)
    for off in (1, 2, 4, 8):
        whole, out = inside(off, dtype)
        whole_z, z = inside(off + 1, torch.bfloat16)
        _, r = inside(off + 3, dtype)
        r.copy_(residual)
        got = api.nvfp4_gemm(*a, *b, bias=bias, activation="silu", residual=r, out=out, preact=z,
                             with_amax=True)
        assert torch.equal(out, want["out"]) and torch.equal(z, want["preact"])
        assert torch.equal(got["amax"], want["amax"])
        assert (whole[:off] == 7).all() and (whole[off + M * N:] == 7).all()
        assert (whole_z[:off + 1] == 7).all() and (whole_z[off + 1 + M * N:] == 7).all()
        out.copy_(residual)  # the residual is the output itself
        api.nvfp4_gemm(*a, *b, bias=bias, activation="silu", residual=out, out=out)
        assert torch.equal(out, want["out"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(5, 136), (300, 520), (2100, 2312), (2100, 2311)])
def test_nan_does_not_count_in_the_amax(dtype, M, N):
    dev = cuda()
    a, b = operand(M, 64, 1, dev), operand(N, 64, 2, dev)
    bias = torch.zeros(N, device=dev)
    bias[::9] = float("nan")
    got = api.nvfp4_gemm(*a, *b, bias=bias, out_dtype=dtype, with_amax=True)
    out = got["out"]
    assert out[:, ::9].isnan().all() and got["amax"].item() == out.abs().nan_to_num(0.0).max().item()
    dy = torch.randn(M, N, device=dev).to(torch.bfloat16)
    dy[:, ::7] = float("nan")
    d, _, amax = api.nvfp4_gemm_epilogue_backward(dy, dy.nan_to_num(1.0), "none")
    assert d[:, ::7].isnan().all() and amax.item() == d.abs().nan_to_num(0.0).max().item()


def test_an_operand_times_itself():
    dev = cuda()
    a = operand(400, 512, 1, dev)
    got = api.nvfp4_gemm(*a, *a, out_dtype=torch.float32)["out"]
    check_product(got, values(*a), values(*a))


def test_epilogue_backward_without_its_sums():
    """The C entry point with neither the bias's gradient nor the amax, and so without a workspace."""
    dev = cuda()
    for M, N in ((1, 40), (300, 264), (300, 13)):
        z = torch.randn(M, N, device=dev).to(torch.bfloat16)
        dy = torch.randn(M, N, device=dev).to(torch.bfloat16)
        want = api.nvfp4_gemm_epilogue_backward(dy, z, "gelu")[0]
        out = torch.empty_like(dy)
        s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert _lib.load().nvfp4_gemm_epilogue_backward(dy.data_ptr(), z.data_ptr(), M, N, 3, out.data_ptr(),
                                                        None, None, None, 0, s) == 0
        assert torch.equal(out, want)


def test_captured_graphs_that_replay_at_once():
    """Two graphs, each with large products whose scales are copied to a workspace of its own, replayed
    on two streams at a time."""
    dev = cuda()
    M, N, K = 1300, 2056, 288
    ops = [(operand(M, K, 5 + i, dev), operand(N, K, 9 + i, dev)) for i in range(2)]
    want = [api.nvfp4_gemm(*a, *b, with_amax=True) for a, b in ops]
    graphs, got = [], []
    for a, b in ops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = api.nvfp4_gemm(*a, *b, with_amax=True)
            r["again"] = api.nvfp4_gemm(*a, *b, bias=None, activation="relu")["out"]
        graphs.append(g)
        got.append(r)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(8):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for r, w in zip(got, want):
        assert torch.equal(r["out"], w["out"]) and torch.equal(r["amax"], w["amax"])
        assert torch.equal(r["again"], w["out"].clamp_min(0))
    assert api.nvfp4_get_status() == (0, 0)


# ---- offsets past 32 bits ----------------------------------------------------------------------------

def few(M):
    """Rows at the start, about the middle and at the end of M."""
    return [slice(0, 40), slice(M // 2 - 20, M // 2 + 20), slice(M - 40, M)]


@pytest.mark.parametrize("dtype,N", [(torch.bfloat16, 32008), (torch.float32, 32007)])
def test_large_output(dtype, N):
    dev = cuda()
    M, K = 70001, 32
    a = random_bytes(dev, M, K // 2), random_scales(dev, M, K // 16), torch.ones(2, device=dev)
    b = random_bytes(dev, N, K // 2), random_scales(dev, N, K // 16), torch.ones(2, device=dev)
    got = api.nvfp4_gemm(*a, *b, activation="relu", out_dtype=dtype, keep_preact=dtype is torch.float32)
    bd = values(*b)
    for r in few(M):
        check_product(got["out"][r], values(a[0][r], a[1][r], a[2]), bd, activation="relu",
                      preact=got["preact"][r] if "preact" in got else None)
    assert api.nvfp4_get_status() == (0, 0)


def test_large_operand():
    """Codes of more than 2^32 bytes, dense and as 3 experts' rows."""
    dev = cuda()
    M, N, K = 540001, 24, 16384
    a = random_bytes(dev, M, K // 2), random_scales(dev, M, K // 16), torch.ones(2, device=dev)
    b = random_bytes(dev, 3, N, K // 2), random_scales(dev, 3, N, K // 16), torch.ones(3, 2, device=dev)
    dense = api.nvfp4_gemm(*a, *(t[2].contiguous() for t in b))["out"]
    ends = torch.tensor([1000, 2000, M], dtype=torch.int32, device=dev)
    grouped = api.nvfp4_gemm_grouped(a[0], a[1], torch.ones(3, 2, device=dev), *b, ends)["out"]
    bd = values(b[0][2], b[1][2], b[2][2])
    for r in few(M):
        check_product(dense[r], values(a[0][r], a[1][r], a[2]), bd)
    assert torch.equal(grouped[2000:], dense[2000:])
    assert api.nvfp4_get_status() == (0, 0)


@pytest.mark.parametrize("accumulate", [False, True])
def test_large_weight_gradients(accumulate):
    dev = cuda()
    E, M, N, n = 9, 16384, 16392, 32
    a = random_bytes(dev, M, E * n // 2), random_scales(dev, M, E * n // 16), torch.ones(E, 2, device=dev)
    b = random_bytes(dev, N, E * n // 2), random_scales(dev, N, E * n // 16), torch.ones(E, 2, device=dev)
    ends = torch.arange(1, E + 1, dtype=torch.int32, device=dev) * n
    out = torch.ones(E, M, N, device=dev)
    api.nvfp4_gemm_grouped_wgrad(*a, *b, ends, out=out, accumulate=accumulate)
    for e in (0, E - 1):
        c, s = slice(e * n // 2, (e + 1) * n // 2), slice(e * n // 16, (e + 1) * n // 16)
        bd = values(b[0][:, c], b[1][:, s], b[2][e])
        for r in few(M):
            check_product(out[e][r], values(a[0][r, c], a[1][r, s], a[2][e]), bd,
                          residual=torch.ones(40, N, device=dev) if accumulate else None)
    assert api.nvfp4_get_status() == (0, 0)


def test_many_tokens():
    dev = cuda()
    T, E, K = (1 << 24) + 37, 256, 4
    x = torch.empty(T, E, dtype=torch.bfloat16, device=dev).normal_()
    ids, w = api.nvfp4_moe_router(x, K)
    gw = torch.randn(T, K, device=dev)
    d = api.nvfp4_moe_router_backward(gw, x, ids)
    for r in few(T):
        some, sw = api.nvfp4_moe_router(x[r], K)
        assert torch.equal(ids[r], some) and torch.equal(w[r], sw)
        assert torch.equal(d[r], api.nvfp4_moe_router_backward(gw[r], x[r], some))
    assert api.nvfp4_get_status() == (0, 0)


@pytest.mark.parametrize("N", [32008, 32007])
def test_large_epilogue_gradient(N):
    dev = cuda()
    M = 70001
    z = torch.empty(M, N, dtype=torch.bfloat16, device=dev).normal_()
    dy = torch.ones_like(z)
    d, db, amax = api.nvfp4_gemm_epilogue_backward(dy, z, "gelu")
    for r in few(M):
        zd = z[r].double().requires_grad_()
        act(zd, "gelu").backward(torch.ones_like(zd))
        err = 24 * 2.0 ** -23 * (1 + z[r].double().abs()) * 1.2  # as for the sizes that are not large
        assert ((d[r].double() - zd.grad).abs() <= err + 2.0 ** -8 * zd.grad.abs() + 1e-37).all()
    assert amax.item() == max(d[i:i + 10000].abs().max().item() for i in range(0, M, 10000))
    d, db, amax = api.nvfp4_gemm_epilogue_backward(dy, z, "none", grad_preact=dy)
    assert (db == M).all() and amax.item() == 1.0  # whole numbers below 2^24: exact


@pytest.mark.parametrize("bits", [32, 8])
def test_large_tensor_in_a_step(bits):
    """A tensor of more than 2^31 elements: its ends as tensors of their own come out the same (with 8 bits
    but for the random part of the square root's codes, at most one code)."""
    dev = cuda()
    n, part = (1 << 31) + 40, 4096
    p = torch.empty(n, device=dev).normal_()
    g = torch.empty(n, dtype=torch.bfloat16, device=dev).normal_()
    w = torch.empty(n, dtype=torch.bfloat16, device=dev)
    last = n - part - 8  # a multiple of 32
    spans = [slice(0, part), slice(last, n)]
    small = [p[s].clone() for s in spans], [g[s].clone() for s in spans], [w[s].clone() for s in spans]
    large, other = api.AdamW([p], [g], [w], state_bits=bits), api.AdamW(*small, state_bits=bits)
    amax = large.step(1)
    other.step(1)
    for i, s in enumerate(spans):
        assert torch.equal(p[s], small[0][i]) and torch.equal(w[s], small[2][i])
        for k, t in large.state.items():
            c = slice(s.start // 32, (s.stop + 31) // 32) if k.endswith("scales") else s
            x, y = t[0][c], other.state[k][i]
            if bits == 8 and k == "exp_avg_sq":
                assert ((x.int() - y.int()).abs() <= 1).all()
            else:
                assert torch.equal(x, y), k
    assert amax.item() == max(w[i:i + (1 << 28)].abs().max().item() for i in range(0, n, 1 << 28))


# ---- the router's order among few close scores ------------------------------------------------------

@pytest.mark.parametrize("E,K,groups,top_groups", [(256, 8, 1, 1), (256, 8, 8, 4), (160, 6, 8, 3), (64, 12, 1, 1),
                                                   (250, 20, 1, 1), (96, 32, 1, 1), (256, 1, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("close", [2, 7, 40])
def test_few_scores_that_binary32_cannot_tell_apart(E, K, groups, top_groups, score, close):
    """`close` experts of a row at steps of one unit in the last place, some of them equal, among others that
    are far: they straddle the last chosen, or are all chosen, or fill every place."""
    dev = cuda()
    g = torch.Generator().manual_seed(E + K + close)
    T = 300
    x = torch.randn(T, E, generator=g)
    above = torch.randint(0, K + 1, (T,), generator=g)  # experts that are far above the close ones
    for t in range(T):
        order = torch.randperm(E, generator=g)
        n = int(above[t])
        x[t, order[:n]] = 5 + 0.125 * torch.arange(n)
        steps = torch.randint(0, max(2, close // 2), (close,), generator=g)
        x[t, order[n:n + close]] = 3.5 + steps * 2.0 ** -22
    bias = (torch.randint(-8, 9, (E,), generator=g) * 2.0 ** -24).float()
    check(x.to(dev), K, bias.to(dev), score=score, groups=groups, top_groups=top_groups)
    check(x.to(dev), K, torch.zeros(E, device=dev), score=score, groups=groups, top_groups=top_groups)
    x[:100, torch.randperm(E, generator=g)[:E - K // 2 - 1]] = -float("inf")  # fewer than K are left
    check(x.to(dev), K, bias.to(dev), score=score, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_equal_logits(dtype):
    dev = cuda()
    for E, groups, top in ((256, 1, 1), (64, 8, 2), (20, 1, 1)):
        for bias in (None, torch.zeros(E, device=dev)):
            for score in ("sigmoid", "softmax"):
                ids, w = api.nvfp4_moe_router(torch.zeros(40, E, dtype=dtype, device=dev), 4, score=score,
                                              bias=bias, groups=groups, top_groups=top)
                assert (ids == torch.arange(4, device=dev)).all() and (w == 0.25).all()


@pytest.mark.parametrize("E,K,groups,top_groups", [(256, 8, 8, 4), (160, 6, 8, 3), (64, 4, 16, 5), (250, 8, 10, 4),
                                                   (32, 4, 32, 9), (256, 8, 4, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_that_binary32_cannot_tell_apart(E, K, groups, top_groups, score, biased):
    """Groups whose two largest are another group's, in another order and up to a unit in the last place."""
    dev = cuda()
    g = torch.Generator().manual_seed(E + groups)
    T, size = 300, E // groups
    x = torch.randn(T, groups, size, generator=g)
    for t in range(T):
        for _ in range(3):
            i, j = torch.randint(0, groups, (2,), generator=g).tolist()
            units = torch.randint(-1, 2, (size,), generator=g) * 2.0 ** -23
            x[t, j] = (x[t, i] * (1 + units))[torch.randperm(size, generator=g)]
    x = x.view(T, E)
    bias = torch.zeros(E) + 2.0 ** -20 if biased else None
    check(x.to(dev), K, None if bias is None else bias.to(dev), score=score, groups=groups, top_groups=top_groups)
    short = x.to(torch.bfloat16)
    check(short.to(dev), K, None if bias is None else bias.to(dev), score=score, groups=groups,
          top_groups=top_groups)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N", [(40, 72), (520, 776), (2056, 1304), (1031, 1301)])
def test_experts_without_tokens_keep_their_gradients(dtype, M, N):
    """With accumulate: bit for bit, whatever is there."""
    dev = cuda()
    counts = [0, 40, 0, 0, 7, 0]
    E, n = len(counts), 64  # 48 + 16 columns of K
    ends = torch.tensor(counts).cumsum(0).to(torch.int32).to(dev)
    a = random_bytes(dev, M, n // 2), random_scales(dev, M, n // 16), torch.ones(E, 2, device=dev)
    b = random_bytes(dev, N, n // 2), random_scales(dev, N, n // 16), torch.ones(E, 2, device=dev)
    whole = torch.int32 if dtype is torch.float32 else torch.int16
    bits = torch.iinfo(whole)
    before = torch.randint(bits.min, bits.max, (E, M, N), dtype=whole, device=dev)
    out = before.clone().view(dtype)
    out[1] = 1.0
    out[4] = 1.0
    api.nvfp4_gemm_grouped_wgrad(*a, *b, ends, out=out, accumulate=True)
    for e in (0, 2, 3, 5):
        assert torch.equal(out[e].view(whole), before[e])
    for e, lo in ((1, 0), (4, 48)):
        hi = lo + (counts[e] + 15) // 16 * 16
        check_product(out[e], values(a[0][:, lo // 2:hi // 2], a[1][:, lo // 16:hi // 16], a[2][e]),
                      values(b[0][:, lo // 2:hi // 2], b[1][:, lo // 16:hi // 16], b[2][e]),
                      residual=torch.ones(M, N, device=dev))
    assert api.nvfp4_get_status() == (0, 0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,K", [(64, 1), (68, 1), (256, 1), (256, 6), (15, 3)])
def test_a_single_choice_has_weight_one_and_no_gradient(score, dtype, E, K):
    """With renormalization, exactly: the weight does not depend on the logit. K > 1: the rest is masked."""
    dev = cuda()
    g = torch.Generator().manual_seed(E)
    x = 4 * torch.randn(500, E, generator=g)
    if K > 1:
        one = torch.randint(0, E, (500, 1), generator=g)
        x = torch.full_like(x, -float("inf")).scatter(1, one, x.gather(1, one))
    x = x.to(dtype).to(dev)
    for bias in (None, torch.randn(E, generator=g).to(dev)):
        ids, w = api.nvfp4_moe_router(x, K, score=score, bias=bias, scale=2.5)
        assert (w[:, 0] == 2.5).all() and not w[:, 1:].any() and (ids[:, 1:] == -1).all()
        d = api.nvfp4_moe_router_backward(torch.randn(500, K, generator=g).to(dev), x, ids, score=score, scale=2.5)
        assert not d.any()
