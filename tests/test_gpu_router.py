"""The router and its gradient against their definition in binary64."""
import math

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import api

pytestmark = pytest.mark.gpu

# exp of binary32 arguments up to 20 in magnitude: 2 + 1.173 * 20 units in the last place (of 2^-23),
# twice (numerator and sum), a division of 2
EXP_TOL = (2 * 26 + 4) * 2.0 ** -23


def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


def scores(x, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-x))
    top = x.max(1, keepdims=True)
    with np.errstate(over="ignore"):
        t = np.exp(x - np.where(np.isfinite(top), top, 0))
    with np.errstate(invalid="ignore"):
        return t / np.maximum(t.sum(1, keepdims=True), 1e-300)


def reference(x, K, score="softmax", bias=None, groups=1, top_groups=None, renormalize=True, scale=1.0):
    """ids and weights row by row, by sorting (value, -index)."""
    T, E = x.shape
    p = scores(x, score)
    top_groups = groups if top_groups is None else top_groups
    ids, w = np.full((T, K), -1), np.zeros((T, K))
    for t in range(T):
        masked = np.isneginf(x[t]) | (False if bias is None else np.isneginf(bias))
        choice = x[t].copy() if bias is None else p[t] + bias
        if np.any(~(x[t] < math.inf)) or np.any(~(choice < math.inf)):
            continue
        choice[masked] = -math.inf
        live = ~masked
        if top_groups < groups:
            value = np.where(masked, -math.inf, p[t] + (0 if bias is None else bias))
            value = value.reshape(groups, -1)
            rank = np.sort(value, 1)[:, -2:].sum(1)
            kept = sorted(range(groups), key=lambda g: (-rank[g], g))[:top_groups]
            live &= np.isin(np.arange(E) // (E // groups), kept)
        order = sorted(np.flatnonzero(live), key=lambda e: (-choice[e], e))[:K]
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[t][order]
        if renormalize and len(order):
            # from the logarithms of p, which do not underflow (softmax: up to their common part)
            v = x[t][order]
            if score == "sigmoid":
                v = np.minimum(v, 0) - np.log1p(np.exp(-np.abs(v)))
            w[t, :len(order)] = np.exp(v - v.max())
            w[t] /= w[t].sum()
    return ids, w * scale


def check(logits, K, bias=None, **kw):
    ids, w = api.nvfp4_moe_router(logits, K, bias=bias, **kw)
    b = None if bias is None else bias.cpu().double().numpy()
    want, ww = reference(logits.cpu().double().numpy(), K, bias=b, **kw)
    assert np.array_equal(ids.cpu().numpy(), want)
    got = w.cpu().double().numpy()
    assert np.all(np.abs(got - ww) <= EXP_TOL * np.abs(ww) + 1e-30)
    return ids, w


CASES = [  # T, E, K, groups, top_groups
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 5, 5, 1, 1), (7, 64, 8, 1, 1), (33, 60, 6, 4, 2),
    (40, 256, 32, 1, 1), (65, 132, 8, 4, 3), (20, 256, 8, 256, 16), (20, 130, 2, 65, 3),
    (300, 128, 4, 2, 1), (29, 33, 3, 33, 7)]


@pytest.mark.parametrize("T,E,K,groups,top_groups", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router(T, E, K, groups, top_groups, score, biased, dtype):
    dev = cuda()
    g = torch.Generator().manual_seed(T * 1000 + E)
    logits = (2 * torch.randn(T, E, generator=g)).to(dtype).to(dev)
    bias = (0.1 * torch.randn(E, generator=g)).to(dev) if biased else None
    for renormalize in (True, False):
        check(logits, K, bias, score=score, groups=groups, top_groups=top_groups,
              renormalize=renormalize, scale=2.5)


def test_ties_go_to_the_lower_index():
    dev = cuda()
    x = torch.zeros(4, 200, device=dev)
    x[1, 100:] = 1.0
    x[2, ::7] = 3.0
    x[3] = torch.tensor([0.0, -0.0], device=dev).repeat(100)  # equal numbers
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.full((200,), 0.25, device=dev)):
            ids, _ = check(x, 6, bias, score=score)
            assert ids[0].tolist() == [0, 1, 2, 3, 4, 5] == ids[3].tolist()


def test_order_is_that_of_the_exact_scores():
    """Scores that binary32 cannot tell apart: logits in steps of one unit in the last place, whose
    sigmoids differ by less than 2^-26, and biases that all but cancel what separates two experts."""
    dev = cuda()
    E, T = 64, 50
    rng = np.random.Generator(np.random.PCG64(5))
    base = np.float32(3.0)
    x = np.full((T, E), base, np.float32)
    for t in range(T):
        x[t] = base + rng.permutation(E).astype(np.float32) * np.spacing(base)
    check(torch.from_numpy(x).to(dev), 8, torch.zeros(E, device=dev), score="sigmoid")
    check(torch.from_numpy(x).to(dev), 8, torch.zeros(E, device=dev), score="softmax")
    check(torch.from_numpy(x).to(dev), 8, None, score="sigmoid", groups=16, top_groups=5)
    y = rng.standard_normal((T, E)).astype(np.float32)
    b = -scores(y[:1].astype(np.float64), "sigmoid")[0]
    check(torch.from_numpy(np.repeat(y[:1], T, 0)).to(dev), 8, torch.from_numpy(b.astype(np.float32)).to(dev),
          score="sigmoid")


def test_masks():
    dev = cuda()
    g = torch.Generator().manual_seed(1)
    x = torch.randn(12, 96, generator=g)
    x[0, 3:] = -math.inf            # three experts are left for four slots
    x[1] = -math.inf                # none
    x[2, ::2] = -math.inf
    x[3, :48] = torch.finfo(torch.float32).min  # the lowest number is not a mask
    x[4] = torch.finfo(torch.float32).min
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(96, device=dev)):
            for groups in (1, 8):
                ids, w = check(x.to(dev), 4, bias, score=score, groups=groups, top_groups=groups)
                assert ids[1].tolist() == [-1] * 4 and w[1].tolist() == [0.0] * 4
                assert ids[0].tolist()[3] == -1 and (ids[4] >= 0).all()
    b = torch.zeros(96)
    b[5:90] = -math.inf
    ids, _ = check(x.to(dev), 8, b.to(dev), score="sigmoid")
    assert ((ids < 5) | (ids >= 90)).all()
    assert api.nvfp4_get_status() == (0, 0)


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_rows_without_an_order_are_dropped_and_flagged(value):
    dev = cuda()
    g = torch.Generator().manual_seed(2)
    x = torch.randn(9, 70, generator=g)
    x[4, 69] = value
    for score in ("softmax", "sigmoid"):
        ids, w = check(x.to(dev), 5, score=score)
        assert ids[4].tolist() == [-1] * 5 and w[4].tolist() == [0.0] * 5
        assert api.nvfp4_get_status()[1] == 4
        d = api.nvfp4_moe_router_backward(torch.ones_like(w), x.to(dev), ids, score=score,
                                          renormalize=False)
        assert torch.isfinite(d).all() and not d[4].any()
    assert api.nvfp4_get_status() == (0, 0)


def test_far_logits_keep_their_weights():
    """Sigmoids far below binary32's range: the renormalized weights are those of the formula."""
    dev = cuda()
    x = torch.tensor([[-200.0, -201.0, -202.5, -300.0], [-104.0, -90.0, 5.0, 80.0],
                      [1000.0, 999.0, -1000.0, 0.0], [90.0, 89.0, 88.0, 87.0]], device=dev)
    for score in ("softmax", "sigmoid"):
        check(x, 3, score=score)
        check(x, 4, score=score)


def test_no_tokens_and_preallocated_outputs():
    dev = cuda()
    ids, w = api.nvfp4_moe_router(torch.zeros(0, 16, device=dev), 2)
    assert ids.shape == w.shape == (0, 2)
    x = torch.randn(5, 16, device=dev)
    ids, w = torch.empty(5, 2, dtype=torch.int32, device=dev), torch.empty(5, 2, device=dev)
    a, b = api.nvfp4_moe_router(x, 2, ids=ids, weights=w)
    assert a is ids and b is w
    assert api.nvfp4_moe_router_backward(w[:0], x[:0], ids[:0]).shape == (0, 16)


def gradient(x, ids, gw, score, renormalize, scale):
    """By autograd in binary64."""
    x = x.double().cpu().requires_grad_()
    p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    held = (ids >= 0).cpu()
    at = ids.long().clamp_min(0).cpu()
    if renormalize and score == "softmax":
        w = torch.softmax(torch.where(held, x.gather(1, at), -math.inf), 1)
        w = torch.where(held, w, 0)
    else:
        w = torch.where(held, p.gather(1, at), 0)
        if renormalize:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    (w * scale * gw.double().cpu()).sum().backward()
    return torch.nan_to_num(x.grad, nan=0.0)


@pytest.mark.parametrize("T,E,K,groups,top_groups", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router_backward(T, E, K, groups, top_groups, score, renormalize, dtype):
    dev = cuda()
    g = torch.Generator().manual_seed(T * 1000 + E + 1)
    logits = (2 * torch.randn(T, E, generator=g)).to(dtype).to(dev)
    ids, w = api.nvfp4_moe_router(logits, K, score=score, groups=groups, top_groups=top_groups,
                                  renormalize=renormalize)
    if T > 2 and K > 1:
        ids[1, 1:] = -1
        ids[2] = -1
    gw = torch.randn(T, K, generator=g).to(dev)
    got = api.nvfp4_moe_router_backward(gw, logits, ids, score=score, renormalize=renormalize, scale=1.5)
    want = gradient(logits, ids, gw, score, renormalize, 1.5)
    assert got.dtype == dtype
    # r (g - sum r g): each factor to EXP_TOL, the difference relative to its parts; one rounding
    parts = 1.5 * gw.double().cpu().abs().amax(1, keepdim=True)
    tol = 4 * EXP_TOL * parts + (2.0 ** -8 if dtype is torch.bfloat16 else 0) * want.abs()
    assert ((got.double().cpu() - want).abs() <= tol).all()
    if T > 2 and K > 1:
        assert not got[2].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_router_backward_against_differences(score, renormalize):
    dev = cuda()
    g = torch.Generator().manual_seed(3)
    x = torch.randn(4, 24, generator=g, dtype=torch.float64)
    gw = torch.randn(4, 3, generator=g, dtype=torch.float64)
    ids, _ = api.nvfp4_moe_router(x.float().to(dev), 3, score=score)
    got = api.nvfp4_moe_router_backward(gw.float().to(dev), x.float().to(dev), ids, score=score,
                                        renormalize=renormalize, scale=2.0).double().cpu()

    def loss(y):
        w = scores(y, score)[np.arange(4)[:, None], ids.cpu().numpy()]
        w = w / w.sum(1, keepdims=True) if renormalize else w
        return (2.0 * w * gw.numpy()).sum()

    y, h = x.float().double().numpy(), 1e-5
    for t in range(4):
        for e in range(24):
            d = np.zeros_like(y)
            d[t, e] = h
            slope = (loss(y + d) - loss(y - d)) / (2 * h)
            # h^2 / 6 times a third derivative of at most about 2 |g|, and rounding 1e-15 / h
            assert abs(got[t, e] - slope) < 1e-8 + 4 * EXP_TOL * 2 * gw[t].abs().max()


def test_ids_twice_and_out_of_range():
    dev = cuda()
    x = torch.randn(3, 40, device=dev)
    ids = torch.tensor([[3, 3], [40, 7], [-5, 39]], dtype=torch.int32, device=dev)
    gw = torch.ones(3, 2, device=dev)
    got = api.nvfp4_moe_router_backward(gw, x, ids, score="sigmoid", renormalize=False).double()
    p = torch.sigmoid(x.double())
    want = torch.zeros(3, 40, dtype=torch.float64, device=dev)
    want[0, 3] = 2 * (p * (1 - p))[0, 3]
    want[1, 7] = (p * (1 - p))[1, 7]
    want[2, 39] = (p * (1 - p))[2, 39]
    assert (got - want).abs().max() < 8 * 2.0 ** -23
    assert api.nvfp4_get_status()[1] == 4


def test_feeds_the_plan_and_the_combination():
    """Router -> plan -> dispatch -> combine, and backwards to the logits, with a masked token."""
    dev = cuda()
    T, E, K, H = 37, 16, 3, 64
    g = torch.Generator().manual_seed(4)
    logits = torch.randn(T, E, generator=g).to(dev)
    logits[5] = -math.inf
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(dev)
    ids, w = api.nvfp4_moe_router(logits, K)
    plan = api.nvfp4_moe_plan(ids, E)
    assert int(plan["offsets"][-1]) == (T - 1) * K
    packed, _ = api.nvfp4_moe_dispatch(x, plan)
    out = api.nvfp4_moe_combine(packed, w, plan)
    # the weights of a token sum to 1 and its experts return its row: K roundings of products, one of the sum
    want = x.double()
    want[5] = 0
    assert ((out.double() - want).abs() <= (2.0 ** -8 + 16 * 2.0 ** -23) * want.abs()).all()
    grad = torch.randn(T, H, generator=g).to(torch.bfloat16).to(dev)
    _, gw = api.nvfp4_moe_combine_backward(grad, packed, w, plan)
    d = api.nvfp4_moe_router_backward(gw, logits, ids)
    # every expert returns the same row: the weights' gradients are equal and the logits' vanish
    bound = 8 * EXP_TOL * gw.abs().amax(1, keepdim=True) + 1e-30
    assert (d.abs() <= bound).all()
    assert api.nvfp4_get_status() == (0, 0)


def test_captured_calls_replay():
    dev = cuda()
    x = torch.randn(64, 128, device=dev)
    bias = torch.zeros(128, device=dev)
    ids, w = api.nvfp4_moe_router(x, 4, bias=bias)
    gw = torch.ones(64, 4, device=dev)
    d = api.nvfp4_moe_router_backward(gw, x, ids)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.nvfp4_moe_router(x, 4, bias=bias, ids=ids, weights=w)
        api.nvfp4_moe_router_backward(gw, x, ids, out=d)
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.normal_()
        gw.normal_()
        graph.replay()
        a, b = api.nvfp4_moe_router(x, 4, bias=bias)
        assert torch.equal(a, ids) and torch.equal(b, w)
        assert torch.equal(d, api.nvfp4_moe_router_backward(gw, x, a))
