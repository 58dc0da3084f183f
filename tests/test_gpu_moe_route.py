"""Token routing (plan, dispatch, combine and their gradients) against plain implementations in
64 bits. Integers and copies are equal; a BF16 sum may be off by half a BF16 step of itself plus
the binary32 rounding of its terms."""
import numpy as np
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


def _ids(T, K, E, drop, seed, skew=False):
    rng = np.random.default_rng(seed)
    logits = rng.gumbel(size=(T, E)) + rng.normal(0, 3 if skew else 1, E)
    if K <= E:
        ids = np.argsort(-logits, axis=1)[:, :K]
    else:
        ids = rng.integers(0, E, (T, K))
    return np.where(rng.random((T, K)) < drop, -1, ids)


def _plan_ref(ids, E):
    """row_of_slot, slot_of_row, offsets of the definition, slot by slot."""
    flat = ids.reshape(-1)
    slots = [s for e in range(E) for s in np.nonzero(flat == e)[0]]
    rows = np.full(flat.size, -1, np.int64)
    rows[slots] = np.arange(len(slots))
    offsets = np.cumsum([(flat == e).sum() for e in range(E)])
    return rows.reshape(ids.shape), np.array(slots + [-1] * (flat.size - len(slots)), np.int64), offsets


def _check_plan(plan, ids, E):
    rows, slots, offsets = _plan_ref(ids, E)
    assert np.array_equal(plan["row_of_slot"].cpu().numpy(), rows)
    assert np.array_equal(plan["slot_of_row"].cpu().numpy(), slots)
    assert np.array_equal(plan["offsets"].cpu().numpy(), offsets)


# one slot; one warp's run; a run's edge and one past it; one CTA and the cluster; odd sizes; runs
# that are sorted before they are written and runs too long for it
PLANS = [(1, 1, 1, 0.0), (1, 8, 256, 0.0), (4, 8, 8, 0.0), (33, 1, 2, 0.0), (16, 32, 5, 0.5),
         (1000, 3, 37, 0.1), (1024, 1, 256, 0.0), (1025, 4, 64, 0.0), (4096, 1, 3, 0.0),
         (4097, 1, 3, 0.02), (5003, 6, 256, 0.06), (9999, 7, 61, 0.3), (40000, 8, 64, 0.01),
         (60000, 8, 20, 0.01)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["int32", "int64"])
@pytest.mark.parametrize("T,K,E,drop", PLANS)
def test_plan(T, K, E, drop, dtype):
    dev = _cuda()
    ids = _ids(T, K, E, drop, seed=T + K, skew=T % 2 == 1)
    plan = api.nvfp4_moe_plan(torch.tensor(ids, dtype=dtype, device=dev), E)
    _check_plan(plan, ids, E)
    assert api.nvfp4_get_status() == (0, 0)


def test_plan_everything_dropped_one_expert_and_no_tokens():
    dev = _cuda()
    for ids in (np.full((100, 4), -1), np.full((3000, 4), 7), np.full((3000, 4), -5)):
        _check_plan(api.nvfp4_moe_plan(torch.tensor(ids, dtype=torch.int32, device=dev), 9), ids, 9)
    plan = api.nvfp4_moe_plan(torch.zeros(0, 4, dtype=torch.int32, device=dev), 9)
    assert plan["offsets"].tolist() == [0] * 9 and plan["row_of_slot"].shape == (0, 4)


@pytest.mark.parametrize("value", [9, 2**31 - 1, 2**40 + 3])
def test_plan_flags_and_drops_ids_past_the_experts(value):
    dev = _cuda()
    api.nvfp4_get_status()
    ids = _ids(200, 2, 9, 0.0, seed=3)
    ids[17, 1] = value
    plan = api.nvfp4_moe_plan(torch.tensor(ids, dtype=torch.int64, device=dev), 9)
    status, bits = api.nvfp4_get_status()
    assert status == 6 and bits == _lib.DEVICE_BAD_ROUTE
    ids[17, 1] = -1
    _check_plan(plan, ids, 9)
    assert api.nvfp4_get_status() == (0, 0)


# T, K, E, H, drop: single tokens, one vector a row, odd vectors, more than 128 vectors, many tokens
SIZES = [(1, 1, 1, 8, 0.0), (1, 8, 256, 7168, 0.0), (3, 32, 5, 24, 0.3), (7, 2, 4, 1032, 0.0),
         (33, 6, 37, 2056, 0.2), (700, 3, 11, 136, 0.1), (1300, 4, 64, 1040, 0.0), (50, 4, 8, 64, 1.0),
         (20, 8, 64, 7168, 0.1), (500, 1, 9, 2056, 0.1), (3700, 5, 16, 264, 0.02)]


def _setup(T, K, E, H, drop, seed=0):
    dev = _cuda()
    ids = _ids(T, K, E, drop, seed=seed + T + H)
    plan = api.nvfp4_moe_plan(torch.tensor(ids, dtype=torch.int64, device=dev), E)
    rows, slots, offsets = _plan_ref(ids, E)
    return dev, plan, rows, slots, offsets


@pytest.mark.parametrize("T,K,E,H,drop", SIZES)
def test_dispatch(T, K, E, H, drop):
    dev, plan, rows, slots, offsets = _setup(T, K, E, H, drop)
    x = workloads.normal_with_outliers(T, H, seed=H, fraction=0.01, gain=50.0)
    out = torch.full((T * K, H), float("nan"), dtype=torch.bfloat16, device=dev)
    packed, amax = api.nvfp4_moe_dispatch(x.to(dev), plan, out=out)
    assert packed is out
    ref = torch.zeros(T * K, H, dtype=torch.bfloat16)
    live = offsets[-1]
    ref[:live] = x[slots[:live] // K]
    assert torch.equal(packed.cpu(), ref)
    begin = np.concatenate([[0], offsets[:-1]])
    want = [float(ref[b:e].abs().max()) if e > b else 0.0 for b, e in zip(begin, offsets)]
    assert amax.tolist() == want
    # what the grouped quantizer makes of it does not depend on where its amax comes from
    if H % 16 == 0:
        a = api.nvfp4_quantize_grouped(packed, plan["offsets"], columnwise=False, amax_row=amax)
        b = api.nvfp4_quantize_grouped(packed, plan["offsets"], columnwise=False)
        for k in a:
            n = live if k != "row_gscale" else E
            assert torch.equal(a[k][:n], b[k][:n]), k
    assert api.nvfp4_get_status() == (0, 0)


def _sum_ref(v, w, rows):
    """(sum, sum of magnitudes) over each token's held rows, in 64 bits."""
    held = rows >= 0
    at = torch.tensor(np.where(held, rows, 0))
    t = v.double()[at] * torch.where(torch.tensor(held), w.double(), 0.0).unsqueeze(2)
    t = torch.where(torch.tensor(held).unsqueeze(2), t, 0.0)
    return t.sum(1), t.abs().sum(1)


def _near(got, ref, off):
    """got is BF16, ref in 64 bits, `off` what the unrounded value may be off by."""
    d = (got.cpu().double() - ref).abs()
    lim = UBF * (ref.abs() + off) + off + TINY
    assert bool((d <= lim).all()), float((d - lim).max())


@pytest.mark.parametrize("T,K,E,H,drop", SIZES)
def test_dispatch_backward(T, K, E, H, drop):
    dev, plan, rows, slots, offsets = _setup(T, K, E, H, drop, seed=1)
    g = workloads.normal(T * K, H, 1e-3, seed=H + 1)
    g[offsets[-1]:] = float("nan")  # rows of no slot are not read
    got = api.nvfp4_moe_dispatch_backward(g.to(dev), plan)
    ref, mag = _sum_ref(g, torch.ones(T, K), rows)
    _near(got, ref, K * U32 * mag)


@pytest.mark.parametrize("T,K,E,H,drop", SIZES)
def test_combine_and_its_gradients(T, K, E, H, drop):
    dev, plan, rows, slots, offsets = _setup(T, K, E, H, drop, seed=2)
    rng = np.random.default_rng(H)
    w = torch.tensor(rng.random((T, K)).astype(np.float32))
    w[torch.tensor(rows < 0)] = float("nan")  # weights of dropped slots do not count
    y = workloads.normal(T * K, H, 1.0, seed=H + 2)
    y[offsets[-1]:] = float("inf")
    got = api.nvfp4_moe_combine(y.to(dev), w.to(dev), plan)
    ref, mag = _sum_ref(y, w, rows)
    _near(got, ref, (K + 1) * U32 * mag)

    g = workloads.normal(T, H, 1e-2, seed=H + 3)
    gy, gw = api.nvfp4_moe_combine_backward(
        g.to(dev), y.to(dev), w.to(dev), plan,
        grad_y=torch.full((T * K, H), float("nan"), dtype=torch.bfloat16, device=dev))
    live = offsets[-1]
    ref_y = torch.zeros(T * K, H, dtype=torch.float64)
    s = slots[:live]
    ref_y[:live] = w.double().reshape(-1)[s].unsqueeze(1) * g.double()[s // K]
    _near(gy, ref_y, U32 * ref_y.abs())
    assert bool((gy[live:] == 0).all())
    prod = g.double()[s // K] * y.double()[:live]
    ref_w, mag_w = torch.zeros(T * K, dtype=torch.float64), torch.zeros(T * K, dtype=torch.float64)
    ref_w[s], mag_w[s] = prod.sum(1), prod.abs().sum(1)
    # no sum passes through more than H / 8 terms in a row and the joins of a CTA
    off = (H / 8 + 24) * U32 * mag_w
    assert bool(((gw.cpu().double().reshape(-1) - ref_w).abs() <= off).all())
    assert bool((gw.cpu()[torch.tensor(rows < 0)] == 0).all())
    assert api.nvfp4_get_status() == (0, 0)


def test_gradients_against_differences():
    """The directional derivatives of L = <g, combine(y, w)> from 64-bit differences."""
    T, K, E, H = 19, 3, 7, 72
    dev, plan, rows, slots, offsets = _setup(T, K, E, H, 0.2, seed=5)
    rng = np.random.default_rng(1)
    y, g = workloads.normal(T * K, H, 1.0, seed=4), workloads.normal(T, H, 1.0, seed=5)
    w = torch.tensor(rng.random((T, K)).astype(np.float32))
    gy, gw = api.nvfp4_moe_combine_backward(g.to(dev), y.to(dev), w.to(dev), plan)
    dx = api.nvfp4_moe_dispatch_backward(gy, plan).cpu().double()
    L = lambda a, b: float((g.double() * _sum_ref(a, b, rows)[0]).sum())
    gy, gw, h = gy.cpu().double(), gw.cpu().double(), 2.0 ** -10
    for seed in range(4):
        rng = np.random.default_rng(seed)
        vy, vw = torch.tensor(rng.normal(size=y.shape)), torch.tensor(rng.normal(size=w.shape))
        d = (L(y.double() + h * vy, w.double()) - L(y.double() - h * vy, w.double())) / (2 * h)
        assert abs(float((gy * vy).sum()) - d) <= UBF * float((gy * vy).abs().sum()) * 1.01
        d = (L(y.double(), w.double() + h * vw) - L(y.double(), w.double() - h * vw)) / (2 * h)
        assert abs(float((gw * vw).sum()) - d) <= 1e-5 * float((gw * vw).abs().sum()) + 1e-4
        # dispatch is linear: <dispatch(v), gy> = <v, its gradient>
        vx = torch.tensor(rng.normal(size=(T, H)))
        s = slots[:offsets[-1]]
        want = float((vx[s // K] * gy[:offsets[-1]]).sum())
        mag = float((vx.abs() * (dx.abs() + K * TINY)).sum())
        assert abs(float((dx * vx).sum()) - want) <= UBF * mag * 1.01 + 1e-9


def test_rows_outside_the_packed_tensor_are_skipped_and_flagged():
    T, K, E, H = 6, 2, 3, 64
    dev, plan, rows, slots, offsets = _setup(T, K, E, H, 0.0)
    bad = dict(plan, row_of_slot=plan["row_of_slot"].clone())
    bad["row_of_slot"][2, 1] = T * K
    bad["row_of_slot"][4, 0] = 2**31 - 1
    x = workloads.normal(T, H, 1.0, seed=1)
    y = workloads.normal(T * K, H, 1.0, seed=2).to(dev)
    w = torch.ones(T, K, device=dev)
    rows = rows.copy()
    rows[2, 1] = rows[4, 0] = -1
    for call in (lambda: api.nvfp4_moe_dispatch(x.to(dev), bad),
                 lambda: api.nvfp4_moe_combine(y, w, bad),
                 lambda: api.nvfp4_moe_dispatch_backward(y, bad),
                 lambda: api.nvfp4_moe_combine_backward(x.to(dev), y, w, bad)):
        api.nvfp4_get_status()
        call()
        assert api.nvfp4_get_status() == (6, _lib.DEVICE_BAD_ROUTE)
    ref, mag = _sum_ref(y.cpu(), w.cpu(), rows)
    _near(api.nvfp4_moe_combine(y, w, bad), ref, (K + 1) * U32 * mag)
    api.nvfp4_get_status()


def test_infinities_and_nan_stay_in_their_tokens():
    T, K, E, H = 40, 4, 8, 64
    dev, plan, rows, slots, offsets = _setup(T, K, E, H, 0.0, seed=9)
    y = workloads.normal(T * K, H, 1.0, seed=2)
    y[rows[3, 1], 5], y[rows[7, 2], 9] = float("inf"), float("nan")
    out = api.nvfp4_moe_combine(y.to(dev), torch.full((T, K), 0.25, device=dev), plan).cpu()
    assert out[3, 5] == float("inf") and bool(out[7, 9].isnan())
    out[3, 5] = out[7, 9] = 0
    assert bool(out.isfinite().all())
    x = workloads.normal(T, H, 1.0, seed=3)
    x[11, 0] = float("-inf")
    packed, amax = api.nvfp4_moe_dispatch(x.to(dev), plan)
    hit = set(np.searchsorted(offsets, rows[11], side="right"))
    assert {e for e, a in enumerate(amax.tolist()) if a == float("inf")} == hit


def test_empty_tokens_and_columns():
    dev = _cuda()
    plan = api.nvfp4_moe_plan(torch.zeros(0, 4, dtype=torch.int32, device=dev), 5)
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=dev)
    packed, amax = api.nvfp4_moe_dispatch(x, plan)
    assert packed.shape == (0, 64) and amax.tolist() == [0.0] * 5
    assert api.nvfp4_moe_combine(x, torch.zeros(0, 4, device=dev), plan).shape == (0, 64)
    plan = api.nvfp4_moe_plan(torch.zeros(3, 2, dtype=torch.int32, device=dev), 5)
    x = torch.zeros(3, 0, dtype=torch.bfloat16, device=dev)
    gy, gw = api.nvfp4_moe_combine_backward(x, x.new_zeros(6, 0), torch.ones(3, 2, device=dev), plan)
    assert gy.shape == (6, 0) and gw.tolist() == [[0.0, 0.0]] * 3


def test_offsets_past_32_bits():
    """A packed tensor of more than 2^31 elements: rows far in it land and are read in place."""
    T, K, E, H = 38000, 8, 16, 7168
    dev = _cuda()
    g = torch.Generator(device=dev).manual_seed(3)
    ids = torch.rand(T, E, generator=g, device=dev).topk(K, dim=1).indices
    plan = api.nvfp4_moe_plan(ids, E)
    x = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    packed, amax = api.nvfp4_moe_dispatch(x, plan)
    assert packed.numel() > 2**31
    order = plan["slot_of_row"].long()
    for a in range(0, T * K, 1 << 15):
        assert torch.equal(packed[a:a + (1 << 15)], x[order[a:a + (1 << 15)] // K])
    w = torch.full((T, K), 0.125, device=dev)
    assert torch.equal(api.nvfp4_moe_combine(packed, w, plan), x)  # eight eighths: exact
    gy, gw = api.nvfp4_moe_combine_backward(x, packed, w, plan)
    for a in range(0, T * K, 1 << 15):
        assert torch.equal(gy[a:a + (1 << 15)], x[order[a:a + (1 << 15)] // K] * 0.125)
    want = x.double().square().sum(1)
    assert bool(((gw.double() - want.unsqueeze(1)).abs() <= (H / 8 + 24) * U32 * want.unsqueeze(1)).all())


def test_graph_replay_and_other_streams():
    T, K, E, H = 64, 4, 16, 512
    dev = _cuda()
    ids = torch.tensor(_ids(T, K, E, 0.1, seed=1), device=dev)
    x = workloads.normal(T, H, 1.0, seed=1).to(dev)
    w = torch.rand(T, K, device=dev)

    def step():
        plan = api.nvfp4_moe_plan(ids, E)
        packed, amax = api.nvfp4_moe_dispatch(x, plan)
        out = api.nvfp4_moe_combine(packed, w, plan)
        gy, gw = api.nvfp4_moe_combine_backward(out, packed, w, plan)
        return [*plan.values(), packed, amax, out, gy, gw, api.nvfp4_moe_dispatch_backward(gy, plan)]

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (2, 3):
        ids.copy_(torch.tensor(_ids(T, K, E, 0.2, seed=seed), device=dev))
        x.copy_(workloads.normal(T, H, 1.0, seed=seed))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            other = step()
        torch.cuda.synchronize()
        for a, b, c in zip(held, step(), other):
            assert torch.equal(a, b) and torch.equal(b, c)


def test_binding_checks_shapes():
    T, K, E, H = 6, 2, 3, 64
    dev, plan, *_ = _setup(T, K, E, H, 0.0)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=dev)
    y = torch.zeros(T * K, H, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(T, K, device=dev)
    with pytest.raises(ValueError):
        api.nvfp4_moe_dispatch(x[1:], plan)
    with pytest.raises(ValueError):
        api.nvfp4_moe_dispatch(x, plan, out=y[1:])
    with pytest.raises(ValueError):
        api.nvfp4_moe_combine(y, w[:, :1], plan)
    with pytest.raises(TypeError):
        api.nvfp4_moe_combine(y, w.double(), plan)
    with pytest.raises(ValueError):
        api.nvfp4_moe_combine(y, w.t().contiguous().t(), plan)
    with pytest.raises(ValueError):
        api.nvfp4_moe_combine_backward(x, y[:-1], w, plan)
    with pytest.raises(ValueError):
        api.nvfp4_moe_dispatch_backward(y[:-1], plan)
    with pytest.raises(ValueError):
        api.nvfp4_moe_dispatch(x, dict(plan, row_of_slot=plan["row_of_slot"].t()))
    with pytest.raises(_lib.NVFP4Error):
        api.nvfp4_moe_plan(torch.zeros(2, 33, dtype=torch.int32, device=dev), 4)
    with pytest.raises(_lib.NVFP4Error):
        api.nvfp4_moe_dispatch(x[:, :60].contiguous(), plan)
