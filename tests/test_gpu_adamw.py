"""AdamW over many tensors: 32-bit states against binary64, 8-bit states bit for bit against the
definition in numpy's binary32."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import api

pytestmark = pytest.mark.gpu
f32 = np.float32


def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda")


SIZES = [1, 7, 8, 31, 32, 33, 64, 100, 2047, 2048, 2049, 5000, 12345]


def tensors(sizes, dev, grad_dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    p = [torch.randn(n, generator=g).mul_(0.02) for n in sizes]
    gr = [(torch.randn(n, generator=g) * 1e-3 * (i + 1)).to(grad_dtype) for i, n in enumerate(sizes)]
    return [t.to(dev) for t in p], [t.to(dev) for t in gr]


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("count", [1, 13, 300])
def test_steps_with_32_bit_states(grad_dtype, count):
    dev = cuda()
    sizes = (SIZES * 30)[:count]
    p, g = tensors(sizes, dev, grad_dtype)
    w = [torch.zeros_like(t, dtype=torch.bfloat16) if i % 4 else None for i, t in enumerate(p)]
    decay = [0.1 if i % 3 else 0.0 for i in range(count)]
    lr, b1, b2, eps = 1e-2, 0.9, 0.95, 1e-8
    opt = api.AdamW(p, g, weights=w, lr=lr, betas=(b1, b2), eps=eps, weight_decay=decay)
    clip = torch.tensor([0.6], device=dev)
    P = [t.double().cpu().numpy() for t in p]
    M, V = [np.zeros_like(t) for t in P], [np.zeros_like(t) for t in P]
    for step in (1, 2, 3):
        amax = opt.step(step, grad_scale=clip)
        for i in range(count):
            x = g[i].double().cpu().numpy() * float(f32(0.6))
            M[i] = b1 * M[i] + (1 - b1) * x
            V[i] = b2 * V[i] + (1 - b2) * x * x
            move = lr * (M[i] / (1 - b1 ** step)) / (np.sqrt(V[i] / (1 - b2 ** step)) + eps)
            P[i] = P[i] - lr * decay[i] * P[i] - move
            got = p[i].double().cpu().numpy()
            # some twenty roundings of 2^-24 a step; the update is at most about lr
            tol = step * (20 * 2.0 ** -23 * lr + 4 * 2.0 ** -24 * np.abs(P[i]))
            assert np.all(np.abs(got - P[i]) <= tol)
            assert np.allclose(opt.state["exp_avg"][i].cpu().double(), M[i], rtol=step * 2.0 ** -21,
                               atol=step * 2.0 ** -22 * np.abs(x).max())
            assert np.allclose(opt.state["exp_avg_sq"][i].cpu().double(), V[i], rtol=step * 2.0 ** -21,
                               atol=1e-30)
            b = p[i].to(torch.bfloat16)
            if w[i] is not None:
                assert torch.equal(w[i], b)
            assert amax[i].item() == b.abs().max().item()
        for t in g:
            t.mul_(-1.3)


def philox(counter, key):
    c = [np.asarray(x, np.uint64) for x in counter]
    k0, k1 = np.uint64(key & 0xFFFFFFFF), np.uint64(key >> 32)
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ k0, b & low, (a >> sh) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & low, (k1 + np.uint64(0xBB67AE85)) & low
    return c


def blocks(x):
    n = x.size
    return np.pad(x, (0, -n % 32)).reshape(-1, 32)


def exponents(top):
    """The smallest e >= -127 with top <= 448 * 2^e."""
    e = np.full(top.shape, -127)
    for i in np.ndindex(top.shape):
        while top[i] > 448.0 * 2.0 ** e[i]:
            e[i] += 1
    return e


def e4m3(codes):
    return torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).float().numpy()


def to_e4m3(x):
    return torch.from_numpy(x.astype(f32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def step8(p, g, m, ms, v, vs, *, lr, b1, b2, eps, decay, step, clip, seed, index):
    """One step of one tensor in binary32, operation by operation."""
    n = p.size
    old = e4m3(m) * np.repeat(np.ldexp(f32(1), ms.astype(int) - 127).astype(f32), 32)[:n]
    r = e4m3(v) * np.repeat(np.ldexp(f32(1), vs.astype(int) - 127).astype(f32), 32)[:n]
    x = g * f32(clip)
    m1 = old * f32(b1) + x * f32(1 - b1)
    v1 = (r * r) * f32(b2) + (x * x) * f32(1 - b2)
    root = np.sqrt(v1)
    move = (m1 * f32(lr / (1 - b1 ** step))) / (root * f32((1 - b2 ** step) ** -0.5) + f32(eps))
    p1 = p * (f32(1) - f32(lr) * f32(decay)) - move
    e = exponents(np.abs(blocks(m1)).max(1).astype(np.float64))
    mc = to_e4m3(np.ldexp(blocks(m1), -e[:, None])).reshape(-1)[:n]
    ms1 = (e + 127).astype(np.uint8)
    e = exponents(blocks(root).max(1).astype(np.float64))
    t = np.ldexp(blocks(root), -e[:, None]).reshape(-1)[:n]
    i = np.arange(n)
    words = philox([i // 8 & 0xFFFFFFFF, i // 8 >> 32, np.full(n, index), np.full(n, step)], seed)
    word = np.choose(i % 8 // 2, words)
    u = ((word >> (16 * (i % 2)).astype(np.uint64)) & np.uint64(0xFFFF)).astype(f32) / f32(65536)
    code_step = np.maximum(np.frexp(t)[1] - 1, -6) - 3
    q = np.floor(np.ldexp(t, -code_step) + u)
    q = np.where(t > 0, np.maximum(q, 1), 0)
    vc = to_e4m3(np.ldexp(q, code_step))
    return p1, mc, ms1, vc, (e + 127).astype(np.uint8)


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("count", [13, 150])
def test_steps_with_8_bit_states(grad_dtype, count):
    dev = cuda()
    sizes = (SIZES[::-1] * 12)[:count]
    p, g = tensors(sizes, dev, grad_dtype, seed=1)
    with torch.no_grad():
        for t in g:
            t[::5] = 0
            t[1::7] *= 1e-6
    lr, b1, b2, eps = 1e-3, 0.9, 0.999, 1e-10
    w = [torch.zeros_like(t, dtype=torch.bfloat16) for t in p]
    opt = api.AdamW(p, g, weights=w, lr=lr, betas=(b1, b2), eps=eps, weight_decay=0.05, state_bits=8)
    clip = torch.tensor([0.7], device=dev)
    keys = ("exp_avg", "exp_avg_scales", "exp_avg_sq", "exp_avg_sq_scales")
    for step in (1, 2, 7):
        before = [[p[i].cpu().numpy()] + [opt.state[k][i].cpu().numpy() for k in keys]
                  for i in range(count)]
        amax = opt.step(step, grad_scale=clip, seed=0x123456789ABCDEF)
        for i in range(count):
            x, m, ms, v, vs = before[i]
            want = step8(x, g[i].float().cpu().numpy(), m, ms, v, vs, lr=lr, b1=b1, b2=b2, eps=eps,
                         decay=0.05, step=step, clip=0.7, seed=0x123456789ABCDEF, index=i)
            for k, y in zip(keys, want[1:]):
                assert np.array_equal(opt.state[k][i].cpu().numpy() & 0x7F if k == "exp_avg" else
                                      opt.state[k][i].cpu().numpy(),
                                      y & 0x7F if k == "exp_avg" else y), (step, i, k)
            # a quotient and a product of roundings of 2^-24 in the update, the rest exact
            tol = 16 * 2.0 ** -24 * (np.abs(want[0] - x) + np.abs(want[0])) + 1e-12
            assert np.all(np.abs(p[i].cpu().numpy().astype(np.float64) - want[0]) <= tol)
            assert amax[i].item() == w[i].abs().max().item() and torch.equal(w[i], p[i].to(torch.bfloat16))


def test_averages_halfway_between_two_codes():
    """Gradients of a few bits: with a clipping factor of 3/4, 0.9 m + 0.1 g falls halfway between two
    codes in one element of two hundred, and the rounding of each operation decides."""
    dev = cuda()
    n = 32 * 4000
    g = torch.Generator().manual_seed(9)
    spread = torch.randn(n // 32, 1, generator=g).exp().expand(-1, 32).reshape(-1) * 1e-3
    grad = (torch.randn(n, generator=g) * spread).to(torch.bfloat16).to(dev)
    p = torch.randn(n, generator=g).to(dev)
    opt = api.AdamW([p], [grad], betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, lr=3e-4, state_bits=8)
    clip = torch.tensor([0.75], device=dev)
    keys = ("exp_avg", "exp_avg_scales", "exp_avg_sq", "exp_avg_sq_scales")
    for step in (40, 41, 42):
        before = [opt.state[k][0].cpu().numpy().copy() for k in keys]
        x = p.cpu().numpy().copy()
        opt.step(step, grad_scale=clip, seed=77)
        want = step8(x, grad.float().cpu().numpy(), *before, lr=3e-4, b1=0.9, b2=0.95, eps=1e-8, decay=0.1,
                     step=step, clip=0.75, seed=77, index=0)
        for k, y in zip(keys, want[1:]):
            got = opt.state[k][0].cpu().numpy()
            if k == "exp_avg":  # either zero
                got, y = np.where(got == 0x80, 0, got), np.where(y == 0x80, 0, y)
            assert np.array_equal(got, y), (step, k, int((got != y).sum()))
        grad.mul_(-1.5)


def test_the_average_of_squares_moves():
    """Constant gradients after larger ones: the kept root follows its average down, which rounding to
    nearest would not (a step is 0.05% of it, half a code 3% to 6%); and the roots are unbiased."""
    dev = cuda()
    n = 1 << 16
    p, g = torch.zeros(n, device=dev), torch.full((n,), 1e-3, device=dev)
    opt = api.AdamW([p], [g], lr=0.0, betas=(0.9, 0.999), state_bits=8)
    v = 0.0
    for step in range(1, 201):
        if step == 101:
            g.fill_(1e-4)
        opt.step(step, seed=step)
        v = 0.999 * v + 0.001 * (1e-3 if step <= 100 else 1e-4) ** 2
    s = opt.state
    root = s["exp_avg_sq"][0].view(torch.float8_e4m3fn).double() * torch.exp2(
        s["exp_avg_sq_scales"][0].double() - 127).repeat_interleave(32)
    # The mean of r^2 follows v: rounding r by d (mean 0) adds mean d^2, at most (r / 8)^2 / 4 of
    # which decays at 0.1% a step and 200 steps add up to. Their sum is below 200 * (1/8)^2 / 4 of v.
    mean = root.square().mean().item()
    assert v < mean * 1.02 and mean < v * (1 + 200 / 256)
    assert root.min() > 0


def test_shapes_state_and_captured_steps():
    dev = cuda()
    shapes = [(3, 5), (64,), (2, 3, 7), (0,), (130, 40)]
    g = torch.Generator().manual_seed(3)
    make = lambda: [torch.randn(s, generator=torch.Generator().manual_seed(i)).to(dev)  # noqa: E731
                    for i, s in enumerate(shapes)]
    grads = [torch.randn(s, generator=g).to(dev) for s in shapes]
    for bits in (32, 8):
        a, b = make(), make()
        one, two = (api.AdamW(x, grads, state_bits=bits) for x in (a, b))
        step = torch.zeros(1, dtype=torch.int32, device=dev)
        step.fill_(1)
        two.step(step, seed=5)
        one.step(1, seed=5)
        graph = torch.cuda.CUDAGraph()
        amax = torch.empty(len(shapes), device=dev)
        with torch.cuda.graph(graph):
            two.step(step, seed=5, amax=amax)
        for t in (2, 3, 4):
            step.fill_(t)
            for x in grads:
                x.mul_(-0.9)
            graph.replay()
            want = one.step(t, seed=5)
            for x, y in zip(a, b):
                # the factors of the step, computed on the device in binary32, are off by a few units;
                # what they scale is at most about lr (1e-3), and 8-bit states do not depend on them;
                # the sum of p (2^10 to 2^13 times that difference's size) and the update is rounded to
                # 2^-24 of p on either side, in every step
                tol = t * (1e-3 * 16 * 2.0 ** -23 + 2 * 2.0 ** -24 * x.abs())
                assert ((x - y).abs() <= tol).all()
            assert torch.allclose(amax, want, rtol=2.0 ** -7)
        for k in one.state:
            for x, y in zip(one.state[k], two.state[k]):
                assert torch.equal(x, y)
        again = api.AdamW(a, grads, state_bits=bits, state=one.state)
        assert all(x is y for k in one.state for x, y in zip(one.state[k], again.state[k]))


def test_guard_bands():
    """Tensors of odd sizes inside one buffer: what lies between them stays."""
    dev = cuda()
    for bits in (32, 8):
        n = 2 * 4096
        flat = {k: torch.full((n,), 7, dtype=t, device=dev) for k, t in (
            ("p", torch.float32), ("g", torch.float32), ("w", torch.bfloat16),
            ("m", torch.uint8 if bits == 8 else torch.float32),
            ("v", torch.uint8 if bits == 8 else torch.float32),
            ("ms", torch.uint8), ("vs", torch.uint8))}
        spans = [(16, 33), (64, 1), (96, 100), (256, 2051), (4096, 2048)]
        cut = lambda k: [flat[k][a:a + m] for a, m in spans]  # noqa: E731
        cut32 = lambda k: [flat[k][a:a + (m + 31) // 32] for a, m in spans]  # noqa: E731
        state = {"exp_avg": cut("m"), "exp_avg_sq": cut("v")}
        if bits == 8:
            state.update(exp_avg_scales=cut32("ms"), exp_avg_sq_scales=cut32("vs"))
        api.AdamW(cut("p"), cut("g"), weights=cut("w"), state_bits=bits, state=state).step(1)
        inside = torch.zeros(n, dtype=torch.bool)
        scales = torch.zeros(n, dtype=torch.bool)
        for a, m in spans:
            inside[a:a + m] = True
            scales[a:a + (m + 31) // 32] = True
        for k, t in flat.items():
            held = scales if k in ("ms", "vs") else inside
            if k in ("ms", "vs") and bits == 32:
                held = torch.zeros_like(inside)
            assert (t.cpu()[~held] == 7).all(), (bits, k)
        assert (flat["p"].cpu()[inside] != 7).all()
