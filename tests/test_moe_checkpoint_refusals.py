"""The routing and checkpoint operators without a GPU: the C ABI's argument checks come before
any CUDA call, and the binding refuses tensors of the wrong type, shape or place before it calls
the library."""
import ctypes

import pytest
import torch

from nvfp4_block_scaled_quantize_gb300 import _lib, api, build

FAKE = 0x10000  # a 16-byte-aligned address never dereferenced: argument checks come first
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 4


def p(v):
    return ctypes.c_void_p(v) if v else None


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def test_plan(L):
    def plan(T=4, K=2, E=8, width=4, ids=FAKE, rows=FAKE, slots=FAKE, offs=FAKE):
        return L.nvfp4_moe_plan(p(ids), width, T, K, E, p(rows), p(slots), p(offs), None)
    assert plan(T=-1) == INVALID and plan(K=0) == INVALID
    assert plan(E=0) == INVALID and plan(E=257) == INVALID
    assert plan(K=33) == UNSUPPORTED
    assert plan(T=2**31 // 2, K=2) == SHAPE
    assert plan(width=2) == INVALID
    assert plan(ids=0) == INVALID and plan(rows=0) == INVALID
    assert plan(slots=0) == INVALID and plan(offs=0) == INVALID
    assert plan(ids=FAKE + 4, width=8) == ALIGN and plan(ids=FAKE + 2) == ALIGN
    assert plan(offs=FAKE + 2) == ALIGN


def test_dispatch_and_combine(L):
    def dispatch(T=4, H=16, K=2, E=8, x=FAKE, rows=FAKE, offs=FAKE, out=FAKE, amax=FAKE):
        return L.nvfp4_moe_dispatch(p(x), p(rows), p(offs), T, H, K, E, p(out), p(amax), None)
    assert dispatch(H=12) == SHAPE and dispatch(T=-1) == INVALID and dispatch(K=40) == UNSUPPORTED
    assert dispatch(E=300) == INVALID
    for k in ("x", "rows", "offs", "out"):
        assert dispatch(**{k: 0}) == INVALID, k
    assert dispatch(x=FAKE + 8) == ALIGN and dispatch(out=FAKE + 2) == ALIGN
    assert dispatch(amax=FAKE + 2) == ALIGN and dispatch(rows=FAKE + 1) == ALIGN

    def back(T=4, H=16, K=2, g=FAKE, rows=FAKE, out=FAKE):
        return L.nvfp4_moe_dispatch_backward(p(g), p(rows), T, H, K, p(out), None)
    assert back(H=4) == SHAPE and back(g=0) == INVALID and back(out=FAKE + 4) == ALIGN
    assert back(T=0, g=0, rows=0, out=0) == OK and back(H=0) == OK

    def combine(T=4, H=16, K=2, y=FAKE, w=FAKE, rows=FAKE, out=FAKE):
        return L.nvfp4_moe_combine(p(y), p(w), p(rows), T, H, K, p(out), None)
    assert combine(w=0) == INVALID and combine(w=FAKE + 2) == ALIGN and combine(y=FAKE + 8) == ALIGN
    assert combine(H=20) == SHAPE and combine(K=0) == INVALID and combine(T=0) == OK

    def combine_back(T=4, H=16, K=2, E=8, g=FAKE, y=FAKE, w=FAKE, rows=FAKE, offs=FAKE, gy=FAKE,
                     gw=FAKE):
        return L.nvfp4_moe_combine_backward(p(g), p(y), p(w), p(rows), p(offs), T, H, K, E, p(gy),
                                            p(gw), None)
    for k in ("g", "y", "w", "rows", "offs", "gy", "gw"):
        assert combine_back(**{k: 0}) == INVALID, k
    assert combine_back(gy=FAKE + 8) == ALIGN and combine_back(gw=FAKE + 1) == ALIGN
    assert combine_back(E=0) == INVALID and combine_back(H=9) == SHAPE and combine_back(T=0) == OK


def test_swiglu(L):
    def fwd(M=4, F=32, offs=FAKE, E=2, h=FAKE, y=FAKE, c=FAKE, s=FAKE, amax=FAKE):
        return L.nvfp4_swiglu_checkpoint(p(h), M, F, p(offs), E, p(y), p(c), p(s), p(amax), None)
    assert fwd(F=16) == SHAPE and fwd(M=-1) == INVALID and fwd(M=2**31) == SHAPE
    assert fwd(offs=0, E=2) == INVALID and fwd(E=0) == INVALID and fwd(E=257) == INVALID
    assert fwd(offs=FAKE + 2) == ALIGN and fwd(h=FAKE + 8) == ALIGN and fwd(c=FAKE + 8) == ALIGN
    for k in ("h", "y", "c", "s"):
        assert fwd(**{k: 0}) == INVALID, k

    def bwd(M=4, F=32, offs=FAKE, E=2, g=FAKE, c=FAKE, s=FAKE, out=FAKE):
        return L.nvfp4_swiglu_checkpoint_backward(p(g), p(c), p(s), M, F, p(offs), E, p(out), None)
    assert bwd(F=48) == SHAPE and bwd(offs=0, E=3) == INVALID and bwd(out=FAKE + 2) == ALIGN
    assert bwd(M=0) == OK and bwd(F=0) == OK
    for k in ("g", "c", "s", "out"):
        assert bwd(**{k: 0}) == INVALID, k


def test_rmsnorm(L):
    nan = float("nan")

    def fwd(M=4, N=32, eps=1e-6, bias=0.0, x=FAKE, w=FAKE, y=FAKE, c=FAKE, s=FAKE, r=FAKE, a=FAKE):
        return L.nvfp4_rmsnorm_checkpoint(p(x), p(w), M, N, eps, bias, p(y), p(c), p(s), p(r),
                                          p(a), None)
    assert fwd(N=48) == SHAPE and fwd(M=-1) == INVALID and fwd(N=32768 + 32) == UNSUPPORTED
    assert fwd(eps=nan) == INVALID and fwd(bias=float("inf")) == INVALID
    for k in ("x", "w", "y", "c", "s", "r", "a"):
        assert fwd(**{k: 0}) == INVALID, k
    assert fwd(x=FAKE + 8) == ALIGN and fwd(r=FAKE + 2) == ALIGN and fwd(a=FAKE + 2) == ALIGN

    n = ctypes.c_size_t(7)
    size = lambda M, N: L.nvfp4_rmsnorm_checkpoint_workspace(M, N, ctypes.byref(n))
    assert size(3, 64) == OK and n.value == 3 * 64 * 4
    assert size(10**6, 64) == OK and n.value % (64 * 4) == 0 and n.value < 10**6
    assert size(4, 40) == SHAPE and size(-1, 32) == INVALID and size(4, 65536) == UNSUPPORTED
    assert L.nvfp4_rmsnorm_checkpoint_workspace(4, 32, None) == INVALID

    def bwd(M=4, N=32, bias=0.0, g=FAKE, c=FAKE, s=FAKE, r=FAKE, w=FAKE, res=0, gx=FAKE, gw=FAKE,
            ws=FAKE, n=4 * 32 * 4):
        return L.nvfp4_rmsnorm_checkpoint_backward(p(g), p(c), p(s), p(r), p(w), M, N, bias,
                                                   p(res), p(gx), p(gw), p(ws), n, None)
    assert bwd(N=16) == SHAPE and bwd(bias=nan) == INVALID and bwd(n=4 * 32 * 4 - 1) == INVALID
    for k in ("g", "c", "s", "r", "w", "gx", "gw", "ws"):
        assert bwd(**{k: 0}) == INVALID, k
    assert bwd(res=FAKE + 8) == ALIGN and bwd(ws=FAKE + 4) == ALIGN and bwd(gw=FAKE + 4) == ALIGN


def test_binding_refuses_before_it_calls_the_library():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    plan = {"row_of_slot": torch.zeros(4, 2, dtype=torch.int32),
            "offsets": torch.zeros(8, dtype=torch.int32)}
    with pytest.raises(TypeError):
        api.nvfp4_moe_plan(torch.zeros(4, 2), 8)                           # float ids
    with pytest.raises(TypeError):
        api.nvfp4_moe_plan(torch.zeros(8, dtype=torch.int32), 8)           # 1-D
    with pytest.raises(TypeError):
        api.nvfp4_moe_plan(torch.zeros(4, 2, dtype=torch.int64), 8)        # host
    for call in (lambda: api.nvfp4_moe_dispatch(x, plan),
                 lambda: api.nvfp4_moe_dispatch_backward(x, plan),
                 lambda: api.nvfp4_moe_combine(x, torch.ones(4, 2), plan),
                 lambda: api.nvfp4_moe_combine_backward(x, x, torch.ones(4, 2), plan),
                 lambda: api.nvfp4_swiglu_checkpoint(x),
                 lambda: api.nvfp4_swiglu_checkpoint_backward(x, x, x),
                 lambda: api.nvfp4_rmsnorm_checkpoint(x, x[0]),
                 lambda: api.nvfp4_rmsnorm_checkpoint_backward(x, x, x, x, x)):
        with pytest.raises(TypeError):
            call()                                                         # host tensors
    cpu = torch.device("cpu")
    api._check(x, "x", torch.bfloat16, (4, 64), cpu)
    with pytest.raises(TypeError):
        api._check(x, "x", torch.float32, (4, 64), cpu)
    with pytest.raises(ValueError):
        api._check(x, "x", torch.bfloat16, (4, 32), cpu)
    with pytest.raises(ValueError):
        api._check(x[:, ::2], "x", torch.bfloat16, (4, 32), cpu)
    with pytest.raises(ValueError):
        api._check(x, "x", torch.bfloat16, (4, 64), torch.device("cuda"))
    with pytest.raises(ValueError):
        api._plan_offsets(dict(plan, offsets=torch.zeros(2, 4, dtype=torch.int32)), cpu)
    with pytest.raises(ValueError):
        api._plan_rows(dict(plan, row_of_slot=torch.zeros(8, dtype=torch.int32)), cpu)
    assert api.nvfp4_rmsnorm_checkpoint_workspace(2, 96) == 2 * 96 * 4
