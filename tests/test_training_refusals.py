"""The router, the matrix products and AdamW without a GPU: argument checks come before any CUDA call,
and the binding refuses tensors of the wrong type, shape or place before it calls the library."""
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


def test_struct_layouts():
    assert ctypes.sizeof(_lib.Operand) == 56 and ctypes.sizeof(_lib.Epilogue) == 48
    assert ctypes.sizeof(_lib.AdamWTensor) == 72 and ctypes.sizeof(_lib.AdamWConfig) == 72


def test_router(L):
    def router(T=4, E=16, K=2, width=4, score=0, groups=1, top=1, renorm=1, scale=1.0, x=FAKE, bias=0,
               ids=FAKE, w=FAKE):
        return L.nvfp4_moe_router(p(x), width, p(bias), T, E, K, score, groups, top, renorm, scale,
                                  p(ids), p(w), None)
    for kw in (dict(T=-1), dict(E=0), dict(E=257), dict(K=0), dict(K=17), dict(width=8), dict(score=2),
               dict(groups=0), dict(groups=17), dict(top=0), dict(groups=2, top=3), dict(renorm=2),
               dict(scale=float("nan")), dict(x=0), dict(ids=0), dict(w=0)):
        assert router(**kw) == INVALID, kw
    assert router(E=64, K=33) == UNSUPPORTED
    assert router(E=15, groups=2) == SHAPE and router(E=16, groups=8, top=1, K=3) == SHAPE
    assert router(T=1 << 40) == SHAPE
    assert router(x=FAKE + 2) == ALIGN and router(x=FAKE + 1, width=2) == ALIGN
    assert router(bias=FAKE + 2) == ALIGN and router(ids=FAKE + 1) == ALIGN and router(w=FAKE + 2) == ALIGN
    assert router(T=0, x=0, ids=0, w=0) == OK

    def back(T=4, E=16, K=2, width=4, g=FAKE, x=FAKE, ids=FAKE, out=FAKE):
        return L.nvfp4_moe_router_backward(p(g), p(x), width, p(ids), T, E, K, 0, 1, 1.0, p(out), None)
    for k in ("g", "x", "ids", "out"):
        assert back(**{k: 0}) == INVALID and back(**{k: FAKE + 2}) == ALIGN, k
    assert back(E=300) == INVALID and back(width=1) == INVALID and back(T=0, g=0) == OK


def operand(codes=FAKE, scales=FAKE, gs=FAKE, pitch=None, spitch=None, batch=0, sbatch=0, K=64):
    return _lib.Operand(codes or None, scales or None, gs or None, K // 2 if pitch is None else pitch,
                        K // 16 if spitch is None else spitch, batch, sbatch)


def epilogue(**kw):
    e = _lib.Epilogue(0, 2, 0, None, None, None, None)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def test_gemm(L):
    def gemm(M=8, N=16, K=64, a=None, b=None, e=None, out=FAKE, ws=0, size=0):
        a = operand(K=K) if a is None else a
        b = operand(K=K) if b is None else b
        e = epilogue() if e is None else e
        return L.nvfp4_gemm(ctypes.byref(a), ctypes.byref(b), M, N, K, ctypes.byref(e), p(out), p(ws), size, None)
    assert gemm(M=-1) == INVALID and gemm(K=48) == SHAPE and gemm(M=2 ** 31) == SHAPE
    assert gemm(out=0) == INVALID and gemm(out=FAKE + 1) == ALIGN
    for bad in (operand(codes=0), operand(scales=0), operand(gs=0)):
        assert gemm(a=bad) == INVALID and gemm(b=bad) == INVALID
    assert gemm(a=operand(codes=FAKE + 8)) == ALIGN and gemm(b=operand(gs=FAKE + 2)) == ALIGN
    assert gemm(a=operand(pitch=40)) == ALIGN and gemm(b=operand(pitch=16)) == SHAPE
    assert gemm(b=operand(spitch=3)) == SHAPE and gemm(a=operand(pitch=-32)) == SHAPE
    for e, want in ((epilogue(activation=5), INVALID), (epilogue(activation=-1), INVALID),
                    (epilogue(out_bytes=8), INVALID), (epilogue(bias=FAKE), INVALID),
                    (epilogue(bias=FAKE + 1, bias_bytes=2), ALIGN),
                    (epilogue(bias=FAKE + 2, bias_bytes=4), ALIGN), (epilogue(residual=FAKE + 1), ALIGN),
                    (epilogue(out_bytes=4, residual=FAKE + 2), ALIGN), (epilogue(preact=FAKE + 1), ALIGN),
                    (epilogue(amax=FAKE + 2), ALIGN)):
        assert gemm(e=e) == want
    assert gemm(out=FAKE + 2, e=epilogue(out_bytes=4)) == ALIGN
    assert gemm(size=16) == INVALID and gemm(ws=FAKE + 8, size=64) == ALIGN
    n, loose = ctypes.c_size_t(), operand(scales=FAKE + 1)
    ask = lambda a, b, E=1: L.nvfp4_gemm_workspace(ctypes.byref(a), ctypes.byref(b), 8, 16, 64, E,  # noqa: E731
                                                   ctypes.byref(n))
    wide = operand(spitch=16)
    assert ask(wide, wide) == OK and n.value == 0
    assert ask(loose, wide) == OK and n.value == 8 * 16
    assert ask(operand(), operand()) == OK and n.value == (8 + 16) * 16
    assert ask(wide, operand(batch=512, sbatch=64), 3) == OK and n.value == 16 * 16 * 3
    assert ask(wide, wide, 0) == INVALID and ask(wide, operand(pitch=16)) == SHAPE
    a, e = operand(), epilogue()
    assert L.nvfp4_gemm(None, ctypes.byref(a), 8, 16, 64, ctypes.byref(e), p(FAKE), None, 0, None) == INVALID
    assert L.nvfp4_gemm(ctypes.byref(a), ctypes.byref(a), 8, 16, 64, None, p(FAKE), None, 0, None) == INVALID


def test_grouped(L):
    def grouped(T=8, N=16, K=64, E=2, a=None, b=None, offsets=FAKE, out=FAKE, ws=0, size=0):
        a = operand(K=K) if a is None else a
        b = operand(K=K, batch=16 * 32, sbatch=64) if b is None else b
        e = epilogue()
        return L.nvfp4_gemm_grouped(ctypes.byref(a), ctypes.byref(b), p(offsets), E, T, N, K,
                                    ctypes.byref(e), p(out), p(ws), size, None)
    assert grouped(E=0) == INVALID and grouped(E=257) == INVALID and grouped(offsets=0) == INVALID
    assert grouped(offsets=FAKE + 2) == ALIGN and grouped(K=16) == SHAPE and grouped(out=0) == INVALID
    assert grouped(b=operand()) == SHAPE and grouped(b=operand(batch=520, sbatch=64)) == ALIGN

    def wgrad(M=8, N=16, cap=64, E=2, width=4, acc=0, offsets=FAKE, out=FAKE, ws=0, size=0):
        a = operand(K=cap)
        return L.nvfp4_gemm_grouped_wgrad(ctypes.byref(a), ctypes.byref(a), p(offsets), E, M, N, cap,
                                          width, acc, p(out), p(ws), size, None)
    assert wgrad(cap=80) == SHAPE and wgrad(width=1) == INVALID and wgrad(acc=2) == INVALID
    assert grouped(ws=FAKE + 4, size=64) == ALIGN and wgrad(ws=FAKE + 4, size=64) == ALIGN
    assert wgrad(offsets=0) == INVALID and wgrad(out=0) == INVALID and wgrad(out=FAKE + 2) == ALIGN
    assert wgrad(E=300) == INVALID and wgrad(M=0, out=0) == OK


def test_epilogue_backward(L):
    n = ctypes.c_size_t()
    assert L.nvfp4_gemm_epilogue_backward_workspace(3, 16, ctypes.byref(n)) == OK and n.value == 0
    assert L.nvfp4_gemm_epilogue_backward_workspace(33, 16, ctypes.byref(n)) == OK and n.value == 33 * 64
    assert L.nvfp4_gemm_epilogue_backward_workspace(3, 2 ** 31, ctypes.byref(n)) == SHAPE
    assert L.nvfp4_gemm_epilogue_backward_workspace(3, 16, None) == INVALID

    def back(M=33, N=16, act=3, g=FAKE, z=FAKE, out=FAKE, db=FAKE, amax=FAKE, ws=FAKE, size=1 << 20):
        return L.nvfp4_gemm_epilogue_backward(p(g), p(z), M, N, act, p(out), p(db), p(amax), p(ws), size,
                                              None)
    assert back(N=2 ** 31) == SHAPE and back(M=-1) == INVALID and back(act=5) == INVALID
    for k in ("g", "z", "out", "ws"):
        assert back(**{k: 0}) == INVALID and back(**{k: FAKE + 8}) == ALIGN, k
    assert back(size=33 * 64 - 1) == INVALID
    assert back(db=FAKE + 2) == ALIGN and back(amax=FAKE + 2) == ALIGN


def test_adamw(L):
    def step(n=8, count=1, param=FAKE, grad=FAKE, m=FAKE, v=FAKE, ms=FAKE, vs=FAKE, w=FAKE, decay=0.1,
             amax=FAKE, table=True, **kw):
        t = (_lib.AdamWTensor * 2)()
        for i in range(2):
            t[i] = _lib.AdamWTensor(n, param or None, grad or None, m or None, v or None, ms or None,
                                    vs or None, w or None, decay)
        c = _lib.AdamWConfig(1e-3, 0.9, 0.95, 1e-8, 1, None, None, 0, 8, 4)
        for k, x in kw.items():
            setattr(c, k, x)
        return L.nvfp4_adamw_step(t if table else None, count, ctypes.byref(c), p(amax), None)
    for kw in (dict(count=-1), dict(table=False), dict(n=-1), dict(param=0), dict(grad=0), dict(m=0),
               dict(v=0), dict(ms=0), dict(vs=0), dict(decay=float("inf")), dict(state_bits=16),
               dict(grad_bytes=1), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(eps=1e-60),
               dict(lr=float("nan")), dict(step=0), dict(step=1 << 31)):
        assert step(**kw) == INVALID, kw
    for k in ("param", "grad", "m", "v", "w"):
        assert step(**{k: FAKE + 8}) == ALIGN, k
    assert step(amax=FAKE + 2) == ALIGN and step(step_device=FAKE + 2) == ALIGN
    assert step(n=(1 << 48) + 1) == SHAPE
    assert step(count=0) == OK
    assert L.nvfp4_adamw_step(None, 0, None, None, None) == INVALID


def test_binding_refuses_host_tensors_and_wrong_types():
    f, b, u = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.uint8)
    gs = torch.zeros(2)
    for call in (lambda: api.nvfp4_moe_router(f, 2), lambda: api.nvfp4_moe_router(f.double(), 2),
                 lambda: api.nvfp4_moe_router(f[0], 2),
                 lambda: api.nvfp4_moe_router_backward(f, f, f.int()),
                 lambda: api.nvfp4_gemm(u, u, gs, u, u, gs), lambda: api.nvfp4_gemm(None, u, gs, u, u, gs),
                 lambda: api.nvfp4_gemm_grouped(u, u, gs, u, u, gs, f.int()),
                 lambda: api.nvfp4_gemm_grouped_wgrad(u, u, gs, u, u, gs, f.int()),
                 lambda: api.nvfp4_gemm_epilogue_backward(b, b, "gelu"),
                 lambda: api.AdamW([f], [f]), lambda: api.AdamW([1], [f])):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: api.AdamW([], []), lambda: api.AdamW([f], []),
                 lambda: api.AdamW([f], [f], state_bits=16)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("name", ["tanh", "GELU", 3])
def test_unknown_names(name):
    with pytest.raises(ValueError):
        api._activation(name)
    with pytest.raises(ValueError):
        api._score(name)
