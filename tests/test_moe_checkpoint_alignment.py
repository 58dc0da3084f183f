"""Alignment of the checkpoint and routing operators' buffers, without a GPU: their 32-byte loads and
stores fault at an address that is 16-byte but not 32-byte aligned, so the C ABI has to refuse it."""
import ctypes

import pytest

from nvfp4_block_scaled_quantize_gb300 import _lib, build

FAKE = 0x10000  # never dereferenced: every call here is refused before any CUDA call
ALIGN = 3


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def p(v):
    return ctypes.c_void_p(v)


# operator -> (call of a dict of buffers, {buffer: its alignment})
def _swiglu(L, b):
    return L.nvfp4_swiglu_checkpoint(p(b["h"]), 4, 32, p(b["offsets"]), 2, p(b["y"]),
                                     p(b["codes"]), p(b["scales"]), p(b["amax"]), None)


def _swiglu_backward(L, b):
    return L.nvfp4_swiglu_checkpoint_backward(p(b["grad_y"]), p(b["codes"]), p(b["scales"]), 4, 32,
                                              p(b["offsets"]), 2, p(b["grad_h"]), None)


def _rmsnorm(L, b):
    return L.nvfp4_rmsnorm_checkpoint(p(b["x"]), p(b["weight"]), 4, 32, 1e-6, 0.0, p(b["y"]),
                                      p(b["codes"]), p(b["scales"]), p(b["rstd"]), p(b["amax"]),
                                      None)


def _rmsnorm_backward(L, b):
    return L.nvfp4_rmsnorm_checkpoint_backward(
        p(b["grad_y"]), p(b["codes"]), p(b["scales"]), p(b["rstd"]), p(b["weight"]), 4, 32, 0.0,
        p(b["residual"]), p(b["grad_x"]), p(b["grad_weight"]), p(b["workspace"]), 4 * 32 * 4, None)


def _dispatch(L, b):
    return L.nvfp4_moe_dispatch(p(b["x"]), p(b["rows"]), p(b["offsets"]), 4, 16, 2, 8,
                                p(b["packed"]), p(b["amax"]), None)


def _combine_backward(L, b):
    return L.nvfp4_moe_combine_backward(p(b["grad"]), p(b["y"]), p(b["weights"]), p(b["rows"]),
                                        p(b["offsets"]), 4, 16, 2, 8, p(b["grad_y"]),
                                        p(b["grad_weights"]), None)


OPERATORS = {
    _swiglu: dict(h=32, y=32, codes=16, offsets=4, amax=4, scales=1),
    _swiglu_backward: dict(grad_y=32, grad_h=32, codes=16, offsets=4, scales=1),
    _rmsnorm: dict(x=32, weight=32, y=32, codes=16, rstd=4, amax=4, scales=1),
    _rmsnorm_backward: dict(grad_y=32, weight=32, residual=32, grad_x=32, codes=16, grad_weight=16,
                            workspace=16, rstd=4, scales=1),
    _dispatch: dict(x=16, packed=16, rows=4, offsets=4, amax=4),
    _combine_backward: dict(grad=16, y=16, grad_y=16, weights=4, rows=4, offsets=4, grad_weights=4),
}
CASES = [(call, name) for call, buffers in OPERATORS.items() for name, need in buffers.items()
         if need > 1]


@pytest.mark.parametrize("call,name", CASES, ids=lambda v: v if isinstance(v, str) else v.__name__)
def test_half_the_alignment_is_refused(L, call, name):
    need = OPERATORS[call][name]
    buffers = dict.fromkeys(OPERATORS[call], FAKE)
    assert call(L, dict(buffers, **{name: FAKE + need // 2})) == ALIGN


def test_the_message_does_not_name_another_alignment(L):
    text = L.nvfp4_status_string(ALIGN).decode()
    assert "align" in text and "16" not in text
