"""Argument checks of the FP8 and clipping entry points through the C ABI (no
GPU: every call returns before it touches the device; its pointers are never
dereferenced)."""
import ctypes

import pytest

from int8_quantized_linear_i8lt_gb300 import _lib
from int8_quantized_linear_i8lt_gb300.build import build

P = 1 << 20          # 256-byte aligned, never dereferenced
BIG = 1 << 40
OK, INVALID, DTYPE, ALIGN, WS = (_lib.I8LT_OK, _lib.I8LT_ERR_INVALID_ARG, _lib.I8LT_ERR_UNSUPPORTED_DTYPE,
                                 _lib.I8LT_ERR_MISALIGNED, _lib.I8LT_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def test_sizes():
    assert [_lib.i8lt_fp8_ld(c) for c in (0, 1, 16, 17, 11008)] == [0, 16, 16, 32, 11008]
    assert [_lib.i8lt_fp8_blocks(c) for c in (0, 1, 128, 129)] == [0, 1, 1, 2]
    assert _lib.i8lt_fp8_workspace_size(-1, 8) == 0 and _lib.i8lt_fp8_workspace_size(4, 0) == 0
    assert _lib.i8lt_fp8_workspace_size(100, 300) >= 256 + 100 * 304 + 100 * 3 * 4
    assert _lib.i8lt_fp8_grad_bias_bytes(300, 40) >= 3 * 40 * 4


def test_quantize():
    q = lambda **kw: _lib.i8lt_fp8_quantize(*(dict(x=P, xt=0, M=4, C=8, codes=P, scales=P) | kw).values())
    w = lambda **kw: _lib.i8lt_fp8_quantize_weight(*(dict(W=P, wt=0, E=2, N=4, K=8, codes=P, scales=P) | kw).values())
    d = lambda **kw: _lib.i8lt_fp8_dequantize_weight(*(dict(codes=P, scales=P, E=2, N=4, K=8, out=P, dt=0) | kw).values())
    assert q(xt=3) == w(wt=3) == d(dt=-1) == DTYPE
    assert q(M=-1) == q(C=-1) == q(x=None) == q(scales=None) == q(M=2 ** 31) == INVALID
    assert w(E=-1) == w(E=1025) == w(N=-1) == w(W=None) == w(codes=None) == w(K=2 ** 31) == INVALID
    assert d(E=-1) == d(out=None) == d(scales=None) == INVALID
    assert q(x=P + 8) == q(codes=P + 8) == w(W=P + 2) == d(codes=P + 4) == d(out=P + 2) == ALIGN
    assert q(M=0, x=None) == w(E=0, W=None) == d(N=0, out=None) == OK


def fwd(**kw):
    a = dict(x=P, xt=0, M=4, codes=P, scales=P, N=8, K=16, bias=P, bt=0, out=P, ws=P, ws_bytes=BIG) | kw
    return _lib.i8lt_fp8_forward(*a.values())


def bwd(**kw):
    a = dict(x=P, xt=0, M=4, codes=P, scales=P, N=8, K=16, out=P, gb=P, bt=0, ws=P, ws_bytes=BIG) | kw
    return _lib.i8lt_fp8_backward_input(*a.values())


def experts(call, **kw):
    a = dict(x=P, xt=0, M=4, codes=P, scales=P, E=2, N=8, K=16, offsets=P, zero_rest=1, out=P, ws=P, ws_bytes=BIG) | kw
    return call(*a.values())


def test_products():
    calls = [fwd, bwd, lambda **kw: experts(_lib.i8lt_fp8_experts_forward, **kw),
             lambda **kw: experts(_lib.i8lt_fp8_experts_backward_input, **kw)]
    for i, call in enumerate(calls):
        C = 8 if i in (1, 3) else 16
        assert call(xt=2) == DTYPE and call(xt=9) == DTYPE
        for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=2 ** 31), dict(codes=None), dict(scales=None), dict(x=None)):
            assert call(**bad) == INVALID, bad
        assert call(x=P + 8) == call(codes=P + 8) == call(out=P + 2) == call(ws=P + 16) == ALIGN
        assert call(ws=None) == WS
        need = _lib.i8lt_fp8_workspace_size(4, C) + (_lib.i8lt_fp8_grad_bias_bytes(4, 8) if i == 1 else 0)
        assert call(ws_bytes=need - 1) == WS
        if i > 1:
            assert call(offsets=None) == call(E=0) == call(E=1025) == call(out=None) == INVALID
    assert fwd(bt=5) == DTYPE and fwd(out=None) == INVALID
    assert bwd(bt=5) == DTYPE and bwd(out=None, gb=None) == INVALID


def clip(grads=(P, P + 4096), dtypes=(0, 2), sizes=(5, 300), count=None, max_norm=1.0, result=P, ws=P, ws_bytes=BIG,
         grad_scale=None, found_inf=None):
    n = len(grads)
    lists = ((ctypes.c_void_p * n)(*grads), (ctypes.c_int32 * n)(*dtypes), (ctypes.c_int64 * n)(*sizes))
    return _lib.i8lt_grad_norm(*lists, n if count is None else count, grad_scale, found_inf, max_norm, result, ws, ws_bytes)


def scale(grads=(P, P + 4096), dtypes=(0, 2), sizes=(5, 300), count=None, factor=P):
    n = len(grads)
    lists = ((ctypes.c_void_p * n)(*grads), (ctypes.c_int32 * n)(*dtypes), (ctypes.c_int64 * n)(*sizes))
    return _lib.i8lt_scale_grads(*lists, n if count is None else count, factor)


def test_gradients():
    for call in (clip, scale):
        assert call(dtypes=(0, 3)) == DTYPE
        assert call(count=-1) == call(sizes=(5, -1)) == INVALID
        assert call(grads=(P + 1, P + 4096)) == call(grads=(P, P + 4098)) == ALIGN
    assert clip(max_norm=-1.0) == clip(max_norm=float("nan")) == clip(result=None) == INVALID
    need = _lib.i8lt_grad_norm_workspace_size()
    assert clip(ws=None) == clip(ws_bytes=need - 1) == WS and clip(ws=P + 16) == clip(result=P + 2) == ALIGN
    assert scale(factor=None) == INVALID and scale(factor=P + 2) == ALIGN
    assert scale(count=0) == scale(sizes=(0, 0)) == scale(grads=(None, None)) == OK


def test_gradients_that_overlap_are_not_scaled():
    assert scale(grads=(P, P)) == INVALID
    assert scale(grads=(P, P + 8), dtypes=(0, 0)) == INVALID          # 5 elements of 2 bytes end at P + 10
    assert scale(grads=(P + 1196, P), dtypes=(0, 2)) == INVALID       # 300 of 4 bytes end at P + 1200


def test_small_operands_are_aligned_to_their_elements():
    """A scale, an offset or a bias that starts inside an element would fault on the device."""
    assert _lib.i8lt_fp8_quantize(P, 0, 4, 8, P, P + 2) == ALIGN
    assert _lib.i8lt_fp8_quantize_weight(P, 0, 2, 4, 8, P, P + 2) == ALIGN
    assert _lib.i8lt_fp8_dequantize_weight(P, P + 1, 2, 4, 8, P, 0) == ALIGN
    assert fwd(scales=P + 2) == fwd(bias=P + 1) == fwd(bias=P + 2, bt=2) == ALIGN
    assert bwd(scales=P + 1) == bwd(gb=P + 1) == bwd(gb=P + 2, bt=2) == ALIGN
    for call in (_lib.i8lt_fp8_experts_forward, _lib.i8lt_fp8_experts_backward_input):
        assert experts(call, scales=P + 2) == experts(call, offsets=P + 2) == ALIGN
    assert clip(grad_scale=P + 2) == clip(found_inf=P + 1) == ALIGN
