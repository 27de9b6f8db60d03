"""Argument checks of the fine-tuning entry points through the C ABI (no GPU:
every call returns before it touches the device; its pointers are never
dereferenced)."""
import ctypes

import pytest

from int8_quantized_linear_i8lt_gb300 import _lib
from int8_quantized_linear_i8lt_gb300.build import build

P = 1 << 20          # 256-byte aligned, never dereferenced
BIG = 1 << 40
INVALID, DTYPE, ALIGN, WS = (_lib.I8LT_ERR_INVALID_ARG, _lib.I8LT_ERR_UNSUPPORTED_DTYPE, _lib.I8LT_ERR_MISALIGNED,
                             _lib.I8LT_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def norm(**kw):
    a = dict(x=P, xt=0, M=4, N=8, w=P, b=P, wt=0, eps=1e-5, y=P, mean=P, rstd=P) | kw
    return _lib.i8lt_layer_norm_forward(*a.values())


def norm_bwd(**kw):
    a = dict(g=P, x=P, xt=0, M=4, N=8, mean=P, rstd=P, w=P, wt=0, gx=P, gw=P, gb=P, ws=P, ws_bytes=BIG) | kw
    return _lib.i8lt_layer_norm_backward(*a.values())


def test_layer_norm():
    for call in (norm, norm_bwd):
        assert call(xt=3) == DTYPE and call(wt=-1) == DTYPE
        assert call(M=-1) == INVALID and call(N=0) == INVALID and call(M=2 ** 31) == INVALID
        assert call(x=None) == INVALID and call(x=P + 8) == ALIGN and call(w=P + 2) == ALIGN
    assert norm(eps=-1.0) == INVALID and norm(eps=float("nan")) == INVALID and norm(y=None) == INVALID
    assert norm(M=0, x=None, y=None) == _lib.I8LT_OK
    assert norm_bwd(gx=None, gw=None, gb=None) == INVALID and norm_bwd(mean=None) == INVALID
    assert norm_bwd(ws=None) == WS and norm_bwd(ws=P + 16) == ALIGN and norm_bwd(gx=P + 4) == ALIGN
    need = _lib.i8lt_layer_norm_backward_workspace_size(4, 8)
    assert need > 0 and norm_bwd(ws_bytes=need - 1) == WS
    assert _lib.i8lt_layer_norm_backward_workspace_size(-1, 8) == 0


def fwd(**kw):
    a = dict(x=P, dt=0, M=4, K=8, A=P, B=P, E=2, r=8, N=8, scale=P, plan=P, base=P, y=P, t=P, ws=P, ws_bytes=BIG) | kw
    return _lib.i8lt_adapters_forward(*a.values())


def bwd(**kw):
    a = dict(g=P, x=P, t=P, dt=0, M=4, K=8, A=P, B=P, E=2, r=8, N=8, scale=P, plan=P, addend=P, gx=P, gA=P, gB=P,
             ws=P, ws_bytes=BIG) | kw
    return _lib.i8lt_adapters_backward(*a.values())


def test_adapters():
    for call in (fwd, bwd):
        assert call(dt=2) == DTYPE and call(dt=9) == DTYPE
        for bad in (dict(M=-1), dict(K=0), dict(N=0), dict(E=0), dict(r=0), dict(r=_lib.I8LT_MAX_RANK + 1),
                    dict(A=None), dict(B=None), dict(plan=None), dict(x=None)):
            assert call(**bad) == INVALID, bad
        assert call(A=P + 8) == ALIGN and call(plan=P + 16) == ALIGN and call(ws=P + 16) == ALIGN
        assert call(ws=None) == WS
        need = _lib.i8lt_adapters_workspace_size(4, 8, 8, 2, 8)
        assert need > 0 and call(ws_bytes=need - 1) == WS
    assert fwd(y=None) == INVALID and fwd(t=None) == INVALID and fwd(base=P + 2) == ALIGN
    assert bwd(gx=None, gA=None, gB=None) == INVALID and bwd(t=None) == INVALID and bwd(addend=P + 2) == ALIGN
    need = _lib.i8lt_adapter_plan_bytes(4, 2)
    assert _lib.i8lt_adapter_plan(P, 4, 2, P, need - 1) == WS
    assert _lib.i8lt_adapter_plan(P + 1, 4, 2, P, need) == ALIGN
    assert _lib.i8lt_adapter_plan(P, 4, 0, P, need) == INVALID and _lib.i8lt_adapter_plan(P, -1, 2, P, need) == INVALID
    assert _lib.i8lt_adapter_plan_bytes(4, 0) == 0


def adamw(bits, params=(P, P), grads=(P, P), sizes=(5, 300), pt=2, gt=2, state=P, step=1, lr=1e-3, b1=0.9, b2=0.99,
          eps=1e-8, wd=0.0, count=None):
    n = len(params)
    lists = ((ctypes.c_void_p * n)(*params), (ctypes.c_void_p * n)(*grads), (ctypes.c_int64 * n)(*sizes))
    count = n if count is None else count
    if bits == 8:
        return _lib.i8lt_adamw_step_8bit(lists[0], pt, lists[1], gt, lists[2], count, state, state, state, state, step,
                                         lr, b1, b2, eps, wd)
    return _lib.i8lt_adamw_step(lists[0], pt, lists[1], gt, lists[2], count, state, state, step, lr, b1, b2, eps, wd)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits):
    assert adamw(bits, pt=3) == DTYPE and adamw(bits, gt=-1) == DTYPE
    nan = float("nan")
    for bad in (dict(count=-1), dict(step=0), dict(lr=nan), dict(b1=1.0), dict(b2=-0.5), dict(b1=nan), dict(eps=-1.0),
                dict(wd=float("inf")), dict(sizes=(5, -1)), dict(params=(P, None)), dict(state=None)):
        assert adamw(bits, **bad) == INVALID, bad
    assert adamw(bits, params=(P, P + 2)) == ALIGN and adamw(bits, grads=(P + 1, P)) == ALIGN
    assert adamw(bits, state=P + 8) == ALIGN
    assert adamw(bits, count=0) == _lib.I8LT_OK and adamw(bits, sizes=(0, 0)) == _lib.I8LT_OK
