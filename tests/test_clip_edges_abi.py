"""Refusals of the scaling entry point through the C ABI (no GPU: every call
returns before it touches the device; its pointers are never dereferenced)."""
import ctypes

import pytest

from int8_quantized_linear_i8lt_gb300 import _lib
from int8_quantized_linear_i8lt_gb300.build import build

P = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def scale(grads, dtypes, sizes, factor):
    n = len(grads)
    return _lib.i8lt_scale_grads((ctypes.c_void_p * n)(*grads), (ctypes.c_int32 * n)(*dtypes),
                                 (ctypes.c_int64 * n)(*sizes), n, factor)


@pytest.mark.parametrize("factor", [P, P + 4, P + 1196, P + 4096, P + 4104])
def test_a_scale_inside_a_tensor_is_refused(factor):
    """300 of 4 bytes from P on, 5 of 2 bytes from P + 4096 on."""
    assert scale([P, P + 4096], [2, 0], [300, 5], factor) == _lib.I8LT_ERR_INVALID_ARG


@pytest.mark.parametrize("factor", [P - 4, P + 1200, P + 4092, P + 4108])
def test_a_scale_beside_a_tensor_is_taken(factor):
    """As far as the device check, which fails here."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the call would run")
    assert scale([P, P + 4096], [2, 0], [300, 5], factor) not in (_lib.I8LT_OK, _lib.I8LT_ERR_INVALID_ARG)
