"""The largest number of experts, through the C ABI (no GPU: every call returns
before it touches the device; its pointers are never dereferenced)."""
import pytest

from int8_quantized_linear_i8lt_gb300 import _lib
from int8_quantized_linear_i8lt_gb300.build import build

P, BIG = 1 << 20, 1 << 40
MOST = _lib.I8LT_FP8_MAX_EXPERTS


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def calls(E):
    yield _lib.i8lt_fp8_quantize_weight(P, 0, E, 4, 8, P, P)
    yield _lib.i8lt_fp8_dequantize_weight(P, P, E, 4, 8, P, 0)
    yield _lib.i8lt_fp8_experts_forward(P, 0, 4, P, P, E, 8, 16, P, 1, P, P, BIG)
    yield _lib.i8lt_fp8_experts_backward_input(P, 0, 4, P, P, E, 8, 16, P, 1, P, P, BIG)
    yield _lib.i8lt_debug_fp8_wait_timeout(1, 0, 0, P, 0, 4, P, P, E, 8, 16, P, 1, P, P, BIG)


def test_one_expert_too_many():
    assert MOST == 512
    assert set(calls(MOST + 1)) == {_lib.I8LT_ERR_INVALID_ARG}


def test_as_many_as_there_may_be():
    """As far as the device check, which fails here."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the calls would run")
    assert not set(calls(MOST)) & {_lib.I8LT_OK, _lib.I8LT_ERR_INVALID_ARG}
