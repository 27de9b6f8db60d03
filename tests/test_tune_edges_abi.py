"""More argument checks of the fine-tuning entry points through the C ABI (no
GPU: every call returns before it touches the device)."""
import ctypes

import pytest

from int8_quantized_linear_i8lt_gb300 import _lib
from int8_quantized_linear_i8lt_gb300.build import build

P = 1 << 20          # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_counted(bits):
    def call(counts=P, count=2, sizes=(5, 300), state=P, lr=1e-3, pt=2):
        lists = ((ctypes.c_void_p * 2)(P, P + 4096), (ctypes.c_void_p * 2)(P, P), (ctypes.c_int64 * 2)(*sizes))
        if bits == 8:
            return _lib.i8lt_adamw_step_8bit_counted(lists[0], pt, lists[1], 2, lists[2], count, state, P, state, P,
                                                     counts, lr, 0.9, 0.99, 1e-8, 0.0)
        return _lib.i8lt_adamw_step_counted(lists[0], pt, lists[1], 2, lists[2], count, state, state, counts, lr, 0.9,
                                            0.99, 1e-8, 0.0)

    assert call(counts=None) == _lib.I8LT_ERR_INVALID_ARG and call(counts=P + 8) == _lib.I8LT_ERR_MISALIGNED
    assert call(lr=float("nan")) == _lib.I8LT_ERR_INVALID_ARG and call(pt=3) == _lib.I8LT_ERR_UNSUPPORTED_DTYPE
    assert call(state=None) == _lib.I8LT_ERR_INVALID_ARG and call(count=-1) == _lib.I8LT_ERR_INVALID_ARG
    assert call(count=0, counts=None) == _lib.I8LT_OK and call(sizes=(0, 0)) == _lib.I8LT_OK


@pytest.mark.parametrize("M,N,rows", [(32768, 64, 608), (32768, 256, 608), (16384, 1000, 1216), (16384, 2048, 608),
                                      (8192, 4096, 304), (16384, 8192, 152), (16384, 28672, 152), (1 << 20, 1 << 20, 152),
                                      (3, 4096, 3), (100, 64, 13), (0, 64, 1)])
def test_layer_norm_workspace_holds_the_sums_of_the_blocks_that_run(M, N, rows):
    """Two fp32 sums per column and block: blocks of one residency of 152 SMs."""
    size = _lib.i8lt_layer_norm_backward_workspace_size(M, N)
    assert 8 * N <= size - 256 <= 8 * N * rows + 256


def test_adapters_outputs_over_their_inputs():
    def fwd(x, y, M=4):
        return _lib.i8lt_adapters_forward(x, 0, M, 8, P, P, 2, 8, 8, P, P, P, y, P, P, 1 << 40)

    def bwd(g, x, gx, gA=P):
        return _lib.i8lt_adapters_backward(g, x, P, 0, 4, 8, P, P, 2, 8, 8, P, P, P, gx, gA, P, P, 1 << 40)

    for call in (lambda: fwd(P, P), lambda: bwd(P, P + 4096, P), lambda: bwd(P + 4096, P, P),
                 lambda: bwd(P, None, P, gA=None)):
        assert call() == _lib.I8LT_ERR_INVALID_ARG


def test_device_status_of_host_memory_is_refused():
    torch = pytest.importorskip("torch")
    import int8_quantized_linear_i8lt_gb300 as I
    with pytest.raises(I.I8LTError):
        I.device_status(torch.zeros(256, dtype=torch.uint8))
