"""The failure path of the FP8 products: waits that run out, made on purpose by
thread blocks that wait, for a short time, for operands that nothing fetches."""
import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300 import _lib

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
LIMIT = 20_000_000   # ns


# tokens, reduction, outputs, stages that come, whether some tiles are done by then
CASES = [
    (5, 8192, 130, 0, False),        # few tokens, a tile shared by a cluster
    (40, 2048, 39200, 20, True),     # few tokens, several tiles a thread block
    (16, 1024, 39201, 10, True),     # the same with rows on no 16 bytes
    (100, 8192, 600, 0, False),      # small products, a tile shared by a cluster
    (128, 16384, 333, 6, False),
    (2600, 1024, 1000, 0, False),    # many tokens
    (5000, 640, 4096, 12, True),
    (5000, 640, 4095, 12, True),
]


def call(t, q, s, K, transposed, E, off, rest, out, fetches):
    M, N = t.shape[0], q.shape[-2]
    ws = torch.full((_lib.i8lt_fp8_workspace_size(M, N if transposed else K),), 255, dtype=torch.uint8, device="cuda")
    assert _lib.i8lt_debug_fp8_wait_timeout(
        LIMIT, fetches, int(transposed), t.data_ptr(), I.functional.DTYPE_CODE[t.dtype], M, q.data_ptr(), s.data_ptr(), E, N, K,
        None if off is None else off.data_ptr(), rest, out.data_ptr(), ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream) == _lib.I8LT_OK
    torch.cuda.synchronize()
    return ws


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,C,R,fetches,some", CASES)
def test_outputs_that_do_not_come_are_nan(M, C, R, fetches, some, transposed):
    N, K = (C, R) if transposed else (R, C)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, s = I.fp8_quantize_weight(torch.randn(N, K, generator=g, device="cuda"))
    t = torch.randn(M, C, generator=g, device="cuda").to(F16 if R % 2 else BF16)
    expect = I.fp8_backward_input(t, q, s, K)[0] if transposed else I.fp8_forward(t, q, s, K)
    out = torch.full((M, R), 7.0, dtype=t.dtype, device="cuda")
    ws = call(t, q, s, K, transposed, 1, None, 0, out, fetches)
    assert I.device_status(ws)[0] == _lib.I8LT_ERR_TIMEOUT
    lost = out.isnan()
    assert bool(lost.any()) and bool(lost.all()) != some
    assert torch.equal(out[~lost], expect[~lost])
    # nothing of it stays behind
    again = I.fp8_backward_input(t, q, s, K, ws=ws)[0] if transposed else I.fp8_forward(t, q, s, K, ws=ws)
    assert I.device_status(ws)[0] == 0 and torch.equal(again, expect)
    # with time for all stages the same call gives the layer's results
    ws = call(t, q, s, K, transposed, 1, None, 0, out, 2 ** 31 - 1)
    assert I.device_status(ws)[0] == 0 and torch.equal(out, expect)


@pytest.mark.parametrize("M,cuts,fetches", [(60, [2, 30, 30, 55], 0), (3000, [100, 1100, 1100, 2900], 0)])
def test_rows_of_no_expert_stay_as_they_are(M, cuts, fetches):
    E, N, K = 3, 2000, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    q, s = I.fp8_quantize_weight(torch.randn(E, N, K, generator=g, device="cuda"))
    x = torch.randn(M, K, generator=g, device="cuda").half()
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    expect = I.fp8_experts_forward(x, q, s, K, off)
    out = torch.full((M, N), 7.0, dtype=F16, device="cuda")
    ws = call(x, q, s, K, False, E, off, 0, out, fetches)
    assert I.device_status(ws)[0] == _lib.I8LT_ERR_TIMEOUT
    inside = slice(cuts[0], cuts[-1])
    lost = out[inside].isnan()
    assert bool(lost.any()) and torch.equal(out[inside][~lost], expect[inside][~lost])
    assert bool((out[:cuts[0]] == 7).all()) and bool((out[cuts[-1]:] == 7).all())
    assert torch.equal(I.fp8_experts_forward(x, q, s, K, off), expect)


def test_refusals():
    t = torch.zeros(4, 16, device="cuda").half()
    q, s = I.fp8_quantize_weight(torch.zeros(8, 16, device="cuda"))
    ws = torch.empty(_lib.i8lt_fp8_workspace_size(4, 16), dtype=torch.uint8, device="cuda")
    for limit, fetches, out in ((0, 0, t), (2_000_000_001, 0, t), (1, -1, t), (1, 0, None)):
        assert _lib.i8lt_debug_fp8_wait_timeout(limit, fetches, 0, t.data_ptr(), 0, 4, q.data_ptr(), s.data_ptr(), 1, 8, 16, None,
                                                0, None if out is None else out.data_ptr(), ws.data_ptr(), ws.numel(),
                                                None) == _lib.I8LT_ERR_INVALID_ARG
