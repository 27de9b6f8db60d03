"""Status words and workspaces of the fine-tuning operators."""
import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300 import _lib
from int8_quantized_linear_i8lt_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


# every class of row lengths, whole and shifted, and a batch of nothing
@pytest.mark.parametrize("M,N", [(0, 64), (3, 64), (3, 200), (3, 512), (3, 515), (5, 2048), (5, 8189), (3, 12288),
                                 (3, 12291), (2, 60000), (2, 70000), (2, 70001)])
@pytest.mark.parametrize("need", [(1, 1, 1), (1, 0, 0), (0, 1, 1)])
def test_layer_norm_backward_clears_the_status(M, N, need):
    x = torch.randn(M, N, device=DEV)
    _, mean, rstd = I.layer_norm(x)
    n = _lib.i8lt_layer_norm_backward_workspace_size(M, N)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    out = [torch.empty(max(M, 1), N, device=DEV), torch.empty(N, device=DEV), torch.empty(N, device=DEV)]
    ptr = [t.data_ptr() if k else None for t, k in zip(out, need)]
    assert _lib.i8lt_layer_norm_backward(x.data_ptr(), x.data_ptr(), 2, M, N, mean.data_ptr(), rstd.data_ptr(), None, 2,
                                         *ptr, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
    assert I.device_status(ws) == (0, 0)


def test_callers_may_give_the_workspace_and_read_its_status():
    x, w = torch.randn(300, 520, device=DEV), torch.randn(520, device=DEV)
    _, mean, rstd = I.layer_norm(x, w)
    ws = torch.full((_lib.i8lt_layer_norm_backward_workspace_size(300, 520),), 255, dtype=torch.uint8, device=DEV)
    ref = I.layer_norm_backward(x, x, mean, rstd, w)
    got = I.layer_norm_backward(x, x, mean, rstd, w, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(ref, got)) and I.device_status(ws) == (0, 0)
    for M in (0, 20, 700):
        h, A, B = (torch.randn(*s, device=DEV).half() for s in ((M, 64), (2, 8, 64), (2, 48, 8)))
        g = torch.randn(M, 48, device=DEV).half()
        plan = I.adapter_plan((torch.arange(M, device=DEV) % 3 - 1).int(), 2)
        ws = torch.full((_lib.i8lt_adapters_workspace_size(M, 64, 48, 2, 8),), 255, dtype=torch.uint8, device=DEV)
        y, t = I.adapters_forward(h, A, B, None, plan, ws=ws)
        assert I.device_status(ws) == (0, 0)
        ws.fill_(255)
        I.adapters_backward(g, h, t, A, B, None, plan, ws=ws)
        assert I.device_status(ws) == (0, 0)
        with pytest.raises(I.I8LTError):
            I.adapters_forward(h, A, B, None, plan, ws=ws[:128])
    with pytest.raises(I.I8LTError):
        I.layer_norm_backward(x, x, mean, rstd, w, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
