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
