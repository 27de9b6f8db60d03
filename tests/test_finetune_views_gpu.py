"""The fine-tuning operators through autograd: batches without tokens, views
at any offset, changes in place, and what has no gradient."""
import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _normal(*shape, seed=0, dt=BF16, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dt)


class Base(torch.nn.Module):
    def __init__(self, K, N, dt):
        super().__init__()
        self.in_features, self.out_features = K, N
        self.W = _normal(K, N, seed=5, dt=dt, std=K ** -0.5)

    def forward(self, x):
        return x @ self.W


def _layer(K, N, r, E, dt=BF16):
    ad = I.LowRankAdapters(Base(K, N, dt), r, E, device=DEV, dtype=dt)
    with torch.no_grad():
        ad.A.copy_(_normal(E, r, K, seed=6, dt=dt, std=K ** -0.5))
        ad.B.copy_(_normal(E, N, r, seed=7, dt=dt, std=0.3))
    return ad


@pytest.mark.parametrize("shape", [(0,), (2, 0), (0, 3)])
def test_a_batch_without_tokens(shape):
    ad = _layer(48, 40, 8, 3)
    x = torch.empty(*shape, 48, dtype=BF16, device=DEV, requires_grad=True)
    for plan in (None, I.adapter_plan(torch.empty(0, dtype=torch.int32, device=DEV), 3)):
        x.grad = ad.A.grad = ad.B.grad = None
        y = ad(x, plan)
        assert y.shape == (*shape, 40)
        y.backward(torch.empty_like(y))
        assert x.grad.shape == x.shape
        assert ad.A.grad.shape == ad.A.shape and not ad.A.grad.any()
        assert ad.B.grad.shape == ad.B.shape and not ad.B.grad.any()
    norm = I.LayerNorm(48, device=DEV)
    norm(x).backward(torch.empty_like(x))
    assert norm.weight.grad.shape == (48,) and not norm.weight.grad.any() and not norm.bias.grad.any()
