"""The fine-tuning operators together: the example's training and serving, and
a whole step inside a CUDA graph."""
import importlib.util
import os

import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("finetune_adapters",
                                                  os.path.join(ROOT, "examples", "finetune_adapters.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_trains_and_serves(example):
    losses, off = example.main(["--steps", "40", "--tokens", "600", "--features", "512"])
    for run in losses:
        assert run[-1] < 0.5 * run[0]
    # both are bf16 results of the same sums in another order: two roundings of 2^-8 apart at most
    assert off < 2.0 ** -7


@pytest.mark.parametrize("base", ["int8", "nf4"])
def test_modules_beside_the_frozen_layers(base):
    """LowRankAdapters over the framework's layers: the base layer's output
    plus the adapters', and both input gradients."""
    M, K, N = 300, 512, 640
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    W = (torch.randn(N, K, generator=g, device=DEV) * 0.05).bfloat16()
    layer = I.Linear8bitLt.from_float(W) if base == "int8" else I.LinearNF4.from_float(W)
    ad = I.LowRankAdapters(layer, 8, 3, scale=0.5, device=DEV)
    with torch.no_grad():
        ad.B.copy_(torch.randn(3, N, 8, generator=g, device=DEV) * 0.3)
    index = torch.randint(-1, 3, (M,), generator=g, device=DEV).int()
    x = torch.randn(2, M // 2, K, generator=g, device=DEV).bfloat16().requires_grad_(True)
    gy = torch.randn(2, M // 2, N, generator=g, device=DEV).bfloat16()
    y = ad(x, I.adapter_plan(index, 3))
    y.backward(gy)
    x2 = x.detach().clone().requires_grad_(True)
    yb = layer(x2)
    yb.backward(gy)
    A, B = ad.A.double(), ad.B.double()
    delta = torch.zeros(M, N, dtype=torch.double, device=DEV)
    dx = torch.zeros(M, K, dtype=torch.double, device=DEV)
    for e in range(3):
        rows = (index == e).nonzero()[:, 0]
        delta[rows] = 0.5 * x.double().reshape(M, K)[rows] @ A[e].T @ B[e].T
        dx[rows] = 0.5 * gy.double().reshape(M, N)[rows] @ B[e] @ A[e]

    def near(got, want):   # bf16 sums and roundings: a few 2^-8 of the values' size
        return float((got.double().reshape(want.shape) - want).norm() / want.norm()) < 2.0 ** -7

    assert near(y, yb.double().reshape(M, N) + delta)
    assert near(x.grad, x2.grad.double().reshape(M, K) + dx)
    assert ad.A.grad.shape == ad.A.shape and ad.B.grad.isfinite().all()


@pytest.mark.parametrize("M,E", [(48, 4), (700, 2)])
def test_a_step_replays_in_a_cuda_graph(M, E):
    K, N, r = 512, 1024, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(M)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g, device=DEV) * std).bfloat16()

    x, gy = normal(M, K), normal(M, N)
    w, b = normal(K), normal(K)
    A0, B0 = normal(E, r, K, std=0.05), normal(E, N, r, std=0.1)
    scale = torch.ones(E, device=DEV)
    index = torch.randint(-1, E, (M,), generator=g, device=DEV).int()

    def make():
        A, B = A0.clone(), B0.clone()
        n = I.adamw_state_size([A, B])
        q = [torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
        top = [torch.zeros(n // 256, device=DEV) for _ in range(2)]
        return A, B, (q[0], top[0], q[1], top[1])

    def step(A, B, state):
        h, mean, rstd = I.layer_norm(x, w, b)
        plan = I.adapter_plan(index, E)
        y, t = I.adapters_forward(h, A, B, scale, plan)
        gh, gA, gB = I.adapters_backward(gy, h, t, A, B, scale, plan)
        gx, gw, gb = I.layer_norm_backward(gh, x, mean, rstd, w)
        I.adamw_step_8bit([A, B], [gA, gB], *state, step=3, lr=1e-2)
        return y, gx, gw, gb

    def bits(ts):
        return [t.view(torch.uint8).clone() for t in ts]

    ref = make()
    want = []
    for _ in range(3):
        out = step(*ref)
        want.append(bits([*out, ref[0], ref[1], *ref[2]]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*make())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    mine = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*mine)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b_ in zip(bits([*out, mine[0], mine[1], *mine[2]]), want[k]):
            assert torch.equal(a, b_)
