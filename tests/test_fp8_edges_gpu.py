"""The block-scaled FP8 layers on a GB300 where they are easily wrong."""
import pytest
import torch

import _fp8 as R
import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300 import _lib

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def normal(*shape, seed, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def test_layers_after_a_conversion():
    """A model's dtype is converted around its FP8 layers, which keep their results."""
    layer = I.LinearFP8.from_float(normal(200, 300, seed=1).cuda(), normal(200, seed=2, dtype=BF16).cuda())
    experts = I.ExpertsFP8.from_float(normal(2, 72, 200, seed=3).cuda())
    x = normal(20, 300, seed=4, dtype=BF16).cuda()
    off = torch.tensor([0, 9, 20], dtype=torch.int32, device="cuda")
    expect = experts(layer(x), off)
    for convert in (lambda m: m.bfloat16(), lambda m: m.half().bfloat16(), lambda m: m.to(F32).to("cuda", BF16),
                    lambda m: m.cpu().cuda()):
        model = convert(torch.nn.ModuleList([layer, experts]))
        assert torch.equal(model[1](model[0](x), off), expect)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,N", [(30, 260, 140), (300, 260, 140), (2600, 300, 140)])
def test_exact_on_whole_numbers(M, K, N, dtype):
    """Whole numbers below 8 and a 7 in every block: the codes hold them, the scales
    are 7 / 448 = 2^-6, and each output is a whole number that the output type
    holds.  So layer and gradient are exact, the layer is linear between such
    inputs, and <g, f(x + e) - f(x)> = <gx, e> to the last bit."""
    top = 2 ** (11 if dtype == F16 else 8)               # whole numbers up to here are exact
    g = torch.Generator().manual_seed(21)
    def sparse(rows, cols, rate, low, high):
        t = torch.randint(low, high + 1, (rows, cols), generator=g).double()
        return t * (torch.rand(rows, cols, generator=g) < rate)
    x, e, G, W = sparse(M, K, 0.04, -6, 6), sparse(M, K, 0.2, -1, 1), sparse(M, N, 0.04, -6, 6), sparse(N, K, 0.04, -6, 6)
    for t in (x, G, W):
        t[:, ::128] = 7                                  # every block's maximum, with or without e
    W[1:, ::128] = 0                                     # one 7 a block of 128 x 128
    W[::128, ::128] = 7
    e[:, ::128] = 0
    y, ye, gx = x @ W.T, (x + e) @ W.T, G @ W
    assert max(float(t.abs().max()) for t in (y, ye, gx)) <= top
    layer = I.LinearFP8.from_float(W.float().cuda())
    assert torch.equal(layer.codes[:, :K].cpu().double(), W * 64) and bool((layer.scales == 2.0 ** -6).all())
    xa = x.to(dtype).cuda().requires_grad_(True)
    ya = layer(xa)
    yb = layer((x + e).to(dtype).cuda())
    ya.backward(G.to(dtype).cuda())
    assert torch.equal(ya.detach().cpu().double(), y) and torch.equal(yb.detach().cpu().double(), ye)
    assert torch.equal(xa.grad.cpu().double(), gx)
    left, right = float((G * (yb - ya).detach().cpu().double()).sum()), float((xa.grad.cpu().double() * e).sum())
    assert left == right == float((G * (e @ W.T)).sum()) and abs(left) >= 16


def groups(E, M):
    """E ranges of uneven lengths, some empty, 2 rows before the first and about 7 behind the last."""
    g = torch.Generator().manual_seed(E)
    share = torch.rand(E, generator=g) * (torch.rand(E, generator=g) < 0.8)
    share[-1] = 1.0                                      # the last expert has rows
    cuts = [0] + (share.cumsum(0) / share.sum() * (M - 9)).round().int().tolist()
    return [c + 2 for c in cuts]


@pytest.mark.parametrize("E,M", [(31, 400), (32, 400), (33, 400), (63, 900), (64, 9000), (65, 300), (511, 700), (512, 700),
                                 (512, 9000), (512, 40000)])
def test_many_experts(E, M):
    """Up to the largest number of experts, around the widths of the scans over them."""
    N, K = 40, 72
    W = normal(E, N, K, seed=5, std=0.05)
    q, s = I.fp8_quantize_weight(W.cuda())
    cuts = groups(E, M)
    assert len(cuts) == E + 1 and cuts[-1] < M and cuts[-1] > cuts[-2] and cuts == sorted(cuts)
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    for transposed in (False, True):
        t = normal(M, N if transposed else K, seed=6, dtype=F16)
        call = I.fp8_experts_backward_input if transposed else I.fp8_experts_forward
        y = call(t.cuda(), q, s, K, off)
        kept = torch.full_like(y, 7.0)
        call(t.cuda(), q, s, K, off, out=kept)
        assert not y[:cuts[0]].any() and not y[cuts[-1]:].any()
        assert bool((kept[:cuts[0]] == 7).all()) and bool((kept[cuts[-1]:] == 7).all())
        assert torch.equal(kept[cuts[0]:cuts[-1]], y[cuts[0]:cuts[-1]])
        for e in range(E):
            a, b = cuts[e], cuts[e + 1]
            if a < b:
                ref, size = R.product(t[a:b], R.expand_weight(*R.weight(W[e])), transposed=transposed)
                R.check(y[a:b], ref, size, t.shape[1], f"expert {e}")


def test_one_expert_too_many_is_refused():
    E = _lib.I8LT_FP8_MAX_EXPERTS + 1
    W = torch.zeros(E, 8, 16, device="cuda")
    with pytest.raises(I.I8LTError):
        I.fp8_quantize_weight(W)
    q = torch.zeros(E, 8, 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.zeros(E, 1, 1, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    for call, C in ((I.fp8_experts_forward, 16), (I.fp8_experts_backward_input, 8)):
        with pytest.raises(I.I8LTError):
            call(torch.zeros(4, C, dtype=F16, device="cuda"), q, s, 16, off)
    assert I.fp8_experts_forward(torch.zeros(4, 16, dtype=F16, device="cuda"), q[1:], s[1:], 16, off[1:]).shape == (4, 8)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("C", [8192, 28672])
def test_long_reductions(C, transposed, dtype):
    """The longest reductions of the framework's workloads, through the kernel for
    many tokens: rows here and there against 64 bits."""
    M, R_ = 4096, 640
    N, K = (C, R_) if transposed else (R_, C)
    W = normal(N, K, seed=8, std=0.02, dtype=BF16)
    q, s = I.fp8_quantize_weight(W.cuda())
    t = normal(M, C, seed=10, dtype=dtype)
    t[:, ::1000] *= 20
    pick = torch.randperm(M, generator=torch.Generator().manual_seed(9))[:200]
    ref, size = R.product(t[pick], R.expand_weight(*R.weight(W)), transposed=transposed)
    y, gb = I.fp8_backward_input(t.cuda(), q, s, K, bias_dtype=F32) if transposed else (I.fp8_forward(t.cuda(), q, s, K), None)
    R.check(y[pick.cuda()], ref, size, C, "gx" if transposed else "y")
    if transposed:
        assert bool(((gb.cpu().double() - t.double().sum(0)).abs() <= t.double().abs().sum(0) * M * 2.0 ** -24).all())
