"""The gradient norm, scaling and clipping where they are easily wrong: the ends
of fp32's range, zeros, views that share memory."""
import math

import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
# 32 squares summed in fp32 (each rounded, up to 32 additions), the rest in
# fp64: 33 half steps of the sum of squares, half of that of the norm; and the
# rounding to fp32
NORM_TOL = (33 / 2 + 1) * 2.0 ** -24


def norm64(ts):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))


@pytest.mark.parametrize("n", [3000, 1000000])
@pytest.mark.parametrize("size,c", [(3e38, 2.0 ** -16), (3e38, 2.0 ** -60), (2.0 ** -146, 2.0 ** 30), (2.0 ** -149, 2.0 ** 100)])
def test_grad_scale_at_the_ends_of_the_range(n, size, c):
    """|c| times the root is rounded once: the norm of the gradients as they are
    may leave fp32's range, above or below."""
    t = torch.full((n,), size, device="cuda")
    norm, scale, inf = I.grad_norm([t], max_norm=1.0, grad_scale=torch.tensor([c], device="cuda"))
    ref = c * norm64([t])
    assert math.isfinite(ref) and 2.0 ** -126 < ref < 3e38
    assert abs(float(norm) - ref) <= ref * NORM_TOL and float(inf) == 0
    expect = c * min(1.0, 1.0 / (ref + 1e-6))
    assert abs(float(scale) - expect) <= expect * (NORM_TOL + 2.0 ** -24) + 2.0 ** -150


def test_a_norm_beyond_the_range_after_scaling():
    t = torch.full((100000,), 3e38, device="cuda")
    norm, scale, inf = I.grad_norm([t], max_norm=1.0, grad_scale=torch.tensor([0.5], device="cuda"))
    assert float(norm) == math.inf and float(scale) == 0 and float(inf) == 1


def test_results_are_rounded_once():
    """Two numbers whose squares and their sum are exact leave only the roundings
    of the norm and of the factor, from 64 bits."""
    for a, b, limit, c in ((3.0, 1.0, 0.7, 1.0), (5.0, 2.0, 3.3, 0.3), (1.0, 1.0, 1.0, 1.0), (4095.0, 77.0, 1e-3, 7e-5)):
        t, k = torch.tensor([a, b], device="cuda"), torch.tensor([c], device="cuda")
        norm, scale, _ = I.grad_norm([t], max_norm=limit, grad_scale=k)
        ref = float(k) * math.sqrt(a * a + b * b)
        assert float(norm) == float(torch.tensor(ref, dtype=torch.float64).float())
        expect = float(k) * min(1.0, limit / (ref + 1e-6))
        assert float(scale) == float(torch.tensor(expect, dtype=torch.float64).float())


def test_scaled_views_that_share_memory_are_refused():
    """Each is scaled through a copy of its own, so one of two scalings would be lost."""
    half = torch.full((), 0.5, device="cuda")
    m = torch.ones(6, 8, device="cuda")
    flat = m.view(-1)
    for views in ([m[:, ::2], m], [m, m[:, ::2]], [m[:, ::2], m[:, ::2]], [m[:, :5], m[:, 4:]], [m[1:, ::2], flat[12:15]],
                  [m.T, m], [m.T, m.T], [m[:, 1:3], m[2:4, 2:5]], [m[:, ::3], m[:, 1::2]]):
        with pytest.raises(I.I8LTError, match="share"):
            I.scale_grads_(views, half)
        assert bool((m == 1).all())


def test_scaled_views_beside_one_another():
    half = torch.full((), 0.5, device="cuda")
    cases = (((6, 8), lambda m: [m[:, ::2], m[:, 1::2]]), ((6, 7), lambda m: [m[:, ::2], m[:, 1::2]]),
             ((6, 7), lambda m: [m[:, 4:], m[:, :2], m[:, 2:3]]), ((6, 8), lambda m: [m[::2], m[1::2, 3:], m[1::2, :2]]),
             ((6, 8), lambda m: [m[:, ::2], m.view(-1)[9:10], m.view(-1)[15:16]]),
             ((3, 5, 4), lambda m: [m[:, :2, 1:], m[:, :2, :1], m[:, 2:, ::2], m[1:, 4, 1:2]]),
             ((8, 9), lambda m: [m[:4].T, m[4:, ::2]]), ((5, 6), lambda m: [m[:0, ::2], m[:, 1:1], m[:, ::5]]))
    for shape, views in cases:
        for dtype in (F32, F16, BF16):
            m = torch.randn(shape, device="cuda").to(dtype)
            expect = m.clone()
            for v in views(expect):
                v.mul_(0.5)
            I.scale_grads_(views(m), half)
            assert torch.equal(m, expect)


def test_tensors_that_require_a_gradient_are_scaled_in_any_layout():
    half = torch.full((), 0.5, device="cuda")
    dense = torch.nn.Parameter(torch.ones(5, device="cuda"))
    loose = torch.nn.Parameter(torch.ones(4, 6, device="cuda").T)
    assert not loose.is_contiguous()
    versions = dense._version, loose._version
    I.scale_grads_([dense, loose], half)
    assert bool((dense == 0.5).all()) and bool((loose == 0.5).all()) and loose.is_leaf and loose.requires_grad
    assert dense._version > versions[0] and loose._version > versions[1]
    p = torch.nn.Parameter(torch.ones(6, 4, device="cuda"))
    p.grad = (torch.ones(4, 6, device="cuda", requires_grad=True) * 1).T     # a gradient with a history
    assert p.grad.requires_grad and not p.grad.is_contiguous()
    norm = I.clip_grad_norm_(p, 1.0)
    f = I.grad_norm([torch.ones(24, device="cuda")], 1.0)[1]
    assert abs(float(norm) - 24 ** 0.5) <= 1e-5 and bool((p.grad == f).all())


def median_time(call):
    times = []
    for _ in range(12):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda._sleep(200000)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return sorted(times[2:])[5]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_zeros_are_read_once(dtype):
    """Gradients of zeros are ordinary (unused layers, the first step of an
    adapter); reading them again, to look for squares lost below fp32's range,
    took five times as long."""
    zeros = torch.zeros(60000000, dtype=dtype, device="cuda")
    zeros[::3] = -0.0
    ones = torch.full_like(zeros, 1e-2)
    assert [float(v) for v in I.grad_norm([zeros], 1.0)] == [0, 1, 0]
    assert median_time(lambda: I.grad_norm([zeros], 1.0)) <= 1.5 * median_time(lambda: I.grad_norm([ones], 1.0))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [5, 8191, 300007])
def test_few_values_among_zeros(n, dtype):
    """Small ones, whose squares fp32 does not hold, beside zeros, in every place of a unit."""
    g = torch.Generator().manual_seed(n)
    smallest = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}[dtype]
    for value in (smallest, -smallest, 2.0 ** -24):
        for place in (0, n - 1, *torch.randint(0, n, (6,), generator=g).tolist()):
            t = torch.zeros(n, dtype=dtype, device="cuda")
            t[place] = value
            assert float(I.grad_norm([t])[0]) == abs(value)
    rows = torch.zeros(n, 40, dtype=dtype, device="cuda")
    rows[::7] = torch.randn(rows[::7].shape, generator=g).to(dtype).cuda()
    assert abs(float(I.grad_norm([rows])[0]) - norm64([rows])) <= norm64([rows]) * NORM_TOL


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_fp32_sums_end_after_32_elements(dtype):
    """Every sum in fp32 starts with a 1 whose half step is above each of the
    squares that follow: those of the same sum are lost, 7 beside each 1 as long as
    a sum of 32 elements has four parts of 8 squares.  That is 7 half steps of
    the sum, 3.5 of the norm, and one for its rounding; parts of 16 squares
    lose 15."""
    b = 2.0 ** -12 * (1 - torch.finfo(dtype).eps / 2)
    t = torch.full((100, 8, 256, 8), b, device="cuda").to(dtype)      # 8 times 8 elements a thread
    assert float(t[0, 0, 0, 0]) == b
    t[:, 0, :, :4] = 1
    ref = norm64([t])
    assert abs(float(I.grad_norm([t])[0]) - ref) <= 4.5 * 2.0 ** -24 * ref


def test_every_scaled_tensor_has_a_new_version():
    ts = [torch.ones(n, dtype=d, device="cuda") for n, d in ((5, F32), (70, BF16), (9000, F16), (33, F32))]
    ts.append(torch.ones(4, 6, device="cuda")[:, ::2])
    versions = [t._version for t in ts]
    I.scale_grads_([ts[0], None, *ts[1:]], torch.full((), 0.5, device="cuda"))
    assert all(t._version > v for t, v in zip(ts, versions))
