"""The gradient norm, scaling and clipping on a GB300 against 64 bits."""
import math

import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
HALF = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
# 32 squares summed in fp32 (each rounded, up to 32 additions), the rest in
# fp64: 33 half steps of the sum of squares, half of that of the norm; and the
# rounding to fp32
NORM_TOL = (33 / 2 + 1) * 2.0 ** -24


def grads(shapes, dtypes, seed=0, std=1e-2):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * std).to(dtypes[i % len(dtypes)]).cuda() for i, s in enumerate(shapes)]


def norm64(ts):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))


SHAPES = [[(1,)], [(7,)], [(3, 5), (0,), (8193,)], [(8192,), (4096, 31)], [(1000, 1000)],
          [(i * 37 + 1,) for i in range(70)], [(i % 7 + 1,) for i in range(2500)], [(i % 5,) for i in range(1100)] + [(20000,)], [(300, 17)] * 33]


@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F16,), (F16, F32, BF16)])
@pytest.mark.parametrize("shapes", SHAPES)
def test_norm(shapes, dtypes):
    ts = grads(shapes, dtypes, len(shapes))
    ref = norm64(ts)
    norm, scale, inf = I.grad_norm(ts, max_norm=0.5 * ref)
    assert norm.shape == () and norm.dtype == F32
    assert abs(float(norm) - ref) <= ref * NORM_TOL
    expect = min(1.0, 0.5 * ref / (ref + 1e-6))
    assert abs(float(scale) - expect) <= expect * (NORM_TOL + 2.0 ** -24) and float(inf) == 0
    again = I.grad_norm(ts, max_norm=0.5 * ref)
    assert all(torch.equal(a, b) for a, b in zip((norm, scale, inf), again))
    assert float(I.grad_norm(ts)[1]) == 1 and float(I.grad_norm(ts, max_norm=3 * ref + 1)[1]) == 1


@pytest.mark.parametrize("start", [0, 1, 3, 7])
def test_norm_of_views(start):
    flat = torch.randn(50000, generator=torch.Generator().manual_seed(start)).cuda()
    for dtype in (F32, F16, BF16):
        f = flat.to(dtype)
        parts = [f[start:start + 3], f[start + 3:9001], f[9001:9002], f[9002:30002].view(7, 3000)]
        ref = norm64(parts)
        assert abs(float(I.grad_norm(parts)[0]) - ref) <= ref * NORM_TOL
    t = flat[:40000].view(200, 200)
    assert abs(float(I.grad_norm([t.T, None, t[:, ::2]])[0]) - norm64([t, t[:, ::2]])) <= 2 * norm64([t]) * NORM_TOL


@pytest.mark.parametrize("size", [2.0 ** -140, 1e-30, 1e-20, 1e18, 1e30])
def test_norm_of_the_whole_range(size):
    t = (torch.rand(70001, generator=torch.Generator().manual_seed(1), dtype=torch.float64) * size).float().cuda()
    ref = norm64([t])
    # below the smallest normal number the result's own step decides
    assert abs(float(I.grad_norm([t])[0]) - ref) <= ref * NORM_TOL + 2.0 ** -149
    mixed = [t, torch.full((5000,), 3.0).cuda()]
    assert abs(float(I.grad_norm(mixed)[0]) - norm64(mixed)) <= norm64(mixed) * NORM_TOL


def test_not_finite():
    for bad in (float("inf"), float("nan"), -float("inf")):
        for dtype in (F16, BF16, F32):
            t = torch.ones(20000, dtype=dtype).cuda()
            t[19999] = bad
            norm, scale, inf = I.grad_norm([t, torch.ones(5).cuda()], max_norm=1.0)
            assert float(inf) == 1 and not math.isfinite(float(norm))
            assert math.isnan(float(scale)) if bad != bad else float(scale) == 0
    big = torch.full((100000,), 3e38).cuda()         # finite gradients whose norm is not
    assert float(I.grad_norm([big])[2]) == 1
    zero, one = torch.zeros(1).cuda(), torch.ones(1).cuda()
    assert float(I.grad_norm([one], found_inf=one)[2]) == 1 and float(I.grad_norm([one], found_inf=zero)[2]) == 0
    assert [float(v) for v in I.grad_norm([torch.zeros(100).cuda()], max_norm=1.0)] == [0, 1, 0]
    assert float(I.grad_norm([one], max_norm=0.0)[1]) == 0


def test_grad_scale():
    ts = grads([(1000,), (77, 3)], (F32,), 5)
    c = torch.tensor([-0.125]).cuda()
    norm, scale, _ = I.grad_norm(ts, max_norm=0.01, grad_scale=c)
    ref = 0.125 * norm64(ts)
    assert abs(float(norm) - ref) <= ref * NORM_TOL
    expect = -0.125 * min(1.0, 0.01 / (ref + 1e-6))
    assert abs(float(scale) - expect) <= abs(expect) * (NORM_TOL + 2.0 ** -24)


@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F16,), (F16, F32, BF16)])
@pytest.mark.parametrize("shapes", SHAPES)
def test_scale(shapes, dtypes):
    ts = grads(shapes, dtypes, len(shapes))
    old = [t.clone() for t in ts]
    c = torch.tensor([0.3]).cuda()
    versions = [t._version for t in ts]
    I.scale_grads_([*ts, None], c)
    assert [t._version for t in ts] > versions
    for t, o in zip(ts, old):
        # one product in fp32, rounded once
        assert torch.equal(t, (o.float() * c).to(o.dtype))


def test_scale_views_and_neighbours():
    flat = torch.randn(30000, generator=torch.Generator().manual_seed(2)).cuda()
    for dtype in (F32, F16, BF16):
        f = flat.to(dtype)
        old = f.clone()
        parts = [f[1:4], f[4:9000], f[9003:20000], f[20001:20002]]
        I.scale_grads_(parts, torch.tensor([2.0]).cuda())
        keep = torch.ones(30000, dtype=torch.bool)
        for a, b in ((1, 4), (4, 9000), (9003, 20000), (20001, 20002)):
            keep[a:b] = False
        assert torch.equal(f[keep.cuda()], old[keep.cuda()])
        assert torch.equal(f[~keep.cuda()], (old[~keep.cuda()].float() * 2).to(dtype))
    m = flat[:20000].view(100, 200).clone()
    expect = m.clone()
    expect[:, ::2] *= 3
    I.scale_grads_([m[:, ::2]], torch.tensor([3.0]).cuda())
    assert torch.equal(m, expect)
    with pytest.raises(I.I8LTError):
        I.scale_grads_([flat, flat[100:200]], torch.ones(1).cuda())


def test_clip_and_step():
    torch.manual_seed(3)
    shapes, dtypes = [(40, 30), (77,), (5, 5)], [F32, BF16, F32]
    params = [torch.nn.Parameter(torch.randn(s).to(d).cuda()) for s, d in zip(shapes, dtypes)]
    params.append(torch.nn.Parameter(torch.ones(3).cuda()))          # without a gradient
    for p in params[:3]:
        p.grad = torch.randn_like(p)
    before = [p.grad.clone() for p in params[:3]]
    ref = norm64(before)
    clones = [torch.nn.Parameter(p.detach().clone()) for p in params]
    for c, p in zip(clones, params):
        c.grad = None if p.grad is None else p.grad.clone()
    # the step that clips, against a step with the factor given
    a, b = I.AdamW(params, lr=1e-2), I.AdamW(clones, lr=1e-2)
    norm = a.step(max_norm=1.0)
    assert abs(float(norm) - ref) <= ref * NORM_TOL
    assert b.step(grad_scale=I.grad_norm([c.grad for c in clones[:3]], 1.0)[1].reshape(1)) is None
    assert all(torch.equal(p, c) for p, c in zip(params, clones))
    assert all(torch.equal(p.grad, g) for p, g in zip(params, before))
    # a norm that is not finite skips the step
    held = [p.detach().clone() for p in params]
    params[1].grad[5] = float("nan")
    a.step(max_norm=1.0)
    assert all(torch.equal(p, h) for p, h in zip(params, held))
    params[1].grad.copy_(before[1])
    got = I.clip_grad_norm_(params, 0.5)
    assert abs(float(got) - ref) <= ref * NORM_TOL
    for p, g in zip(params, before):
        f = float(I.grad_norm(before, 0.5)[1])
        assert torch.equal(p.grad, (g.float() * torch.tensor(f)).to(g.dtype))


def test_captured_and_replayed():
    ts = grads([(5000,), (129, 77)], (F32, BF16), 9)
    limit = 0.01
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        I.grad_norm(ts, limit)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, scale, inf = I.grad_norm(ts, limit)
        I.scale_grads_(ts, scale)
    for seed in (1, 2):
        for t, n in zip(ts, grads([(5000,), (129, 77)], (F32, BF16), seed)):
            t.copy_(n)
        ref = norm64(ts)
        graph.replay()
        assert abs(float(norm) - ref) <= ref * NORM_TOL
        assert abs(norm64(ts) - limit) <= limit * (HALF[BF16] + 1e-3)


def test_refusals():
    one = torch.ones(4).cuda()
    for call in (lambda: I.grad_norm([]), lambda: I.grad_norm([None]), lambda: I.grad_norm([one.cpu()]),
                 lambda: I.grad_norm([one, one.cpu()]), lambda: I.grad_norm([one.long()]),
                 lambda: I.grad_norm([one], max_norm=-1.0), lambda: I.grad_norm([one], max_norm=float("nan")),
                 lambda: I.grad_norm([one], grad_scale=one), lambda: I.grad_norm([one], found_inf=one.double()[:1]),
                 lambda: I.scale_grads_([one], one), lambda: I.scale_grads_([one], torch.ones(1)),
                 lambda: I.scale_grads_([one, one], torch.ones(1).cuda())):
        with pytest.raises(I.I8LTError):
            call()
    I.scale_grads_([], torch.ones(1).cuda())
    I.scale_grads_([None], torch.ones(1).cuda())


def test_an_expanded_gradient_is_refused_before_any_is_scaled():
    a = torch.ones(40, device="cuda")
    wide = torch.ones(1, 8, device="cuda").expand(5, 8)
    with pytest.raises(I.I8LTError, match="expanded"):
        I.scale_grads_([a, wide], torch.full((), 0.5, device="cuda"))
    assert bool((a == 1).all()) and bool((wide == 1).all())
    norm = I.grad_norm([a, wide])[0]                 # it may be read
    assert abs(norm.item() - 80 ** 0.5) <= 80 ** 0.5 * 2.0 ** -22
    column = torch.ones(6, 3, device="cuda")[:, 1:2]     # a step of 0 along one element is no sharing
    I.scale_grads_([column], torch.full((), 0.5, device="cuda"))
    assert bool((column == 0.5).all())
