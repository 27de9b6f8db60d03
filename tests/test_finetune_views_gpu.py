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


def _off(t, by=1):
    """The same values, contiguous, `by` elements off a 16-byte boundary."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    v = flat[by:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16 != 0
    return v


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("N", [64, 4099])
def test_layer_norm_on_views(N, dt):
    x, g, w, b = _normal(9, N, seed=1, dt=dt), _normal(9, N, seed=2, dt=dt), _normal(N, seed=3, dt=dt), _normal(N, seed=4, dt=dt)
    ref = I.layer_norm(x, w, b)
    got = I.layer_norm(_off(x), _off(w), _off(b, 3))
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    back = I.layer_norm_backward(g, x, ref[1], ref[2], w)
    got = I.layer_norm_backward(_off(g), _off(x), _off(ref[1]), _off(ref[2]), _off(w))
    assert all(torch.equal(p, q) for p, q in zip(got, back))
    # what torch.cat's and narrow's backward hand on: parts of one gradient
    norm = I.LayerNorm(N, device=DEV, dtype=dt)
    parts = [x[:3].clone().requires_grad_(True), x[3:].clone().requires_grad_(True)]
    torch.cat([norm(p) for p in parts]).backward(g)
    for p, gy in zip(parts, (g[:3].clone(), g[3:].clone())):
        alone = p.detach().clone().requires_grad_(True)
        norm(alone).backward(gy)
        assert torch.equal(p.grad, alone.grad)
    with pytest.raises(I.I8LTError):                # a caller's output is not copied
        I.layer_norm(x, w, b, out=_off(x))


@pytest.mark.parametrize("K,N,r", [(64, 128, 8), (515, 257, 5)])
@pytest.mark.parametrize("M", [40, 700])
def test_adapters_on_views(M, K, N, r):
    E = 3
    A, B, scale = _normal(E, r, K, seed=1), _normal(E, N, r, seed=2), torch.rand(E, device=DEV)
    x, base, g, addend = (_normal(M, c, seed=s) for c, s in ((K, 3), (N, 4), (N, 5), (K, 6)))
    index = (torch.arange(M, device=DEV) * 7 % (E + 1) - 1).int()
    plan, plan2 = I.adapter_plan(index, E), I.adapter_plan(_off(index), E)
    y, t = I.adapters_forward(x, A, B, scale, plan, base=base)
    y2, t2 = I.adapters_forward(_off(x), _off(A), _off(B), _off(scale), plan2, base=_off(base))
    assert torch.equal(y, y2) and torch.equal(t, t2)
    ref = I.adapters_backward(g, x, t, A, B, scale, plan, addend=addend)
    got = I.adapters_backward(_off(g), _off(x), _off(t), _off(A), _off(B), scale, plan, addend=_off(addend))
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    ad = _layer(K, N, r, E)
    cut = M // 2 + 1
    parts = [x[:cut].clone().requires_grad_(True), x[cut:].clone().requires_grad_(True)]
    ys = [ad(p, I.adapter_plan(i, E)) for p, i in zip(parts, (index[:cut], index[cut:]))]
    torch.cat(ys).backward(g)
    for p, i, gy in zip(parts, (index[:cut], index[cut:]), (g[:cut].clone(), g[cut:].clone())):
        alone = p.detach().clone().requires_grad_(True)
        ad(alone, I.adapter_plan(i.clone(), E)).backward(gy)
        assert torch.equal(p.grad, alone.grad)
    with pytest.raises(I.I8LTError):
        I.adapters_forward(x, A, B, scale, plan, base=base, out=_off(base))


def test_adamw_on_gradients_of_any_offset():
    p, q, g = _normal(300, dt=F32), _normal(300, dt=F32), _normal(300, seed=1, dt=F32)
    m, v, m2, v2 = (torch.zeros(512, device=DEV) for _ in range(4))
    I.adamw_step([p], [g], m, v, step=1, lr=1e-2)
    I.adamw_step([q], [_off(g)], m2, v2, step=1, lr=1e-2)
    assert torch.equal(p, q) and torch.equal(m, m2) and torch.equal(v, v2)


def test_changes_in_place_are_reported():
    """What a backward pass still needs may not change under it unnoticed."""
    x, w = _normal(6, 64, dt=F32), _normal(64, seed=1, dt=F32)

    def stale(change):
        p = w.clone().requires_grad_(True)
        h = _normal(6, 64, seed=2, dt=F32).requires_grad_(True)
        y = (h * p).sum()                           # keeps p
        change(p)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()

    z = lambda *s: torch.zeros(*s, device=DEV)      # noqa: E731
    codes = lambda: torch.zeros(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)   # noqa: E731
    stale(lambda p: I.adamw_step([p], [w], z(256), z(256), step=1, lr=1e-2))
    stale(lambda p: I.adamw_step_8bit([p], [w], codes(), z(1), codes(), z(1), step=1, lr=1e-2))

    def by_optimizer(p):
        opt = I.AdamW([p], lr=1e-2)
        p.grad = w.clone()
        opt.step()

    stale(by_optimizer)
    # outputs that a caller gives
    a = torch.ones(6, 64, device=DEV)
    p = w.clone().requires_grad_(True)
    y = (a * p).sum()
    I.layer_norm(x, out=a)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    a = torch.ones(6, 64, device=DEV, dtype=F16)
    p = w.half().requires_grad_(True)
    y = (a * p).sum()
    I.adapters_forward(x.half(), _normal(1, 4, 64, dt=F16), _normal(1, 64, 4, dt=F16), None,
                       I.adapter_plan(None, 1, 6, DEV), base=a, out=a)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_a_step_between_a_forward_and_its_backward():
    ad = _layer(64, 48, 8, 1)
    opt = I.AdamW([ad.A, ad.B], lr=1e-2)
    x = _normal(20, 64, seed=3).requires_grad_(True)
    y = ad(x)
    y.sum().backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_a_scale_that_wants_a_gradient_is_refused():
    ad = _layer(64, 48, 8, 2)
    x = _normal(20, 64, seed=3).requires_grad_(True)
    plan = I.adapter_plan(None, 2, 20, DEV)
    scale = torch.ones(2, device=DEV, requires_grad=True)
    y = I.AdaptersFunction.apply(x, ad.base(x), ad.A, ad.B, scale, plan)
    with pytest.raises(I.I8LTError, match="scale"):
        y.sum().backward()
    y = I.AdaptersFunction.apply(x, ad.base(x), ad.A, ad.B, scale.detach(), plan)
    y.sum().backward()


def test_second_derivatives_are_refused():
    """A penalty on a gradient would otherwise lose its own gradient."""
    ad, norm = _layer(64, 48, 8, 1), I.LayerNorm(64, device=DEV)
    for f in (lambda x: ad(x), lambda x: norm(x)):
        x = _normal(20, 64, seed=3).requires_grad_(True)
        y = (f(x).float() ** 2).sum()
        g, = torch.autograd.grad(y, x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (y + (g.float() ** 2).sum()).backward()


@pytest.mark.parametrize("M", [20, 700])
def test_an_output_over_the_tokens_is_refused(M):
    x, plan = _normal(M, 64), I.adapter_plan(None, 1, M, DEV)
    A, B = _normal(1, 8, 64, seed=1), _normal(1, 64, 8, seed=2)
    with pytest.raises(I.I8LTError):
        I.adapters_forward(x, A, B, None, plan, out=x)
    y, _ = I.adapters_forward(x, A, B, None, plan, base=x)
    assert torch.equal(I.adapters_forward(x, A, B, None, plan, base=x.clone())[0], y)
