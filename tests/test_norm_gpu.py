"""Layer norm, forward and backward, against its formulas in 64 bits.

Tolerances.  With u the output type's unit roundoff and fp32 sums of at most
n terms in a row, a sum is off by at most n 2^-24 of its terms' magnitudes.
A row of up to 28672 values is summed as 256 or more partial sums of at most
112 terms and a tree: 128 * 2^-24 = 2^-17, doubled for the roundings of the
terms themselves: EPS = 2^-16.  The sums over the tokens have at most M
terms."""
import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}
EPS = 2.0 ** -16
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _data(M, N, dt, wt, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = (torch.randn(M, N, generator=g, device=DEV) * 2 + torch.randn(M, 1, generator=g, device=DEV)).to(dt)
    w = (1 + 0.3 * torch.randn(N, generator=g, device=DEV)).to(wt)
    b = torch.randn(N, generator=g, device=DEV).to(wt)
    gy = torch.randn(M, N, generator=g, device=DEV).to(dt)
    return x, w, b, gy


def _forward64(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1)
    rstd = ((x - mean[..., None]) ** 2).mean(-1).add(eps).rsqrt()
    h = (x - mean[..., None]) * rstd[..., None]
    y = h * (1 if w is None else w.double()) + (0 if b is None else b.double())
    return y, mean, rstd, h


def _check_forward(x, w, b, eps, got):
    y, mean, rstd = got
    ref, mean64, rstd64, h = _forward64(x, w, b, eps)
    aw = 1.0 if w is None else w.double().abs()
    off = EPS * (aw * (rstd64 * x.double().abs().mean(-1))[..., None] + aw * h.abs()
                 + (0 if b is None else b.double().abs()))
    assert y.dtype == x.dtype and y.shape == x.shape
    assert ((y.double() - ref).abs() <= U[x.dtype] * ref.abs() + 1.01 * off + TINY[x.dtype]).all()
    assert ((mean.double() - mean64).abs() <= EPS * x.double().abs().mean(-1)).all()
    assert ((rstd.double() - rstd64).abs() <= EPS * rstd64).all()


SIZES = [(1, 1), (1, 8), (3, 7), (5, 33), (2, 256), (7, 1000), (4, 1100), (33, 2048), (3, 4096), (5, 4099), (2, 8192),
         (3, 11008), (2, 16389), (2, 28672), (1, 40001), (300, 64), (1000, 24)]


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("M,N", SIZES)
def test_forward(M, N, dt):
    x, w, b, _ = _data(M, N, dt, dt, M + N)
    eps = 1e-5 if N > 1 else 1e-3
    _check_forward(x, w, b, eps, I.layer_norm(x, w, b, eps))


@pytest.mark.parametrize("dt,wt", [(F16, F32), (BF16, F32), (F32, BF16), (BF16, F16)])
def test_forward_parameter_types_and_absent_parameters(dt, wt):
    x, w, b, _ = _data(9, 520, dt, wt, 3)
    for ww, bb in ((w, b), (w, None), (None, b), (None, None)):
        _check_forward(x, ww, bb, 1e-5, I.layer_norm(x, ww, bb))


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("M,N", SIZES)
def test_backward(M, N, dt):
    x, w, b, g = _data(M, N, dt, dt, 2 * M + N)
    _, mean, rstd = I.layer_norm(x, w, b, 1e-3)
    _check_backward(x, w, g, mean, rstd, I.layer_norm_backward(g, x, mean, rstd, w))


def _check_backward(x, w, g, mean, rstd, got):
    gx, gw, gb = got
    M, u = x.shape[0], U[x.dtype]
    r = rstd.double()[:, None]
    h = (x.double() - mean.double()[:, None]) * r
    ah = h.abs() + 2 * (x.double().abs() + mean.double().abs()[:, None]) * r * 2.0 ** -8   # the difference's own rounding
    gd = g.double()
    p = gd if w is None else gd * w.double()
    ref = r * (p - p.mean(1, keepdim=True) - h * (p * h).mean(1, keepdim=True))
    if gx is not None:
        off = EPS * r * (p.abs() + p.abs().mean(1, keepdim=True) + ah * (p.abs() * ah).mean(1, keepdim=True))
        assert ((gx.double() - ref).abs() <= u * ref.abs() + 1.01 * off + TINY[x.dtype]).all()
    pt = x.dtype if w is None else w.dtype
    sums = (M + 16) * 2.0 ** -24 + EPS
    if gw is not None:
        ref = (gd * h).sum(0)
        assert gw.dtype == pt
        assert ((gw.double() - ref).abs() <= U[pt] * ref.abs() + 1.01 * sums * (gd.abs() * ah).sum(0) + TINY[pt]).all()
    if gb is not None:
        ref = gd.sum(0)
        assert ((gb.double() - ref).abs() <= U[pt] * ref.abs() + 1.01 * sums * gd.abs().sum(0) + TINY[pt]).all()


# Rows that do not start on 16 bytes, more of them than blocks: every class of
# lengths, either side of its limit.
SHIFTED = [(2500, 513), (2500, 1017), (1300, 1018), (1300, 2041), (700, 2047), (700, 4090), (330, 4094), (330, 6141),
           (170, 6143), (160, 8185), (160, 8190), (90, 8193), (90, 16377), (40, 16378), (40, 20003), (30, 32761),
           (20, 32763), (20, 40003), (9, 8195), (1, 8193), (3, 12006), (12, 25597), (12, 25598), (6, 51193),
           (6, 51194), (160, 20003)]


@pytest.mark.parametrize("dt,wt", [(F16, F32), (BF16, BF16), (F32, F16)])
@pytest.mark.parametrize("M,N", SHIFTED)
def test_shifted_rows(M, N, dt, wt):
    x, w, b, g = _data(M, N, dt, wt, M + 3 * N)
    got = I.layer_norm(x, w, b)
    _check_forward(x, w, b, 1e-5, got)
    back = I.layer_norm_backward(g, x, got[1], got[2], w)
    _check_backward(x, w, g, got[1], got[2], back)
    for need in ((1, 0, 0), (0, 1, 1)):
        some = I.layer_norm_backward(g, x, got[1], got[2], w, *map(bool, need))
        assert all(p is None or torch.equal(p, q) for p, q in zip(some, back))


@pytest.mark.parametrize("N", [75, 1001, 5003, 9001, 20003])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_do_not_touch_each_other(N, bad):
    x, w, b, g = _data(41, N, BF16, F32, N)
    y, mean, rstd = I.layer_norm(x, w, b)
    gx, _, _ = I.layer_norm_backward(g, x, mean, rstd, w)
    x2, g2 = x.clone(), g.clone()
    x2[::2], g2[::2] = bad, bad             # every other row
    y2, mean2, rstd2 = I.layer_norm(x2, w, b)
    gx2, _, _ = I.layer_norm_backward(g2, x2, mean2, rstd2, w)
    for one, two in ((y, y2), (mean, mean2), (rstd, rstd2), (gx, gx2)):
        assert torch.equal(one[1::2], two[1::2]) and not two[::2].float().isfinite().all()


@pytest.mark.parametrize("need", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)])
def test_backward_parts(need):
    x, w, b, g = _data(700, 1032, BF16, F32, 5)
    _, mean, rstd = I.layer_norm(x, w, b)
    whole = I.layer_norm_backward(g, x, mean, rstd, w)
    some = I.layer_norm_backward(g, x, mean, rstd, w, need_x=need[0], need_weight=need[1], need_bias=need[2])
    for n, a, s in zip(need, whole, some):
        assert (s is None) == (not n) and (s is None or torch.equal(a, s))
    _check_backward(x, w, g, mean, rstd, whole)
    _check_backward(x, None, g, mean, rstd, I.layer_norm_backward(g, x, mean, rstd))


def test_many_tokens():
    x, w, b, g = _data(40000, 136, F16, F16, 6)
    y = I.layer_norm(x, w, b)
    _check_forward(x, w, b, 1e-5, y)
    _check_backward(x, w, g, y[1], y[2], I.layer_norm_backward(g, x, y[1], y[2], w))


def test_offsets_past_32_bits():
    """Rows whose elements start past 2^31 (bf16, 4.4 GB)."""
    M, N = 270000, 8192
    x = torch.zeros(M, N, dtype=BF16, device=DEV)
    tail = _data(5, N, BF16, BF16, 8)
    x[-5:] = tail[0]
    y, mean, rstd = I.layer_norm(x, tail[1], tail[2])
    _check_forward(x[-5:], tail[1], tail[2], 1e-5, (y[-5:], mean[-5:], rstd[-5:]))
    assert torch.equal(y[0], tail[2]) and torch.equal(y[M // 2], tail[2])
    y.zero_()
    y[-5:] = tail[3]
    gx, gw, gb = I.layer_norm_backward(y, x, mean, rstd, tail[1])
    _check_backward(x[-5:], tail[1], tail[3], mean[-5:], rstd[-5:], (gx[-5:], None, None))
    h = (tail[0].double() - mean[-5:].double()[:, None]) * rstd[-5:].double()[:, None]
    ref = (tail[3].double() * h).sum(0)
    assert ((gw.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2 * EPS * (tail[3].double() * h).abs().sum(0)).all()


def test_rows_without_variance_and_with_non_finite_values():
    x, w, b, g = _data(6, 4096, F16, F16, 7)
    x[1] = 3.0                                # no variance: y is the bias up to the mean's rounding
    x[2, 17] = float("inf")
    x[3, 5] = float("nan")
    x[4] = 65504.0                            # the type's largest value
    y, mean, rstd = I.layer_norm(x, w, b)
    ok = [0, 1, 4, 5]
    _check_forward(x[ok], w, b, 1e-5, (y[ok], mean[ok], rstd[ok]))
    assert y[2].isnan().all() and y[3].isnan().all()
    gx, _, _ = I.layer_norm_backward(g, x, mean, rstd, w)
    assert gx[2].isnan().any() and gx[3].isnan().all() and gx[[0, 5]].isfinite().all()


def test_strides_shapes_streams_and_repeats():
    x, w, b, g = _data(64, 520, BF16, F32, 9)
    wide = torch.empty(64, 777, dtype=BF16, device=DEV)
    wide[:, 3:523] = x
    ref = I.layer_norm(x, w, b)
    for other in (wide[:, 3:523], x.t().contiguous().t()):
        assert all(torch.equal(p, q) for p, q in zip(I.layer_norm(other, w, b), ref))
    y, mean, rstd = I.layer_norm(x.view(4, 16, 520), w, b)
    assert y.shape == (4, 16, 520) and mean.shape == (4, 16) and torch.equal(y.view(64, 520), ref[0])
    gref = I.layer_norm_backward(g, x, ref[1], ref[2], w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = I.layer_norm(x, w, b)
        g2 = I.layer_norm_backward(g, x, y2[1], y2[2], w)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip((*y2, *g2), (*ref, *gref)))
    out = torch.empty_like(x)
    assert I.layer_norm(x, w, b, out=out)[0] is out and torch.equal(out, ref[0])
    assert torch.equal(I.layer_norm(x, w, b, out=x)[0], ref[0])          # in place


def test_no_tokens():
    w = torch.ones(24, device=DEV)
    x = torch.empty(0, 24, device=DEV)
    y, mean, rstd = I.layer_norm(x, w, w)
    assert y.shape == (0, 24) and mean.shape == (0,)
    gx, gw, gb = I.layer_norm_backward(x, x, mean, rstd, w)
    assert gx.shape == (0, 24) and not gw.any() and not gb.any()


@pytest.mark.parametrize("bias", [True, False])
def test_autograd_against_differences(bias):
    """The gradients along random directions against central differences of
    the 64-bit forward (step 1e-4: its own error is below 1e-6)."""
    x, w, b, c = _data(12, 200, F32, F32, 11)
    norm = I.LayerNorm(200, bias=bias, device=DEV)
    with torch.no_grad():
        norm.weight.copy_(w)
        if bias:
            norm.bias.copy_(b)
    x.requires_grad_(True)
    (norm(x) * c).sum().backward()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)

    def loss(dx, dw, db):
        return (_forward64(x.double() + dx, w.double() + dw, b.double() * bias + db, 1e-5)[0] * c.double()).sum()

    for which, grad in enumerate([x.grad, norm.weight.grad] + ([norm.bias.grad] if bias else [])):
        d = torch.randn(grad.shape, generator=gen, device=DEV).double()
        h = [0.0, 0.0, 0.0]
        h[which] = 1e-4 * d
        diff = (loss(*h) - loss(*[-v for v in h])) / 2e-4
        assert abs(float((grad.double() * d).sum() - diff)) <= 1e-5 * float((grad.double() * d).norm()) * 15


def test_refusals():
    x, w, b, g = _data(4, 24, F16, F16, 1)
    y, mean, rstd = I.layer_norm(x, w, b)
    for call in (lambda: I.layer_norm(x.cpu(), w, b), lambda: I.layer_norm(x, w[:20], b),
                 lambda: I.layer_norm(x, w, b.float()), lambda: I.layer_norm(x.long(), w, b),
                 lambda: I.layer_norm(x, w.long(), None), lambda: I.layer_norm(x, w, b, eps=-1.0),
                 lambda: I.layer_norm(x, w, b, eps=float("nan")), lambda: I.layer_norm(x[:, :0], None, None),
                 lambda: I.layer_norm(x, w, b, out=y.float()), lambda: I.layer_norm(x, w, b, out=y[:, ::2]),
                 lambda: I.layer_norm_backward(g[:2], x, mean, rstd, w),
                 lambda: I.layer_norm_backward(g, x, mean[:2], rstd, w),
                 lambda: I.layer_norm_backward(g, x, mean.double(), rstd, w),
                 lambda: I.layer_norm_backward(g, x, mean, rstd, w, param_dtype=F32),
                 lambda: I.layer_norm_backward(g.float(), x, mean, rstd, w)):
        with pytest.raises(I.I8LTError):
            call()
