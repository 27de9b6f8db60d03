"""AdamW at the edges of its numbers and of its lists of tensors.

Values are compared with the same single fp32 operations in torch on the CPU
(states: equal; a NaN equals a NaN) and parameters with the 64-bit formula on
these states, within 8 * 2^-24 of the update and of the parameter."""
import math

import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _states(n, bits):
    if bits == 32:
        return torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    q = [torch.zeros(n, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
    top = [torch.zeros(n // 256, device=DEV) for _ in range(2)]
    return q[0], top[0], q[1], top[1]


def _call(bits):
    return I.adamw_step_8bit if bits == 8 else I.adamw_step


def _moments(m, v, g):
    b1, b2 = torch.tensor(HYPER["beta1"]), torch.tensor(HYPER["beta2"])
    c1, c2 = torch.tensor(1 - HYPER["beta1"]), torch.tensor(1 - HYPER["beta2"])
    return m * b1 + g * c1, v * b2 + (g * g) * c2


def _decode(q, top):
    return (q.cpu().view(-1, 256).float() * (top.cpu() * torch.tensor(1.0 / 448.0))[:, None]).view(-1)


def _param64(p, m, r, step):
    upd = HYPER["lr"] / (1 - HYPER["beta1"] ** step) * m.double() / \
        (r.double() / math.sqrt(1 - HYPER["beta2"] ** step) + HYPER["eps"])
    return p.double() * (1 - HYPER["lr"] * HYPER["weight_decay"]) - upd, upd


def _grad(n, seed, std=1e-2):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(n, generator=g, device=DEV) * std


@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_gradient_whose_square_overflows(bits, gt):
    """v is then infinite and the update zero: the parameter decays only,
    whatever its neighbours' gradients are."""
    n = 256 * 4
    g = _grad(n, 1)
    g[256:512] = 0.0                                # neighbours without a gradient
    g[5], g[256 + 77], g[512] = 3e19, -2e30, 2e19
    g = g.to(gt)
    p = _grad(n, 2, 0.1)
    before = p.cpu().clone()
    st = _states(n, bits)
    _call(bits)([p], [g], *st, step=1, **HYPER)
    m, v = _moments(torch.zeros(n), torch.zeros(n), g.cpu().float())
    assert v.isinf().sum() == 3
    want, upd = _param64(before, m, v.sqrt(), 1)
    assert ((p.cpu().double() - want).abs() <= 8 * 2.0 ** -24 * (upd.abs() + before.double().abs())).all()
    if bits == 32:
        assert torch.equal(st[0].cpu(), m) and torch.equal(st[1].cpu(), v)
    else:
        top = v.sqrt().view(-1, 256).amax(1)
        assert torch.equal(st[3].cpu(), top) and torch.equal(st[1].cpu(), m.abs().view(-1, 256).amax(1))
        r = _decode(st[2], st[3]).view(-1, 256)
        assert not r[top.isinf()].isfinite().any() and r[top.isfinite()].isfinite().all()


def test_roots_over_their_whole_range():
    """r's absmax is the rounded root of v: blocks whose second moments span
    every octave, subnormal numbers among them, and every significand of two
    octaves in steps of 2^-13."""
    v = torch.cat([2.0 ** torch.arange(-149, 127, 0.25, dtype=torch.double).float(),
                   1 + torch.arange(0, 3 * 2 ** 13).double().mul(2.0 ** -13).float(),
                   torch.nextafter(2.0 ** torch.arange(-140, 127).float(), torch.tensor(0.0)),
                   torch.nextafter(2.0 ** torch.arange(-140, 127).float(), torch.tensor(1e38))])
    # one value per block: g with c2 = 1 - 0 = 1 and v = g * g
    g = v.sqrt()
    n = 256 * len(g)
    grad = torch.zeros(n, device=DEV)
    grad[::256] = g.to(DEV)
    st = _states(n, 8)
    I.adamw_step_8bit([torch.zeros(n, device=DEV)], [grad], *st, step=1, lr=1e-3, beta1=0.9, beta2=0.0)
    assert torch.equal(st[3].cpu(), (g * g).sqrt())


@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("rest", [1e-2, 0.0])
def test_a_non_finite_gradient_makes_its_block_non_finite(rest, bad, gt):
    """8 bits: all 256 values of both moments; other blocks keep theirs."""
    n = 256 * 3
    g = _grad(n, 3, rest)
    g[256 + 100] = bad
    g = g.to(gt)
    st = _states(n, 8)
    p = _grad(n, 4, 0.1)
    clean = [t.clone() for t in st]
    I.adamw_step_8bit([p], [g], *st, step=1, **HYPER)
    hit = torch.zeros(n, dtype=torch.bool)
    hit[256:512] = True
    for q, top in ((st[0], st[1]), (st[2], st[3])):
        value = _decode(q, top)
        assert not value[hit].isfinite().any() and value[~hit].isfinite().all()
        assert not top[1].isfinite()
    assert not p[356].isfinite() and p[:256].isfinite().all() and p[512:].isfinite().all()
    alone, q = _grad(n, 4, 0.1), clean
    g[256 + 100] = 0.0
    I.adamw_step_8bit([alone], [g], *q, step=1, **HYPER)
    for a, b in zip(st, q):
        assert torch.equal(a.view(torch.uint8).view(3, -1)[::2], b.view(torch.uint8).view(3, -1)[::2])
    keep = torch.arange(n, device=DEV) != 356
    assert torch.equal(p[keep], alone[keep])


@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_non_finite_gradient_in_32_bits(bad):
    """32 bits: the moments of that element."""
    n = 600
    g = _grad(n, 3)
    g[300] = bad
    st = _states(I.adamw_state_size([g]), 32)
    p = _grad(n, 4, 0.1)
    I.adamw_step([p], [g], *st, step=1, **HYPER)
    for t in (*st, p):
        assert not t[300].isfinite() and t[:300].isfinite().all() and t[301:].isfinite().all()


@pytest.mark.parametrize("odd", [False, True])
def test_what_lies_past_a_tensors_end_is_not_used(odd):
    """8 bits: codes there enter neither the block's absmax nor its codes, and
    are 0 afterwards."""
    sizes = [300, 1, 513]
    ps = [_grad(n + 1, n, 0.1)[1:] if odd else _grad(n, n, 0.1) for n in sizes]
    gs = [_grad(n, n + 1) for n in sizes]
    total = I.adamw_state_size(ps)
    inside = torch.zeros(total, dtype=torch.bool, device=DEV)
    for at, n in zip((0, 512, 768), sizes):
        inside[at:at + n] = True
    clean, dirty = _states(total, 8), _states(total, 8)
    for st in (clean, dirty):
        for top in (st[1], st[3]):
            top.fill_(1e-2)
    for k in (0, 2):
        dirty[k].view(torch.uint8).masked_fill_(~inside, 0x7e)      # 448
    qs = [p.clone() for p in ps]
    for st, params in ((clean, ps), (dirty, qs)):
        I.adamw_step_8bit(params, gs, *st, step=2, **HYPER)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(clean, dirty))
    assert all(torch.equal(a, b) for a, b in zip(ps, qs))
    assert not dirty[0].view(torch.uint8)[~inside].any() and not dirty[2].view(torch.uint8)[~inside].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_given_twice_is_refused(bits):
    p, g = _grad(300, 1), _grad(300, 2)
    flat = _grad(600, 3)
    with pytest.raises(I.I8LTError):
        I.AdamW([p, _grad(4, 4), p], bits=bits)
    with pytest.raises(I.I8LTError):
        I.AdamW([flat[:400], flat[300:]], bits=bits)
    n = I.adamw_state_size([p, p])
    with pytest.raises(I.I8LTError):
        _call(bits)([p, p], [g, g], *_states(n, bits), step=1, lr=1e-3)
    I.AdamW([flat[:300], flat[300:], flat[:0], flat[:0]], bits=bits)      # neighbours, and tensors of nothing
