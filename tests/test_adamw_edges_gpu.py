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


def _adamw64(p, grads, lr, b1=0.9, b2=0.95, eps=1e-8, wd=0.01):
    """The formulas in 64 bits over one tensor's gradients, its own steps
    counted (None: no update)."""
    p, m, v, n = p.double().cpu(), 0.0, 0.0, 0
    for g in grads:
        if g is None:
            continue
        g, n = g.double().cpu(), n + 1
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        p = p * (1 - lr * wd) - lr / (1 - b1 ** n) * m / ((v / (1 - b2 ** n)) ** 0.5 + eps)
    return p


# An E4M3 code is off by 2^-4 of the value: an update of 8-bit states by about
# an eighth of lr a step, against 0.55 lr where the bias corrections are those
# of step 100 (0.1 / 0.2236 in place of 1).  32 bits: 2^-24 of p and of 16
# operations a step.
def _near(got, want, steps, lr, bits):
    tol = steps * (lr / 4 if bits == 8 else 16 * 2.0 ** -24 * (lr + float(want.abs().max())))
    return float((got.double().cpu() - want).abs().max()) <= tol


@pytest.mark.parametrize("bits", [32, 8])
def test_a_late_first_gradient(bits):
    """A parameter whose first gradient comes with the optimizer's 100th step:
    its first update is of size lr."""
    lr = 1e-2
    ps = [_grad(700, 1, 0.1), _grad(300, 2, 0.1), _grad(256, 3, 0.1)]
    start = [p.clone() for p in ps]
    opt = I.AdamW(ps, lr=lr, betas=(0.9, 0.95), bits=bits)
    seen = [[], [], []]
    for step in range(101):
        gs = [_grad(700, 10), None if step < 99 else _grad(300, 20 + step), _grad(256, 11) if step % 2 else None]
        for p, g, s in zip(ps, gs, seen):
            p.grad = g
            s.append(g)
        opt.step()
    assert _near(ps[1], _adamw64(start[1], seen[1], lr), 2, lr, bits)
    if bits == 32:
        for k in (0, 2):
            assert _near(ps[k], _adamw64(start[k], seen[k], lr), 101, lr, bits)


@pytest.mark.parametrize("bits", [32, 8])
def test_skipped_first_steps(bits):
    """Steps that found_inf skips (a loss scaler's first ones) do not count,
    for the tensors they concern."""
    lr = 1e-2
    ps = [_grad(700, 1, 0.1), _grad(300, 2, 0.1)]
    start = [p.clone() for p in ps]
    opt = I.AdamW(ps, lr=lr, betas=(0.9, 0.95), bits=bits)
    for step in range(40):
        ps[0].grad, ps[1].grad = _grad(700, 7) * INF, _grad(300, 8) * INF
        opt.step(found_inf=torch.ones(1, device=DEV))
    gs = [_grad(700, 9), _grad(300, 10)]
    for p, g in zip(ps, gs):
        p.grad = g
    opt.step(found_inf=torch.zeros(1, device=DEV))
    for p, s, g in zip(ps, start, gs):
        assert _near(p, _adamw64(s, [g], lr), 1, lr, bits)
    opt.step()
    for p, s, g in zip(ps, start, gs):
        assert _near(p, _adamw64(s, [g, g], lr), 2, lr, bits)


@pytest.mark.parametrize("bits", [32, 8])
def test_counts_in_the_state_dict(bits):
    def made():
        ps = [_grad(700, 1, 0.1), _grad(300, 2, 0.1), _grad(64, 2, 0.1).bfloat16()]
        return ps, I.AdamW(ps, lr=1e-2, bits=bits)

    def steps(ps, opt, first, last):
        for step in range(first, last):
            for k, p in enumerate(ps):
                p.grad = _grad(p.numel(), 30 * k + step).to(p.dtype) if (step + k) % 3 else None
            opt.step(found_inf=torch.full((1,), float(step % 4 == 1), device=DEV))

    whole, opt = made()
    steps(whole, opt, 0, 12)
    half, opt = made()
    steps(half, opt, 0, 5)
    fresh = I.AdamW(half, lr=1e-2, bits=bits)
    fresh.load_state_dict(opt.state_dict())
    steps(half, fresh, 5, 12)
    assert all(torch.equal(a, b) for a, b in zip(whole, half))


@pytest.mark.parametrize("bits", [32, 8])
def test_counted_steps(bits):
    """Update counts in place of a step number: the same bits, in lists of any
    length, with empty tensors and with several lists, and in a replayed CUDA
    graph."""
    sizes = [300, 0, 13, 513] * 300
    p0, gs = [_grad(n, n, 0.1) for n in sizes], [_grad(n, n + 1) for n in sizes]
    ps, qs, rs = ([p.clone() for p in p0] for _ in range(3))
    n = I.adamw_state_size(ps)
    one, two, three = _states(n, bits), _states(n, bits), _states(n, bits)
    counts, again = I.adamw_counts(ps), I.adamw_counts(ps)
    for step in (1, 2, 3):
        some = [g if k % 7 else None for k, g in enumerate(gs)]
        _call(bits)(ps, some, *one, step=step, **HYPER)
        _call(bits)(qs, some, *two, step=counts, **HYPER)
    for a, b in zip((*ps, *one), (*qs, *two)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert counts[:, 0].tolist() == [3 if k % 7 and sizes[k] else 0 for k in range(len(sizes))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _call(bits)([p.clone() for p in p0], some, *_states(n, bits), step=I.adamw_counts(ps), **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(bits)(rs, some, *three, step=again, **HYPER)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*ps, *one), (*rs, *three)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for bad in (counts[:5], counts.int(), counts.cpu(), counts.t().contiguous().t()):
        with pytest.raises(I.I8LTError):
            _call(bits)(ps, gs, *one, step=bad, **HYPER)
