"""AdamW over many tensors, states in 32 and in 8 bits.

The states are single fp32 operations in a fixed order: they are compared bit
for bit with the same operations in torch on the CPU.  The parameters are
compared with the 64-bit formula: their update is a handful of fp32
operations (8 * 2^-24 of the update and of the parameter), rounded once to
the parameter's type."""
import math

import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32, F8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _encode(x, floor):
    b = x.view(-1, 256)
    top = b.abs().amax(1, keepdim=True)
    one = torch.ones_like(top)
    inv = torch.where(top >= 2.0 ** -100, one / torch.where(top >= 2.0 ** -100, top, one), torch.zeros_like(top))
    y = b * (inv * 448.0)
    if floor:
        y = torch.where(b > 0, y.clamp(min=2.0 ** -9), y)
    return y.to(F8).view(-1), top.view(-1)


def _decode(q, top):
    return (q.view(-1, 256).float() * (top * torch.tensor(1.0 / 448.0))[:, None]).view(-1)


def _flat(ts, sizes):
    out = torch.zeros(sum(-(-n // 256) * 256 for n in sizes))
    at = 0
    for t, n in zip(ts, sizes):
        out[at:at + n] = t.float().cpu().view(-1)
        at += -(-n // 256) * 256
    return out


def _moments(m, v, g, h=HYPER):
    """The fp32 chain of the definition (CPU)."""
    b1, b2 = torch.tensor(h["beta1"]), torch.tensor(h["beta2"])
    c1, c2 = torch.tensor(1 - h["beta1"]), torch.tensor(1 - h["beta2"])
    return m * b1 + g * c1, v * b2 + (g * g) * c2


def _param64(p, m, r, step, h=HYPER):
    upd = h["lr"] / (1 - h["beta1"] ** step) * m.double() / (r.double() / math.sqrt(1 - h["beta2"] ** step) + h["eps"])
    return p.double() * (1 - h["lr"] * h["weight_decay"]) - upd, upd


def _tensors(sizes, pt, gt, seed, std=1e-2, odd_start=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def one(n, s, dt):
        t = (torch.randn(n + 1, generator=g, device=DEV) * s).to(dt)
        return t[1:] if odd_start else t[1:].clone()
    return [one(n, 0.1, pt) for n in sizes], [one(n, std, gt) for n in sizes]


SIZES = [[1], [256], [255, 257], [5, 0, 1000, 512], [4096 * 16, 16 * 11008 + 3], [13] * 40, [300] * 1030, [100003]]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,gt,odd", [(F32, F32, False), (BF16, BF16, False), (F16, F16, True), (F32, BF16, False),
                                       (F32, F32, True), (BF16, F32, False)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_steps(sizes, pt, gt, odd, bits):
    ps, _ = _tensors(sizes, pt, gt, 1, odd_start=odd)
    total = I.adamw_state_size(ps)
    m, r = torch.zeros(total), torch.zeros(total)        # the reference's values between steps
    v = torch.zeros(total)
    if bits == 8:
        q = [torch.zeros(total, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
        top = [torch.zeros(total // 256, device=DEV) for _ in range(2)]
        state = (q[0], top[0], q[1], top[1])
    else:
        state = (torch.zeros(total, device=DEV), torch.zeros(total, device=DEV))
    for step in (1, 2, 3):
        _, gs = _tensors(sizes, pt, gt, 10 + step, odd_start=odd)
        before = _flat(ps, sizes)
        (I.adamw_step_8bit if bits == 8 else I.adamw_step)(ps, gs, *state, step=step, **HYPER)
        if bits == 8:
            v = r * r
        m, v = _moments(m, v, _flat(gs, sizes))
        r = v.sqrt()
        want, upd = _param64(before, m, r, step)
        got = _flat(ps, sizes)
        # the chain's roundings reach p through the update; then one rounding to pt
        tol = U[pt] * want.abs() + 8 * 2.0 ** -24 * (upd.abs() + before.double().abs()) + 2.0 ** -25 * (pt == F16)
        inside = _flat([torch.ones(n) for n in sizes], sizes) > 0
        assert ((got.double() - want).abs() <= tol)[inside].all()
        if bits == 8:
            q1, t1 = _encode(m, False)
            q2, t2 = _encode(r, True)
            for a, b in zip(state, (q1, t1, q2, t2)):
                assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
            m, r = _decode(q1, t1), _decode(q2, t2)
        else:
            assert torch.equal(state[0].cpu()[inside], m[inside]) and torch.equal(state[1].cpu()[inside], v[inside])


def test_8bit_codes_over_their_whole_range():
    """Blocks that span many octaves, blocks of zeros, blocks so small that
    their reciprocal would overflow, one value above zero among zeros."""
    n = 256 * 6
    g = torch.logspace(-12, 2, n, base=10, device=DEV) * torch.where(torch.arange(n, device=DEV) % 3 == 0, -1.0, 1.0)
    g[256:512] = 0.0
    g[512:768] = 1e-38
    g[768:1024] = 0.0
    g[800] = 3e-5
    g[1024:1280] = torch.logspace(-15, 3, 256, base=10, device=DEV)
    p = torch.zeros(n, device=DEV)
    q = [torch.zeros(n, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
    top = [torch.zeros(6, device=DEV) for _ in range(2)]
    I.adamw_step_8bit([p], [g], q[0], top[0], q[1], top[1], step=1, **HYPER)
    m, v = _moments(torch.zeros(n), torch.zeros(n), g.cpu())
    q1, t1 = _encode(m, False)
    q2, t2 = _encode(v.sqrt(), True)
    for a, b in zip((q[0], top[0], q[1], top[1]), (q1, t1, q2, t2)):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
    codes = q[1].view(torch.uint8)
    assert (codes[(v.sqrt() > 0).to(DEV)] > 0).all()          # a second moment above zero keeps a code above zero
    assert not codes[256:512].any() and p.isfinite().all()


@pytest.mark.parametrize("bits", [32, 8])
def test_grad_scale_found_inf_and_missing_gradients(bits):
    sizes = [700, 300, 256]

    def run(grads, **kw):
        ps, _ = _tensors(sizes, F32, F32, 1)
        opt = I.AdamW(ps, lr=1e-2, bits=bits)
        for p, g in zip(ps, grads):
            p.grad = g
        opt.step(**kw)
        return ps, opt.states[0]

    start, gs = _tensors(sizes, F32, F32, 1)
    half = torch.tensor([0.5], device=DEV)
    a, sa = run([g * 0.5 for g in gs])
    b, sb = run(gs, grad_scale=half)
    same = lambda x, y: all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(x, y))  # noqa: E731
    assert same(a, b) and same(sa, sb)
    c, sc = run([g * float("inf") for g in gs], found_inf=torch.tensor([1.0], device=DEV))
    assert same(c, start) and not any(t.float().any() for t in sc)
    d, sd = run(gs, found_inf=torch.tensor([0.0], device=DEV), grad_scale=half)
    assert same(a, d) and same(sa, sd)
    e, se = run([gs[0] * 0.5, None, gs[2] * 0.5])
    assert torch.equal(e[0], a[0]) and torch.equal(e[1], start[1]) and torch.equal(e[2], a[2])
    assert not se[0].float()[768:768 + 512].any() and torch.equal(se[0].float()[1280:], sa[0].float()[1280:])


def test_optimizer_types_streams_and_state_dict():
    ps, gs = _tensors([1000, 64], BF16, BF16, 3)
    ps2, gs2 = _tensors([512], F32, F32, 4)
    ps, gs = ps + ps2, gs + gs2

    def train(bits, steps, opt=None, qs=None):
        qs = [p.clone() for p in ps] if qs is None else qs
        opt = opt or I.AdamW(qs, lr=1e-2, bits=bits)
        for q, g in zip(qs, gs):
            q.grad = g
        for _ in range(steps):
            opt.step()
        return qs, opt

    for bits in (32, 8):
        whole, _ = train(bits, 4)
        half, opt = train(bits, 2)
        fresh = I.AdamW(half, lr=1e-2, bits=bits)
        fresh.load_state_dict(opt.state_dict())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            train(bits, 2, fresh, half)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(whole, half))
        with pytest.raises(I.I8LTError):
            I.AdamW(ps[:1], bits=bits).load_state_dict(opt.state_dict())


def test_refusals():
    ps, gs = _tensors([300, 256], F32, F32, 5)
    n = I.adamw_state_size(ps)
    assert n == 768
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    kw = dict(step=1, lr=1e-3)
    call = I.adamw_step
    two = torch.zeros(512, 2, device=DEV)
    for bad in (lambda: call(ps, gs[:1], m, v, **kw), lambda: call(ps, [gs[0], gs[0]], m, v, **kw),
                lambda: call(ps, gs, m[:512], v, **kw), lambda: call(ps, gs, m, v.half(), **kw),
                lambda: call(ps, gs, m.cpu(), v, **kw), lambda: call([ps[0], ps[1].half()], gs, m, v, **kw),
                lambda: call(ps, [gs[0], gs[1].half()], m, v, **kw), lambda: call(ps, gs, m, v, step=0, lr=1e-3),
                lambda: call(ps, gs, m, v, step=1, lr=float("nan")), lambda: call(ps, gs, m, v, beta1=1.0, **kw),
                lambda: call(ps, gs, m, v, beta2=-0.1, **kw), lambda: call(ps, gs, m, v, eps=-1.0, **kw),
                lambda: call([two[:, 0]], [two[:, 1]], m, v, **kw), lambda: call([p.cpu() for p in ps], gs, m, v, **kw),
                lambda: call(ps, gs, m, v, grad_scale=torch.ones(2, device=DEV), **kw),
                lambda: call(ps, gs, m, v, found_inf=torch.ones(1, dtype=F16, device=DEV), **kw),
                lambda: call([p.long() for p in ps], gs, m, v, **kw),
                lambda: I.adamw_step_8bit(ps, gs, m, m[:3], v, v[:3], **kw), lambda: I.AdamW(ps, bits=16)):
        with pytest.raises(I.I8LTError):
            bad()
    call([], [], m[:0], v[:0], **kw)
    call(ps, [None, None], m, v, **kw)
