"""Low-rank adapters of many requests beside a shared projection, against
their formulas in 64 bits.

Tolerances.  u: the compute type's unit roundoff; an fp32 sum of n products
is off by at most n 2^-23 of its terms' magnitudes (whatever the order and
the accumulator's rounding mode).  t and u are rounded to the compute type
and their error passes on through the second product; every output is rounded
once."""
import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F16: 2.0 ** -24, BF16: 2.0 ** -126}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _data(M, K, N, r, E, dt, order="mixed", seed=0):
    g = _gen(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dt)

    d = dict(x=normal(M, K), A=normal(E, r, K, std=K ** -0.5), B=normal(E, N, r, std=0.3), base=normal(M, N),
             g=normal(M, N), addend=normal(M, K), scale=0.5 + torch.rand(E, generator=g, device=DEV))
    if order == "mixed":
        index = torch.randint(-1, E, (M,), generator=g, device=DEV)
    elif order == "one":                    # every token the last adapter
        index = torch.full((M,), E - 1, device=DEV)
    elif order == "none":                   # no token has an adapter
        index = torch.randint(0, 2, (M,), generator=g, device=DEV) * (E + 5) - 1
    else:                                   # whole requests, adapters in any order
        cuts = torch.rand(M, generator=g, device=DEV) < 8.0 / max(M, 1)
        index = torch.randint(-1, E, (M + 1,), generator=g, device=DEV)[torch.cumsum(cuts, 0)]
    d["index"] = index.int()
    return d


def _reference(d, train=True, use_scale=True):
    """Values and tolerances by name."""
    x, A, B = (d[k].double() for k in ("x", "A", "B"))
    E, r, K = A.shape
    N, dt = B.shape[1], d["x"].dtype
    u = U[dt]
    y = torch.zeros(len(x), N, dtype=torch.double, device=DEV) if d["base"] is None else d["base"].double()
    toly = torch.zeros_like(y)
    out = {}
    if train:
        g = d["g"].double()
        gx = torch.zeros_like(x) if d["addend"] is None else d["addend"].double()
        tolx, gA, gB = torch.zeros_like(gx), torch.zeros_like(A), torch.zeros_like(B)
        tolA, tolB = torch.zeros_like(A), torch.zeros_like(B)
    for e in range(E):
        rows = (d["index"] == e).nonzero()[:, 0]
        s, n = float(d["scale"][e]) if use_scale else 1.0, len(rows)
        t = x[rows] @ A[e].T
        dt_ = u * t.abs() + 1.01 * K * 2.0 ** -23 * (x[rows].abs() @ A[e].abs().T) + TINY[dt]
        at = t.abs() + dt_
        y[rows] += s * (t @ B[e].T)
        toly[rows] = s * (dt_ @ B[e].abs().T + (r + 4) * 2.0 ** -23 * (at @ B[e].abs().T))
        if train:
            v = s * (g[rows] @ B[e])
            dv = u * v.abs() + 1.01 * N * 2.0 ** -23 * s * (g[rows].abs() @ B[e].abs()) + TINY[dt]
            av = v.abs() + dv
            gx[rows] += v @ A[e]
            tolx[rows] = dv @ A[e].abs() + (r + 4) * 2.0 ** -23 * (av @ A[e].abs())
            gA[e], gB[e] = v.T @ x[rows], s * (g[rows].T @ t)
            tolA[e] = dv.T @ x[rows].abs() + (n + 4) * 2.0 ** -23 * (av.T @ x[rows].abs())
            tolB[e] = s * (g[rows].abs().T @ dt_ + (n + 4) * 2.0 ** -23 * (g[rows].abs().T @ at))
    out["y"] = (y, toly + u * y.abs())
    if train:
        out.update(gx=(gx, tolx + u * gx.abs()), gA=(gA, tolA + u * gA.abs()), gB=(gB, tolB + u * gB.abs()))
    return out


def _run(d, train=True, use_scale=True):
    plan = I.adapter_plan(d["index"], d["A"].shape[0])
    scale = d["scale"] if use_scale else None
    y, t = I.adapters_forward(d["x"], d["A"], d["B"], scale, plan, base=d["base"])
    got = {"y": y}
    if train:
        got["gx"], got["gA"], got["gB"] = I.adapters_backward(d["g"], d["x"], t, d["A"], d["B"], scale, plan,
                                                              addend=d["addend"])
    return got


def _check(got, ref, dt):
    for k, v in got.items():
        want, tol = ref[k]
        assert v.dtype == dt and v.shape == want.shape, k
        worst = ((v.double() - want).abs() - 1.01 * tol - TINY[dt]).max() if v.numel() else 0.0
        assert float(worst) <= 0.0, f"{k}: over its tolerance by {float(worst)}"


CASES = [
    # M, K, N, r, E, order
    (1, 64, 64, 8, 1, "one"), (1, 4096, 4096, 16, 4, "one"), (7, 256, 512, 16, 64, "mixed"),
    (64, 1024, 768, 16, 64, "mixed"), (16, 2048, 256, 64, 2, "mixed"), (33, 512, 520, 32, 3, "mixed"),
    (129, 320, 1032, 24, 2, "runs"), (300, 1100, 520, 8, 5, "runs"), (300, 512, 512, 128, 2, "mixed"),
    (777, 640, 300, 12, 3, "mixed"), (640, 1024, 1536, 64, 1, "one"), (1000, 4096, 1024, 16, 8, "runs"),
    (2500, 512, 384, 48, 4, "mixed"), (1500, 256, 256, 16, 200, "mixed"), (1025, 8192, 64, 16, 2, "runs"),
    # odd sizes: rows on no 16-byte boundary
    (5, 37, 41, 3, 2, "mixed"), (130, 1101, 519, 5, 3, "mixed"), (257, 100, 2049, 1, 2, "runs"),
    (1, 1, 1, 1, 1, "one"), (200, 130, 66, 127, 2, "runs"),
    # nothing to do for some or all
    (90, 256, 128, 16, 4, "none"), (400, 256, 128, 16, 3, "one"),
]


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("M,K,N,r,E,order", CASES)
def test_forward_and_backward(M, K, N, r, E, order, dt):
    d = _data(M, K, N, r, E, dt, order, seed=M + K)
    _check(_run(d), _reference(d), dt)


# long batches: tiles of two accumulators, strips of 256 columns
LONG = [(6500, 256, 320, 16, 3, "mixed"), (6144, 512, 264, 64, 1, "one"), (7001, 320, 384, 128, 2, "runs"),
        (6300, 2056, 2048, 8, 5, "runs"), (6200, 1024, 2048, 72, 5, "mixed"), (6400, 130, 77, 12, 2, "mixed"),
        (6500, 128, 128, 16, 300, "mixed"), (6145, 9736, 72, 16, 1, "one")]


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("M,K,N,r,E,order", LONG)
def test_long_batches(M, K, N, r, E, order, dt):
    d = _data(M, K, N, r, E, dt, order, seed=M + K)
    _check(_run(d), _reference(d), dt)


# more strips of 128 columns than CTAs: adapters without tokens among others
@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("M,K,N,r,E,order", [(1500, 2056, 4104, 64, 24, "runs"), (900, 4104, 1032, 128, 40, "mixed"),
                                             (2000, 1544, 2048, 8, 70, "runs"), (300, 520, 4360, 24, 200, "one")])
def test_many_strips(M, K, N, r, E, order, dt):
    d = _data(M, K, N, r, E, dt, order, seed=M + N)
    got, want = _run(d), _reference(d)
    _check(got, want, dt)
    _, t = I.adapters_forward(d["x"], d["A"], d["B"], d["scale"], I.adapter_plan(d["index"], E))
    for need in ("gA", "gB"):               # one gradient alone: the same bits
        some = I.adapters_backward(d["g"], d["x"], t, d["A"], d["B"], d["scale"], I.adapter_plan(d["index"], E),
                                   need_x=False, need_A=need == "gA", need_B=need == "gB")
        assert torch.equal(some[1 if need == "gA" else 2], got[need])


@pytest.mark.parametrize("M", [40, 700])
def test_absent_base_addend_and_scale(M):
    d = _data(M, 512, 384, 16, 3, BF16, "mixed", 4)
    d["base"] = d["addend"] = None
    _check(_run(d, use_scale=False), _reference(d, use_scale=False), BF16)


@pytest.mark.parametrize("M", [40, 700])
def test_one_adapter_without_an_index(M):
    d = _data(M, 512, 384, 16, 1, F16, "one", 4)
    plan = I.adapter_plan(None, 1, M, DEV)
    y, t = I.adapters_forward(d["x"], d["A"], d["B"], d["scale"], plan, base=d["base"])
    g = I.adapters_backward(d["g"], d["x"], t, d["A"], d["B"], d["scale"], plan, addend=d["addend"])
    _check(dict(y=y, gx=g[0], gA=g[1], gB=g[2]), _reference(d), F16)


@pytest.mark.parametrize("M,K", [(24, 512), (600, 512), (90, 333)])
def test_parts_in_place_streams_and_repeats(M, K):
    d = _data(M, K, 640, 16, 3, BF16, "mixed", 6)
    whole = _run(d)
    again = _run(d)
    assert all(torch.equal(whole[k], again[k]) for k in whole)
    plan = I.adapter_plan(d["index"], 3)
    _, t = I.adapters_forward(d["x"], d["A"], d["B"], d["scale"], plan)
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1)):
        some = I.adapters_backward(d["g"], d["x"] if need[1] else None, t if need[2] else None, d["A"], d["B"],
                                   d["scale"], plan, addend=d["addend"], need_x=need[0], need_A=need[1],
                                   need_B=need[2])
        for n, s, k in zip(need, some, ("gx", "gA", "gB")):
            assert (s is None) == (not n) and (s is None or torch.equal(s, whole[k]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _run(d)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(whole[k], other[k]) for k in whole)
    wide = torch.zeros(M, K + 9, dtype=BF16, device=DEV)
    wide[:, 5:5 + K] = d["x"]
    y, _ = I.adapters_forward(wide[:, 5:5 + K], d["A"], d["B"], d["scale"], plan, base=d["base"])
    assert torch.equal(y, whole["y"])
    y, _ = I.adapters_forward(d["x"], d["A"], d["B"], d["scale"], plan, base=d["base"], out=d["base"])
    assert y is d["base"] and torch.equal(y, whole["y"])                  # in place


@pytest.mark.parametrize("M", [24, 600])
def test_non_finite_tokens_stay_in_their_rows(M):
    d = _data(M, 512, 640, 16, 3, F16, "mixed", 7)
    d["index"][:4] = torch.tensor([0, 1, 2, -1], device=DEV)
    clean = _run(d, train=False)["y"]
    d["x"][1, 3] = float("inf")
    d["x"][3, 9] = float("nan")                 # a token without an adapter: its x is not used
    y = _run(d, train=False)["y"]
    keep = torch.arange(M, device=DEV) != 1
    assert torch.equal(y[keep], clean[keep]) and not y[1].isfinite().all()


@pytest.mark.parametrize("K", [512, 77])
def test_no_tokens(K):
    d = _data(0, K, 24, 8, 3, F16)
    got = _run(d)
    assert got["y"].shape == (0, 24) and got["gx"].shape == (0, K) and not got["gA"].any() and not got["gB"].any()


def test_offsets_past_32_bits():
    """Tokens whose rows start past 2^31 elements."""
    M, K, N, r = 270000, 64, 8192, 8
    d = _data(8, K, N, r, 2, BF16, "mixed", 3)
    d["index"][:] = 1
    x = torch.zeros(M, K, dtype=BF16, device=DEV)
    x[-8:] = d["x"]
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    index[-8:] = 1
    plan = I.adapter_plan(index, 2)
    y, t = I.adapters_forward(x, d["A"], d["B"], d["scale"], plan)
    assert not y[:-8].any()
    small = dict(d, base=None, addend=None)
    ref = _reference(small)
    _check({"y": y[-8:]}, ref, BF16)
    y.zero_()
    y[-8:] = d["g"]
    gx, gA, gB = I.adapters_backward(y, x, t, d["A"], d["B"], d["scale"], plan)
    _check({"gx": gx[-8:], "gA": gA, "gB": gB}, ref, BF16)
    assert not gx[:-8].any() and not gA[0].any() and not gB[0].any()


def test_plan_sorts_stably():
    index = torch.tensor([2, -1, 0, 2, 7, 0, 2, 1, -5], dtype=torch.int32, device=DEV)
    plan = I.adapter_plan(index, 3)
    words = plan.data.view(torch.int32)
    assert words[:5].tolist() == [0, 2, 3, 6, 9]
    assert words[64:73].tolist() == [2, 5, 7, 0, 3, 6, 1, 4, 8]


def test_autograd_against_differences():
    """Gradients along random directions against central differences of the
    64-bit forward; the fp16 products are off by 2^-10 of their terms."""
    M, K, N, r, E = 40, 96, 64, 8, 2
    d = _data(M, K, N, r, E, F16, "mixed", 9)

    class Base(torch.nn.Module):
        in_features, out_features = K, N

        def forward(self, x):
            return x @ d["addend"][:N % K + 1].sum(0)[:, None].expand(K, N) * 0.01

    layer = I.LowRankAdapters(Base(), r, E, device=DEV, dtype=F16)
    with torch.no_grad():
        layer.A.copy_(d["A"]), layer.B.copy_(d["B"]), layer.scale.copy_(d["scale"])
    plan = I.adapter_plan(d["index"], E)
    x = d["x"].clone().requires_grad_(True)
    y = layer(x, plan)
    y.backward(d["g"])
    Wb = (d["addend"][:N % K + 1].sum(0)[:, None].expand(K, N)).double() * 0.01

    def loss(dx, dA, dB):
        xx = d["x"].double() + dx
        A, B = d["A"].double() + dA, d["B"].double() + dB
        y = xx @ Wb
        for e in range(E):
            sel = (d["index"] == e)[:, None]
            y = y + float(d["scale"][e]) * torch.where(sel, xx, 0.0) @ A[e].T @ B[e].T
        return (y * d["g"].double()).sum()

    gen = _gen(2)
    for which, grad in enumerate((x.grad, layer.A.grad, layer.B.grad)):
        v = torch.randn(grad.shape, generator=gen, device=DEV).double()
        h = [0.0, 0.0, 0.0]
        h[which] = 1e-3 * v
        diff = float((loss(*h) - loss(*[-w for w in h])) / 2e-3)
        assert abs(float((grad.double() * v).sum()) - diff) <= 2.0 ** -10 * float((grad.double() * v).abs().sum())


def test_refusals():
    d = _data(6, 32, 24, 8, 2, F16)
    plan = I.adapter_plan(d["index"], 2)
    x, A, B, s = d["x"], d["A"], d["B"], d["scale"]
    y, t = I.adapters_forward(x, A, B, s, plan)
    f, b = I.adapters_forward, I.adapters_backward
    g = d["g"]
    for call in (lambda: f(x.cpu(), A, B, s, plan), lambda: f(x[:5], A, B, s, plan), lambda: f(x[:, :30], A, B, s, plan),
                 lambda: f(x.bfloat16(), A, B, s, plan), lambda: f(x.float(), A.float(), B.float(), s, plan),
                 lambda: f(x, A, B[:, :, :4], s, plan), lambda: f(x, A[0], B[0], s, plan),
                 lambda: f(x, A, B, s.half(), plan), lambda: f(x, A, B, s[:1], plan),
                 lambda: f(x, A[:1], B[:1], s[:1], plan), lambda: f(x, A, B, s, plan, base=x),
                 lambda: f(x, A, B, s, plan, out=torch.empty(24, 6, dtype=F16, device=DEV).t()),
                 lambda: f(x, torch.zeros(2, 129, 32, dtype=F16, device=DEV),
                           torch.zeros(2, 24, 129, dtype=F16, device=DEV), s, plan),
                 lambda: I.adapter_plan(d["index"].long(), 2), lambda: I.adapter_plan(d["index"], 0),
                 lambda: I.adapter_plan(d["index"].cpu(), 2), lambda: I.adapter_plan(None, 2),
                 lambda: I.adapter_plan(None, 2, 5, "cpu"), lambda: I.adapter_plan(d["index"], 2, tokens=5),
                 lambda: b(g, None, t, A, B, s, plan), lambda: b(g, x, None, A, B, s, plan),
                 lambda: b(g[:, :20], x, t, A, B, s, plan), lambda: b(g, x, t[:, :4], A, B, s, plan),
                 lambda: b(g, x, t, A, B, s, plan, addend=g)):
        with pytest.raises(I.I8LTError):
            call()
