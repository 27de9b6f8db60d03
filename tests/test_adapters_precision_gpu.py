"""Low-rank adapters: how much of an output's error is its own last rounding.

t and u are kept as two 16-bit parts, the second of what the first left over
(in fp16 times 2^11).  With u the type's unit roundoff the pair is off by at
most u^2 |t|, in fp16 by 2^-36 more (half the last place of an fp16 number,
2^-25, over 2^11).  So every output's error is its last rounding:

* norm-wise, e0 = |round(exact) - exact| is the error that any result in the
  type has.  The fp32 sums add an error that is independent of it.  A sum of n
  <= 4096 terms of mixed signs on the tensor cores makes at most n / 16
  additions, each off by 2^-23 of a partial sum no larger than about the
  result: 2^-15 of it, against e0 >= 0.3 * 2^-11.  2^-15 is a fifth of that and
  in quadrature adds 2 %; the pair's own error is smaller still.  5 % are
  allowed.  A t of one part would add an error as large as e0: 41 %.
* element by element, a sum of K products is off by K 2^-23 of their
  magnitudes, and the second product sees r of them twice."""
import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300.build import build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F16: 2.0 ** -24, BF16: 2.0 ** -126}
LAST = {F16: 2.0 ** -36, BF16: 2.0 ** -126}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _data(M, K, N, r, E, dt, seed, x=1.0, A=None, B=0.3, g=1.0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dt)

    d = dict(x=normal(M, K, std=x), A=normal(E, r, K, std=K ** -0.5 if A is None else A), B=normal(E, N, r, std=B),
             g=normal(M, N, std=g), scale=0.5 + torch.rand(E, generator=gen, device=DEV))
    d["index"] = torch.randint(0, E, (M,), generator=gen, device=DEV).int()
    if E > 1 and M > 300:                   # whole requests
        d["index"] = d["index"].sort()[0]
    return d


def _run(d):
    plan = I.adapter_plan(d["index"], d["A"].shape[0])
    y, t = I.adapters_forward(d["x"], d["A"], d["B"], d["scale"], plan)
    gx, gA, gB = I.adapters_backward(d["g"], d["x"], t, d["A"], d["B"], d["scale"], plan)
    return dict(y=y, gx=gx, gA=gA, gB=gB)


def _exact(d):
    """The outputs without base and addend, and the tolerances of y and gx."""
    x, A, B, g = (d[k].double() for k in ("x", "A", "B", "g"))
    E, r, K = A.shape
    N, dt = B.shape[1], d["x"].dtype
    y, gx, gA, gB = g.clone().zero_(), x.clone().zero_(), A.clone().zero_(), B.clone().zero_()
    toly, tolx = y.clone(), gx.clone()
    for e in range(E):
        m = (d["index"] == e).nonzero()[:, 0]
        s = float(d["scale"][e])
        t, v = x[m] @ A[e].T, s * (g[m] @ B[e])
        y[m], gx[m], gA[e], gB[e] = s * (t @ B[e].T), v @ A[e], v.T @ x[m], s * (g[m].T @ t)
        dt_ = U[dt] ** 2 * t.abs() + 1.01 * K * 2.0 ** -23 * (x[m].abs() @ A[e].abs().T) + LAST[dt]
        dv = U[dt] ** 2 * v.abs() + 1.01 * N * 2.0 ** -23 * s * (g[m].abs() @ B[e].abs()) + LAST[dt]
        n = (2 * r + 4) * 2.0 ** -23
        toly[m] = s * (dt_ @ B[e].abs().T + n * ((t.abs() + dt_) @ B[e].abs().T))
        tolx[m] = dv @ A[e].abs() + n * ((v.abs() + dv) @ A[e].abs())
    return dict(y=y, gx=gx, gA=gA, gB=gB), dict(y=toly + U[dt] * y.abs(), gx=tolx + U[dt] * gx.abs())


def _check(d, names=("y", "gx", "gA", "gB")):
    dt = d["x"].dtype
    got, (want, tol) = _run(d), _exact(d)
    for k in names:
        e0 = float((want[k].to(dt).double() - want[k]).norm())
        e = float((got[k].double() - want[k]).norm())
        assert e <= 1.05 * e0, f"{k}: {e / e0:.3f} of the error of its last rounding"
        if k in tol:
            worst = float(((got[k].double() - want[k]).abs() - 1.01 * tol[k] - TINY[dt]).max())
            assert worst <= 0.0, f"{k}: over its tolerance by {worst}"


# every way to the outputs: one launch for few tokens, boxes, gathered rows,
# rows on 8, 4 and 2 bytes; ranks in one block of 64 and in two
SIZES = [(64, 512, 640, 16, 8), (200, 256, 384, 64, 2), (256, 256, 256, 128, 1), (640, 512, 640, 64, 1),
         (2000, 1024, 1032, 16, 4), (250, 264, 520, 24, 40), (700, 256, 512, 128, 2), (513, 1100, 516, 12, 3),
         (333, 518, 642, 6, 2), (333, 641, 517, 5, 2), (300, 520, 392, 100, 3), (3000, 136, 200, 72, 2)]


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("M,K,N,r,E", SIZES)
def test_outputs_are_off_by_their_last_rounding(M, K, N, r, E, dt):
    _check(_data(M, K, N, r, E, dt, M + r))


# Second factors and gradients so small that t and u fall to fp16's smallest
# numbers (2^-24 = 6e-8): the outputs sum thousands of them, or multiply them
# by large values, and are well inside the type's range.
@pytest.mark.parametrize("u", [1e-4, 1e-5, 1e-6, 1e-7])
@pytest.mark.parametrize("M,K,N,r,E", [(4096, 256, 512, 64, 1), (4000, 320, 512, 16, 3), (3000, 256, 384, 128, 2),
                                       (2000, 520, 256, 64, 24), (2000, 258, 514, 10, 2), (1000, 257, 511, 7, 2)])
def test_small_u_in_fp16(M, K, N, r, E, u):
    """u = s g B of about `u` gives gA and gx."""
    d = _data(M, K, N, r, E, F16, r, A=4.0, B=1e-3, g=u / (1e-3 * N ** 0.5))
    _check(d, ("gA", "gx"))


@pytest.mark.parametrize("t", [1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("M,K,N,r,E", [(100, 256, 512, 64, 4), (1500, 320, 512, 16, 3), (900, 256, 384, 128, 2),
                                       (600, 258, 514, 10, 2), (600, 257, 511, 7, 2)])
def test_small_t_in_fp16(M, K, N, r, E, t):
    """t = x A of about `t` gives y and gB."""
    d = _data(M, K, N, r, E, F16, r, x=1e-2, A=100 * t * K ** -0.5, B=50.0, g=50.0)
    _check(d, ("y", "gB"))
