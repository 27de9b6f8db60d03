"""The block-scaled FP8 layer in 64 bits (plain, on the CPU) and the bounds its
outputs are held to."""
from __future__ import annotations

import torch

BLK = 128
HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def e4m3(v: torch.Tensor) -> torch.Tensor:
    """The E4M3 values nearest to v (float64), ties to even, at most 448."""
    e = torch.frexp(v)[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return torch.where(v.isnan(), v, (torch.round(v / step) * step).clamp(-448, 448))


def _codes_scales(blocks: torch.Tensor, dims):
    a = blocks.abs().amax(dims, keepdim=True)        # a NaN stays one
    r = torch.where(a >= 2.0 ** -100, 448.0 / a, torch.zeros_like(a)).float().double()
    s = (a * float(torch.tensor(1 / 448, dtype=torch.float32))).float().double()
    return e4m3((blocks * r).float().double()), s


def _padded(x, rows, cols):
    out = torch.zeros(-(-x.shape[0] // rows) * rows, -(-x.shape[1] // cols) * cols, dtype=torch.float64)
    out[:x.shape[0], :x.shape[1]] = x
    return out


def rows(x: torch.Tensor):
    """(codes [M, C], scales [C / 128, M]) of tokens."""
    M, C = x.shape
    X = _padded(x.double().cpu(), 1, BLK).view(M, -1, BLK)
    q, s = _codes_scales(X, 2)
    return q.view(M, -1)[:, :C], s[..., 0].T


def weight(W: torch.Tensor):
    """(codes [N, K], scales [N / 128, K / 128])."""
    N, K = W.shape
    X = _padded(W.double().cpu(), BLK, BLK)
    X = X.view(X.shape[0] // BLK, BLK, X.shape[1] // BLK, BLK)
    q, s = _codes_scales(X, (1, 3))
    return q.reshape(X.shape[0] * BLK, -1)[:N, :K], s[:, 0, :, 0]


def expand_rows(q, s):
    return q * s.T.repeat_interleave(BLK, 1)[:, :q.shape[1]]


def expand_weight(q, s):
    return q * s.repeat_interleave(BLK, 0)[:q.shape[0]].repeat_interleave(BLK, 1)[:, :q.shape[1]]


def product(x, W, bias=None, transposed=False):
    """(y, sum of the magnitudes of the terms) of x W^T, or x W, in 64 bits
    from the rounded operands; W: float64 [N, K] as the codes stand for it."""
    X = expand_rows(*rows(x))
    Wt = W if transposed else W.T
    y, size = X @ Wt, X.abs() @ Wt.abs()
    if bias is not None:
        y, size = y + bias.double().cpu(), size + bias.double().cpu().abs()
    return y, size


def bound(y, size, C, dtype):
    """Half a step of the output; for the sums in 32 bits: 128 products of a
    block in any order, each addition off by a step of 2^-23 of what is summed,
    and the blocks' sums, two products and an addition of 2^-24 each."""
    blocks = -(-C // BLK)
    sums = size * (128 * 2.0 ** -23 + (blocks + 4) * 2.0 ** -24)
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]
    return sums + (y.abs() + sums) * HALF_ULP[dtype] + tiny


def check(got, y, size, C, what=""):
    err = (got.double().cpu() - y).abs()
    lim = bound(y, size, C, got.dtype)
    assert bool((err <= lim).all()), f"{what}: worst {float((err / lim).max())} of the bound, {int((err > lim).sum())} beyond"
