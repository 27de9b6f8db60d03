"""Torch-facing calls of the int8 quantized linear layer.

PyTorch supplies device memory (the caching allocator), the current stream
and autograd; every arithmetic step runs in libi8lt's CUDA kernels.  The
calls fail loudly when the library is missing or the device is not sm_103.

Method: the memory-efficient Linear8bitLt of bitsandbytes PR #33 "Memory
efficient backward" (see include/i8lt.h for the formulas).
"""
from __future__ import annotations

import array
import math
import operator
import warnings

import torch
from torch.autograd.function import once_differentiable

from . import _lib

DTYPE_CODE = {torch.float16: _lib.I8LT_F16, torch.bfloat16: _lib.I8LT_BF16, torch.float32: _lib.I8LT_F32}


class I8LTError(RuntimeError):
    pass


def _check(status: int, what: str):
    if status != _lib.I8LT_OK:
        raise I8LTError(f"{what}: {_lib.i8lt_status_string(status)} (status {status})")


def _code(dtype: torch.dtype) -> int:
    try:
        return DTYPE_CODE[dtype]
    except KeyError:
        raise I8LTError(f"unsupported dtype {dtype}") from None


def _stream(t: torch.Tensor) -> int:
    # the handle of torch.cuda.current_stream(t.device) without the object around it
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise I8LTError("libi8lt runs on CUDA tensors only (no CPU path)")


def default_max_outliers(K: int) -> int:
    """Capacity for outlier columns: all K columns, so the capacity can never
    be exceeded (the input of a second MLP layer can hold thousands of
    sporadic outlier columns).  Pass a smaller ``max_outliers`` to shrink the
    workspace (subA and subB are M x cap and N x cap fp16)."""
    return K


def weight_ld(K: int) -> int:
    return _lib.i8lt_weight_ld(K)


def quantize_weight(W: torch.Tensor):
    """W [N, K] (f16 / bf16 / f32, CUDA) -> (CB int8 [N, ld], SCB fp32 [N])."""
    _require_cuda(W)
    W = W.contiguous()
    N, K = W.shape
    CB = torch.empty(N, weight_ld(K), dtype=torch.int8, device=W.device)
    SCB = torch.empty(N, dtype=torch.float32, device=W.device)
    _check(_lib.i8lt_quantize_weight(W.data_ptr(), _code(W.dtype), N, K, CB.data_ptr(), SCB.data_ptr(),
                                     _stream(W)), "i8lt_quantize_weight")
    return CB, SCB


def forward_workspace(M: int, K: int, N: int, max_outliers: int, device) -> torch.Tensor:
    n = _lib.i8lt_forward_workspace_size(M, K, N, max_outliers)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def backward_workspace(M: int, N: int, dtype: torch.dtype, device, K: int | None = None) -> torch.Tensor:
    """Workspace of i8lt_backward_input.  Without ``K``: the fused schedule
    (the fp16 weight is rebuilt tile by tile inside the GEMM, no N x K
    buffer).  With ``K`` it has room for the materialized dequantized weight
    (K_pad x N_pad fp16), which selects the materialized schedule."""
    if K is None:
        n = _lib.i8lt_backward_workspace_size(M, N, _code(dtype))
    else:
        n = _lib.i8lt_backward_workspace_size_dq(M, N, K, _code(dtype))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def forward(A: torch.Tensor, CB: torch.Tensor, SCB: torch.Tensor, K: int, bias: torch.Tensor | None = None,
            threshold: float = 6.0, residual: torch.Tensor | None = None, max_outliers: int | None = None,
            out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
            acc_i32: torch.Tensor | None = None, merge_colmax=None, colmax_ready: bool = False):
    """out [M, N] = int8 linear of A [M, K] (see i8lt_forward).  Returns
    (out, ws); ``ws`` holds the quantized activations and the outlier set.

    ``merge_colmax``: for a token-sharded batch, a callable that receives the
    K column maxima of this call's rows (an int32 view into ``ws``, ordered
    like the magnitudes) and replaces them in place with the maxima over
    all shards, e.g. an all-reduce MAX; the outlier set is then the whole
    batch's (i8lt_forward_colmax / i8lt_forward_from_colmax).
    ``colmax_ready``: the column maxima of A are already in ``ws`` (written
    by the previous layer's forward_silu); only the rest of the forward runs."""
    _require_cuda(A, CB, SCB, bias, residual)
    A = A.contiguous()
    M = A.shape[0]
    if A.shape[1] != K:
        raise I8LTError(f"A has {A.shape[1]} features, the weight {K}")
    N = CB.shape[0]
    cap = _capacity(K, threshold, max_outliers)
    if out is None:
        out = torch.empty(M, N, dtype=A.dtype, device=A.device)
    if ws is None:
        if colmax_ready:
            raise I8LTError("colmax_ready needs the workspace that holds the column maxima")
        ws = forward_workspace(M, K, N, cap, A.device)
    if residual is not None:
        residual = residual.contiguous()
    bias_c = None if bias is None else bias.contiguous()
    args = (_ptr(bias_c), _code(bias_c.dtype) if bias_c is not None else 0, float(threshold),
            _ptr(residual), out.data_ptr(), ws.data_ptr(), ws.numel(), cap)
    if merge_colmax is None and not colmax_ready:
        _check(_lib.i8lt_forward(A.data_ptr(), _code(A.dtype), M, K, CB.data_ptr(), SCB.data_ptr(), N, *args,
                                 acc_i32=_ptr(acc_i32), stream=_stream(A)), "i8lt_forward")
        return out, ws
    if not colmax_ready:
        _check(_lib.i8lt_forward_colmax(A.data_ptr(), _code(A.dtype), M, K, N, ws.data_ptr(), ws.numel(), cap,
                                        stream=_stream(A)), "i8lt_forward_colmax")
    if merge_colmax is not None:
        lay = _lib.i8lt_forward_workspace_layout(M, K, N, cap)
        merge_colmax(ws[lay.colmax:lay.colmax + 4 * K].view(torch.int32))
    _check(_lib.i8lt_forward_from_colmax(A.data_ptr(), _code(A.dtype), M, K, CB.data_ptr(), SCB.data_ptr(), N,
                                         *args, acc_i32=_ptr(acc_i32), stream=_stream(A)),
           "i8lt_forward_from_colmax")
    return out, ws


def _capacity(K: int, threshold: float, max_outliers: int | None) -> int:
    if not (math.isfinite(threshold) and threshold > 0):
        return 0
    return default_max_outliers(K) if max_outliers is None else int(max_outliers)


def colmax_region(ws: torch.Tensor, M: int, K: int, N: int, threshold: float,
                  max_outliers: int | None = None) -> torch.Tensor:
    """The K column maxima of a forward workspace (int32 view)."""
    lay = _lib.i8lt_forward_workspace_layout(M, K, N, _capacity(K, threshold, max_outliers))
    return ws[lay.colmax:lay.colmax + 4 * K].view(torch.int32)


def forward_silu(A: torch.Tensor, CB: torch.Tensor, SCB: torch.Tensor, K: int, bias: torch.Tensor | None = None,
                 threshold: float = 6.0, max_outliers: int | None = None, act_colmax: torch.Tensor | None = None):
    """MLP hidden layer (i8lt_forward_silu): returns (h, silu(h), ws).
    ``act_colmax`` (int32 [N], e.g. ``colmax_region`` of the next layer's
    workspace) receives the column maxima of |fp16(silu(h))|."""
    _require_cuda(A, CB, SCB, bias)
    A = A.contiguous()
    M = A.shape[0]
    if A.shape[1] != K:
        raise I8LTError(f"A has {A.shape[1]} features, the weight {K}")
    N = CB.shape[0]
    cap = _capacity(K, threshold, max_outliers)
    h = torch.empty(M, N, dtype=A.dtype, device=A.device)
    a = torch.empty_like(h)
    if act_colmax is None:
        act_colmax = torch.empty(N, dtype=torch.int32, device=A.device)
    ws = forward_workspace(M, K, N, cap, A.device)
    bias_c = None if bias is None else bias.contiguous()
    _check(_lib.i8lt_forward_silu(A.data_ptr(), _code(A.dtype), M, K, CB.data_ptr(), SCB.data_ptr(), N,
                                  _ptr(bias_c), _code(bias_c.dtype) if bias_c is not None else 0, float(threshold),
                                  None, h.data_ptr(), a.data_ptr(), act_colmax.data_ptr(), ws.data_ptr(), ws.numel(),
                                  cap, stream=_stream(A)), "i8lt_forward_silu")
    return h, a, ws


def allreduce_colmax(group=None):
    """``merge_colmax`` for torch.distributed: an all-reduce MAX of the column
    maxima over ``group`` (one K-sized int32 exchange per forward)."""
    import torch.distributed as dist

    def merge(t: torch.Tensor):
        dist.all_reduce(t, op=dist.ReduceOp.MAX, group=group)
    return merge


def backward_input(G: torch.Tensor, CB: torch.Tensor, SCB: torch.Tensor, K: int, need_grad_A: bool = True,
                   bias_dtype: torch.dtype | None = None, addend: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None, fused: bool = True):
    """(grad_A [M, K] or None, grad_bias [N] or None) from grad_output G [M, N].
    ``fused`` (default): the dequantized weight is rebuilt tile by tile inside
    the GEMM and never stored.  ``fused=False``: it is first written to the
    workspace (K x N fp16) by a memory-bound prepass, then read by a plain
    fp16 GEMM -- more memory, a little faster.  A caller-supplied ``ws``
    decides by its size instead.  Both give the same bits."""
    _require_cuda(G, CB, SCB, addend)
    G = G.contiguous()
    M, N = G.shape
    grad_A = torch.empty(M, K, dtype=G.dtype, device=G.device) if need_grad_A else None
    grad_bias = torch.empty(N, dtype=bias_dtype, device=G.device) if bias_dtype is not None else None
    if ws is None:
        ws = backward_workspace(M, N, G.dtype, G.device, K=None if (fused or not need_grad_A) else K)
    if addend is not None:
        addend = addend.contiguous()
    _check(_lib.i8lt_backward_input(G.data_ptr(), _code(G.dtype), M, N, CB.data_ptr(), SCB.data_ptr(), K,
                                    _ptr(addend), _ptr(grad_A), _ptr(grad_bias),
                                    _code(bias_dtype) if bias_dtype is not None else 0,
                                    ws.data_ptr(), ws.numel(), _stream(G)), "i8lt_backward_input")
    return grad_A, grad_bias


def silu(h: torch.Tensor) -> torch.Tensor:
    _require_cuda(h)
    h = h.contiguous()
    out = torch.empty_like(h)
    _check(_lib.i8lt_silu_forward(h.data_ptr(), _code(h.dtype), h.numel(), out.data_ptr(), _stream(h)),
           "i8lt_silu_forward")
    return out


def silu_backward(g: torch.Tensor, h: torch.Tensor) -> torch.Tensor:
    _require_cuda(g, h)
    g, h = g.contiguous(), h.contiguous()
    out = torch.empty_like(h)
    _check(_lib.i8lt_silu_backward(g.data_ptr(), h.data_ptr(), _code(h.dtype), h.numel(), out.data_ptr(),
                                   _stream(h)), "i8lt_silu_backward")
    return out


def device_status(ws: torch.Tensor):
    """(status code, outlier columns found) of the last call that used ``ws``
    (synchronizes the current stream; clears a recorded error)."""
    _require_cuda(ws)
    r, st, found = _lib.i8lt_read_device_status(ws.data_ptr(), _stream(ws))
    return st, found


# ---------------------------------------------------------------------------
# autograd
# ---------------------------------------------------------------------------

_warned_cast = False


def _warn_cast(dtype):
    global _warned_cast
    if dtype != torch.float16 and not _warned_cast:
        _warned_cast = True
        warnings.warn(f"Linear8bitLt: input of dtype {dtype} is cast to float16 for the int8 "
                      "quantization; the output is cast back to the input's dtype.")


class Int8LinearFunction(torch.autograd.Function):
    """y = int8 linear(x); the weight is frozen (memory-efficient backward:
    grad to the input and the bias only)."""

    @staticmethod
    def forward(ctx, x, CB, SCB, bias, threshold, max_outliers):
        _warn_cast(x.dtype)
        shape = x.shape
        K = shape[-1]
        x2 = x.reshape(-1, K)
        out, _ = forward(x2, CB, SCB, K, bias, threshold, max_outliers=max_outliers)
        ctx.save_for_backward(CB, SCB)
        ctx.K = K
        ctx.x_shape = shape
        ctx.bias_dtype = None if bias is None else bias.dtype
        return out.reshape(*shape[:-1], CB.shape[0])

    @staticmethod
    def backward(ctx, grad_out):
        CB, SCB = ctx.saved_tensors
        need_x = ctx.needs_input_grad[0]
        need_b = ctx.needs_input_grad[3] and ctx.bias_dtype is not None
        G = grad_out.reshape(-1, grad_out.shape[-1])
        gA, gb = backward_input(G, CB, SCB, ctx.K, need_grad_A=need_x,
                                bias_dtype=ctx.bias_dtype if need_b else None)
        if gA is not None:
            gA = gA.reshape(ctx.x_shape)
        return gA, None, None, gb, None, None


def grad_weight(G: torch.Tensor, A: torch.Tensor, out_dtype: torch.dtype | None = None,
                ws: torch.Tensor | None = None) -> torch.Tensor:
    """grad_W [N, K] = G^T A over the tokens, int8 with column-wise scales
    (i8lt_grad_weight); G [M, N], A [M, K]."""
    _require_cuda(G, A)
    G, A = G.contiguous(), A.contiguous()
    M, N = G.shape
    K = A.shape[1]
    if A.shape[0] != M:
        raise I8LTError(f"G has {M} tokens, A {A.shape[0]}")
    out_dtype = out_dtype or G.dtype
    gW = torch.empty(N, K, dtype=out_dtype, device=G.device)
    if ws is None:
        ws = torch.empty(max(_lib.i8lt_grad_weight_workspace_size(M, N, K), 256), dtype=torch.uint8,
                         device=G.device)
    _check(_lib.i8lt_grad_weight(G.data_ptr(), _code(G.dtype), A.data_ptr(), _code(A.dtype), M, N, K, gW.data_ptr(),
                                 _code(out_dtype), ws.data_ptr(), ws.numel(), _stream(G)), "i8lt_grad_weight")
    return gW


class Int8LinearTrainableFunction(torch.autograd.Function):
    """y = int8 linear(x) with a trainable float weight W (bitsandbytes'
    has_fp16_weights=True): every forward quantizes W row-wise (CB, SCB) and
    runs the same int8 forward; the backward gives grad_A through the
    dequantized CB (as the memory-efficient mode does), grad_W through the
    int8 column-wise product (i8lt_grad_weight) and grad_bias."""

    @staticmethod
    def forward(ctx, x, W, bias, threshold, max_outliers):
        _warn_cast(x.dtype)
        shape = x.shape
        K = shape[-1]
        x2 = x.reshape(-1, K)
        CB, SCB = quantize_weight(W)
        out, _ = forward(x2, CB, SCB, K, bias, threshold, max_outliers=max_outliers)
        ctx.save_for_backward(x2, CB, SCB)
        ctx.K = K
        ctx.x_shape = shape
        ctx.w_dtype = W.dtype
        ctx.bias_dtype = None if bias is None else bias.dtype
        return out.reshape(*shape[:-1], CB.shape[0])

    @staticmethod
    def backward(ctx, grad_out):
        x2, CB, SCB = ctx.saved_tensors
        need_x = ctx.needs_input_grad[0]
        need_w = ctx.needs_input_grad[1]
        need_b = ctx.needs_input_grad[2] and ctx.bias_dtype is not None
        G = grad_out.reshape(-1, grad_out.shape[-1])
        gA, gb = backward_input(G, CB, SCB, ctx.K, need_grad_A=need_x,
                                bias_dtype=ctx.bias_dtype if need_b else None)
        gW = grad_weight(G, x2, ctx.w_dtype) if need_w else None
        if gA is not None:
            gA = gA.reshape(ctx.x_shape)
        return gA, gW, gb, None, None


class SiLUFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h):
        ctx.save_for_backward(h)
        return silu(h)

    @staticmethod
    def backward(ctx, g):
        (h,) = ctx.saved_tensors
        return silu_backward(g, h)


# MLP hidden layer: run the SiLU and fc2's column maxima inside fc1's GEMM
# epilogue (i8lt_forward_silu) instead of as separate passes.  Same bits
# either way.  Off by default: on GB300 the longer epilogue delays the
# GEMM's next tile about as much as the two memory-bound passes it saves
# cost (mlp_7b fc1 alone: 0.765 ms fused against 0.714 ms + 0.03 ms; the
# whole block forward + backward: 2.857 ms against 2.866 ms).
FUSED_SILU = False


class Int8MLPFunction(torch.autograd.Function):
    """y = fc2(silu(fc1(x))) (+ x): the two int8 layers, the SiLU and the
    residual add (fused into fc2's epilogue forward, and into fc1's backward
    as an addend) all in libi8lt kernels."""

    @staticmethod
    def forward(ctx, x, CB1, SCB1, b1, CB2, SCB2, b2, threshold, residual, max_outliers):
        _warn_cast(x.dtype)
        shape = x.shape
        K = shape[-1]
        x2 = x.reshape(-1, K)
        H, N2 = CB1.shape[0], CB2.shape[0]
        M = x2.shape[0]
        res = x2 if residual else None
        if FUSED_SILU:
            # fc1's epilogue applies the SiLU and writes fc2's column maxima
            # into fc2's workspace, so fc2 starts at its outlier index
            ws2 = forward_workspace(M, H, N2, _capacity(H, threshold, max_outliers), x.device)
            h, a, _ = forward_silu(x2, CB1, SCB1, K, b1, threshold, max_outliers=max_outliers,
                                   act_colmax=colmax_region(ws2, M, H, N2, threshold, max_outliers))
            y, _ = forward(a, CB2, SCB2, H, b2, threshold, residual=res, max_outliers=max_outliers, ws=ws2,
                           colmax_ready=True)
        else:
            h, _ = forward(x2, CB1, SCB1, K, b1, threshold, max_outliers=max_outliers)
            a = silu(h)
            y, _ = forward(a, CB2, SCB2, H, b2, threshold, residual=res, max_outliers=max_outliers)
        ctx.save_for_backward(CB1, SCB1, CB2, SCB2, h)
        ctx.K = K
        ctx.H = CB1.shape[0]
        ctx.shape = shape
        ctx.residual = residual
        ctx.b1_dtype = None if b1 is None else b1.dtype
        ctx.b2_dtype = None if b2 is None else b2.dtype
        return y.reshape(*shape[:-1], CB2.shape[0])

    @staticmethod
    def backward(ctx, g):
        CB1, SCB1, CB2, SCB2, h = ctx.saved_tensors
        G = g.reshape(-1, g.shape[-1])
        ga, gb2 = backward_input(G, CB2, SCB2, ctx.H, bias_dtype=ctx.b2_dtype if ctx.needs_input_grad[6] else None)
        gh = silu_backward(ga, h)
        gx, gb1 = backward_input(gh, CB1, SCB1, ctx.K, addend=G if ctx.residual else None,
                                 bias_dtype=ctx.b1_dtype if ctx.needs_input_grad[3] else None)
        return gx.reshape(ctx.shape), None, None, gb1, None, None, gb2, None, None, None


# ---------------------------------------------------------------------------
# 4-bit weight-only layers (QLoRA fine-tuning: frozen 4-bit base weights,
# 16-bit compute; NF4 and FP4 share one storage and one set of matmul
# kernels, see i8lt_nf4_forward / i8lt_fp4_forward in include/i8lt.h)
# ---------------------------------------------------------------------------

FORMATS_4BIT = ("nf4", "fp4")


def _fmt4(fmt: str) -> str:
    if fmt not in FORMATS_4BIT:
        raise I8LTError(f"unknown 4-bit format {fmt!r} (expected one of {FORMATS_4BIT})")
    return fmt


def _fn4(fmt: str, name: str):
    return getattr(_lib, f"i8lt_{_fmt4(fmt)}_{name}")


def levels_4bit(fmt: str = "nf4") -> list[float]:
    """The 16 levels of a 4-bit format, by code."""
    st, lv = _fn4(fmt, "levels")()
    _check(st, f"i8lt_{fmt}_levels")
    return lv


def nf4_levels() -> list[float]:
    return levels_4bit("nf4")


def fp4_levels() -> list[float]:
    return levels_4bit("fp4")


def quantize_4bit(W: torch.Tensor, fmt: str = "nf4"):
    """W [N, K] (f16 / bf16 / f32, CUDA) -> (packed uint8 [N, row_bytes],
    absmax fp32 [N, ceil(K / 64)]) in the 4-bit format ``fmt``."""
    _require_cuda(W)
    W = W.contiguous()
    N, K = W.shape
    packed = torch.empty(N, _lib.i8lt_nf4_row_bytes(K), dtype=torch.uint8, device=W.device)
    absmax = torch.empty(N, _lib.i8lt_nf4_blocks(K), dtype=torch.float32, device=W.device)
    _check(_fn4(fmt, "quantize")(W.data_ptr(), _code(W.dtype), N, K, packed.data_ptr(), absmax.data_ptr(),
                                 _stream(W)), f"i8lt_{fmt}_quantize")
    return packed, absmax


def nf4_quantize(W: torch.Tensor):
    return quantize_4bit(W, "nf4")


def fp4_quantize(W: torch.Tensor):
    return quantize_4bit(W, "fp4")


def dequantize_4bit(packed: torch.Tensor, absmax: torch.Tensor, K: int, dtype: torch.dtype,
                    fmt: str = "nf4") -> torch.Tensor:
    """The dequantized weight [N, K] in ``dtype``."""
    _require_cuda(packed, absmax)
    N = packed.shape[0]
    out = torch.empty(N, K, dtype=dtype, device=packed.device)
    _check(_fn4(fmt, "dequantize")(packed.data_ptr(), absmax.data_ptr(), N, K, out.data_ptr(), _code(dtype),
                                   _stream(packed)), f"i8lt_{fmt}_dequantize")
    return out


def nf4_dequantize(packed: torch.Tensor, absmax: torch.Tensor, K: int, dtype: torch.dtype) -> torch.Tensor:
    return dequantize_4bit(packed, absmax, K, dtype, "nf4")


def fp4_dequantize(packed: torch.Tensor, absmax: torch.Tensor, K: int, dtype: torch.dtype) -> torch.Tensor:
    return dequantize_4bit(packed, absmax, K, dtype, "fp4")


def double_quantize_absmax(absmax: torch.Tensor):
    """The 8-bit storage of a 4-bit weight's absmax values (the ``-dq``
    options): (q uint8 with absmax's shape, absmax2 fp32 [ceil(n / 256)],
    offset fp32 [1]) -- FP8 E4M3 codes of absmax - offset in blocks of 256
    with one fp32 scale each, offset the mean of all the values."""
    _require_cuda(absmax)
    a = absmax.contiguous()
    n = a.numel()
    q = torch.empty(a.shape, dtype=torch.uint8, device=a.device)
    a2 = torch.empty(_lib.i8lt_absmax8_blocks(n), dtype=torch.float32, device=a.device)
    off = torch.empty(1, dtype=torch.float32, device=a.device)
    ws = torch.empty(_lib.i8lt_absmax8_workspace_size(), dtype=torch.uint8, device=a.device)
    _check(_lib.i8lt_absmax8_quantize(a.data_ptr(), n, q.data_ptr(), a2.data_ptr(), off.data_ptr(), ws.data_ptr(),
                                      ws.numel(), _stream(a)), "i8lt_absmax8_quantize")
    return q, a2, off


def dequantize_absmax(q: torch.Tensor, absmax2: torch.Tensor, offset: torch.Tensor,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """The fp32 absmax values decoded from double_quantize_absmax's storage."""
    _require_cuda(q, absmax2, offset)
    q = q.contiguous()
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    _check(_lib.i8lt_absmax8_dequantize(q.data_ptr(), absmax2.data_ptr(), offset.data_ptr(), q.numel(),
                                        out.data_ptr(), _stream(q)), "i8lt_absmax8_dequantize")
    return out


def _nf4_ws(device, ws, K, N, materialized, extra=0):
    """Workspace of the 4-bit matmuls: the status word (and ``extra`` bytes
    of grad_bias partial sums), the weight then decoded inside the GEMM; or
    room for the dequantized weight after them (``materialized``: a prepass
    writes it, a plain 16-bit GEMM reads it; same bits, faster, N * K * 2
    bytes more)."""
    if ws is None:
        n = _lib.i8lt_nf4_workspace_size_dq(K, N) if materialized else _lib.i8lt_nf4_workspace_size()
        ws = torch.empty(n + extra, dtype=torch.uint8, device=device)
    return ws


def forward_4bit(A: torch.Tensor, packed: torch.Tensor, absmax: torch.Tensor, K: int,
                 bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None, materialized: bool = False, fmt: str = "nf4") -> torch.Tensor:
    """out [M, N] = A [M, K] @ Wdq^T (+ bias) in A's dtype (f16 or bf16)."""
    _require_cuda(A, packed, absmax, bias)
    A = A.contiguous()
    M = A.shape[0]
    N = packed.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=A.dtype, device=A.device)
    ws = _nf4_ws(A.device, ws, K, N, materialized)
    _check(_fn4(fmt, "forward")(A.data_ptr(), _code(A.dtype), M, K, packed.data_ptr(), absmax.data_ptr(), N,
                                _ptr(bias), _code(bias.dtype) if bias is not None else 0, out.data_ptr(),
                                ws.data_ptr(), ws.numel(), _stream(A)), f"i8lt_{fmt}_forward")
    return out


def nf4_forward(A, packed, absmax, K, bias=None, out=None, ws=None, materialized=False) -> torch.Tensor:
    return forward_4bit(A, packed, absmax, K, bias, out, ws, materialized, "nf4")


def fp4_forward(A, packed, absmax, K, bias=None, out=None, ws=None, materialized=False) -> torch.Tensor:
    return forward_4bit(A, packed, absmax, K, bias, out, ws, materialized, "fp4")


def backward_input_4bit(G: torch.Tensor, packed: torch.Tensor, absmax: torch.Tensor, K: int,
                        need_grad_A: bool = True, bias_dtype: torch.dtype | None = None,
                        out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                        materialized: bool = False, fmt: str = "nf4"):
    """(grad_A [M, K] = G [M, N] @ Wdq in G's dtype (f16 or bf16) or None,
    grad_bias [N] in ``bias_dtype`` or None).  grad_bias is reduced inside
    the GEMM (or by a pass of its own when grad_A is not needed)."""
    _require_cuda(G, packed, absmax)
    G = G.contiguous()
    M, N = G.shape
    if need_grad_A and out is None:
        out = torch.empty(M, K, dtype=G.dtype, device=G.device)
    gb = torch.empty(N, dtype=bias_dtype, device=G.device) if bias_dtype is not None else None
    extra = _lib.i8lt_nf4_grad_bias_bytes(M, N) if gb is not None else 0
    ws = _nf4_ws(G.device, ws, K, N, materialized, extra)
    _check(_fn4(fmt, "backward_input")(G.data_ptr(), _code(G.dtype), M, N, packed.data_ptr(), absmax.data_ptr(), K,
                                       _ptr(out) if need_grad_A else None, _ptr(gb),
                                       _code(bias_dtype) if bias_dtype is not None else 0, ws.data_ptr(), ws.numel(),
                                       _stream(G)), f"i8lt_{fmt}_backward_input")
    return (out if need_grad_A else None), gb


def nf4_backward_input(G, packed, absmax, K, out=None, ws=None, materialized=False) -> torch.Tensor:
    """grad_A [M, K] = G [M, N] @ Wdq in G's dtype (f16 or bf16)."""
    return backward_input_4bit(G, packed, absmax, K, out=out, ws=ws, materialized=materialized, fmt="nf4")[0]


def fp4_backward_input(G, packed, absmax, K, out=None, ws=None, materialized=False) -> torch.Tensor:
    return backward_input_4bit(G, packed, absmax, K, out=out, ws=ws, materialized=materialized, fmt="fp4")[0]


class Linear4bitFunction(torch.autograd.Function):
    """y = x @ Wdq^T + bias with the frozen 4-bit weight (format ``fmt``)
    decoded inside the matmuls; gradients to x and to the bias (summed over
    the tokens inside the input-gradient GEMM)."""

    @staticmethod
    def forward(ctx, x, packed, absmax, K, bias, materialized=False, fmt="nf4"):
        shape = x.shape
        x2 = x.reshape(-1, K)
        y = forward_4bit(x2, packed, absmax, K, bias, materialized=materialized, fmt=fmt)
        ctx.save_for_backward(packed, absmax)
        ctx.K, ctx.shape, ctx.materialized, ctx.fmt = K, shape, materialized, fmt
        ctx.bias_dtype = bias.dtype if bias is not None else None
        return y.reshape(*shape[:-1], packed.shape[0])

    @staticmethod
    def backward(ctx, gy):
        packed, absmax = ctx.saved_tensors
        g2 = gy.reshape(-1, packed.shape[0])
        need_x = ctx.needs_input_grad[0]
        need_b = ctx.bias_dtype is not None and ctx.needs_input_grad[4]
        if not (need_x or need_b):
            return None, None, None, None, None, None, None
        gx, gb = backward_input_4bit(g2, packed, absmax, ctx.K, need_grad_A=need_x,
                                     bias_dtype=ctx.bias_dtype if need_b else None,
                                     materialized=ctx.materialized, fmt=ctx.fmt)
        if gx is not None:
            gx = gx.reshape(ctx.shape)
        return gx, None, None, None, gb, None, None


# the NF4 layer's function under its own name
NF4LinearFunction = Linear4bitFunction


# ---------------------------------------------------------------------------
# fine-tuning on top of the frozen layers: layer norm, low-rank adapters, AdamW
# ---------------------------------------------------------------------------

def _aligned(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy of it that is contiguous and starts on 16 bytes, as the
    library wants it: views need not (x[1:] of odd rows, the parts of a
    gradient that torch.cat's backward hands on)."""
    if not t.is_contiguous():
        return t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _checked(what: str, t: torch.Tensor, dev: int, shape, dtype) -> torch.Tensor:
    """t, on CUDA device ``dev``, of ``shape`` and of ``dtype`` (None: any)."""
    if t.get_device() != dev:
        raise I8LTError(f"{what}: a tensor on {t.device}, expected cuda:{dev}" if t.is_cuda else
                        "libi8lt runs on CUDA tensors only (no CPU path)")
    if t.shape != shape:
        raise I8LTError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise I8LTError(f"{what}: dtype {t.dtype}, expected {dtype}")
    return t


def _arg(what: str, t, dev: int, shape, dtype):
    """An optional input after its checks, as the library wants it."""
    return None if t is None else _aligned(_checked(what, t, dev, shape, dtype))


def _out(what: str, t: torch.Tensor, dev: int, shape, dtype):
    """A caller's output buffer after its checks (the library refuses one that
    does not start on 16 bytes)."""
    if not t.is_contiguous():
        raise I8LTError(f"{what}: not contiguous")
    return _checked(what, t, dev, shape, dtype)


def _workspace(what: str, ws, size: int, device) -> torch.Tensor:
    """The caller's workspace after its checks (the library checks its size),
    or a new one."""
    if ws is None:
        return torch.empty(max(size, 256), dtype=torch.uint8, device=device)
    if ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise I8LTError(f"{what}: a workspace is a contiguous uint8 tensor on {device}")
    return ws


# Tells autograd that tensors were written in place: a backward pass that
# still needs what they held then raises instead of using what they hold now.
_written = torch.autograd.graph.increment_version


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5, out: torch.Tensor | None = None):
    """(y, mean, rstd) of the layer norm over the last dimension of x [..., N]
    (f16 / bf16 / f32); weight and bias [N] of one dtype (any of the three).
    mean and rstd are fp32 with x's leading shape, for the backward.  ``out``
    may be x itself."""
    _require_cuda(x)
    shape = x.shape
    if not shape:
        raise I8LTError("layer_norm: x has no dimension to normalise")
    dev, dtype, N = x.get_device(), x.dtype, shape[-1]
    x = _aligned(x)
    weight = _arg("layer_norm weight", weight, dev, (N,), None)
    par = weight if weight is not None else bias
    bias = _arg("layer_norm bias", bias, dev, (N,), None if par is None else par.dtype)
    y = torch.empty_like(x) if out is None else _out("layer_norm out", out, dev, shape, dtype)
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    _check(_lib.i8lt_layer_norm_forward(x.data_ptr(), _code(dtype), mean.numel(), N, _ptr(weight), _ptr(bias),
                                        0 if par is None else _code(par.dtype), eps, y.data_ptr(), mean.data_ptr(),
                                        rstd.data_ptr(), _stream(x)), "i8lt_layer_norm_forward")
    if out is not None:
        _written(out)
    return y, mean, rstd


def layer_norm_backward(g: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, need_x: bool = True, need_weight: bool = True,
                        need_bias: bool = True, param_dtype: torch.dtype | None = None,
                        ws: torch.Tensor | None = None):
    """(gx, gw, gb) of ``layer_norm`` (None where not needed).  gw and gb have
    ``param_dtype`` (default: weight's, else x's).  ``ws``: a workspace of
    i8lt_layer_norm_backward_workspace_size bytes, for a caller that reads its
    ``device_status``."""
    _require_cuda(x)
    shape = x.shape
    dev, dtype, N = x.get_device(), x.dtype, shape[-1]
    x = _aligned(x)
    g = _arg("layer_norm_backward g", g, dev, shape, dtype)
    mean = _arg("layer_norm_backward mean", mean, dev, shape[:-1], torch.float32)
    rstd = _arg("layer_norm_backward rstd", rstd, dev, shape[:-1], torch.float32)
    weight = _arg("layer_norm_backward weight", weight, dev, (N,), None)
    if weight is None:
        ptype = param_dtype or dtype
    elif param_dtype not in (None, weight.dtype):
        raise I8LTError(f"layer_norm_backward: param_dtype {param_dtype} with a weight of {weight.dtype}")
    else:
        ptype = weight.dtype
    if not (need_x or need_weight or need_bias):
        return None, None, None
    M = x.numel() // N if N else 0
    gx = torch.empty_like(x) if need_x else None
    gw = torch.empty(N, dtype=ptype, device=x.device) if need_weight else None
    gb = torch.empty(N, dtype=ptype, device=x.device) if need_bias else None
    n = _lib.i8lt_layer_norm_backward_workspace_size(M, N)
    ws = _workspace("layer_norm_backward", ws, n, x.device)
    _check(_lib.i8lt_layer_norm_backward(g.data_ptr(), x.data_ptr(), _code(dtype), M, N, mean.data_ptr(),
                                         rstd.data_ptr(), _ptr(weight), _code(ptype), _ptr(gx), _ptr(gw), _ptr(gb),
                                         ws.data_ptr(), ws.numel(), _stream(x)), "i8lt_layer_norm_backward")
    return gx, gw, gb


class LayerNormFunction(torch.autograd.Function):
    """y = layer norm of x over its last dimension."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.param_dtype = None if bias is None or weight is not None else bias.dtype
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        gx, gw, gb = layer_norm_backward(g, x, mean, rstd, weight, need_x=need[0],
                                         need_weight=need[1] and weight is not None,
                                         need_bias=need[2] and ctx.has_bias, param_dtype=ctx.param_dtype)
        return gx, gw, gb, None


class AdapterPlan:
    """The tokens of a batch sorted by adapter (``adapter_plan``): made once
    per batch, used by every layer and both directions."""

    def __init__(self, data: torch.Tensor, tokens: int, adapters: int):
        self.data, self.tokens, self.adapters = data, tokens, adapters


def adapter_plan(index: torch.Tensor | None, adapters: int, tokens: int | None = None,
                 device=None) -> AdapterPlan:
    """The plan of a batch whose token m uses adapter index[m] (int32; a value
    outside [0, adapters) uses none).  index None: ``tokens`` tokens on
    ``device`` that all use adapter 0."""
    if index is None:
        if tokens is None or device is None:
            raise I8LTError("adapter_plan: without an index it needs tokens and device")
        device = torch.device(device)
        if device.type != "cuda":
            raise I8LTError("libi8lt runs on CUDA tensors only (no CPU path)")
        M = int(tokens)
    else:
        _require_cuda(index)
        if index.dtype != torch.int32:
            raise I8LTError(f"adapter_plan: index has dtype {index.dtype}, expected torch.int32")
        if not index.is_contiguous():
            index = index.contiguous()
        M, device = index.numel(), index.device
        if tokens is not None and tokens != M:
            raise I8LTError(f"adapter_plan: {M} indices for {tokens} tokens")
    n = _lib.i8lt_adapter_plan_bytes(M, adapters)
    data = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
    _check(_lib.i8lt_adapter_plan(_ptr(index), M, adapters, data.data_ptr(), data.numel(), _stream(data)),
           "i8lt_adapter_plan")
    return AdapterPlan(data, M, adapters)


def _adapter_args(what, tokens, A, B, scale, plan):
    """(device, M, K, E, r, N, A, B, scale) of an adapter call, checked, on
    tokens [M, K or N]."""
    _require_cuda(tokens, plan.data)
    dev, dtype = tokens.get_device(), tokens.dtype
    if tokens.dim() != 2:
        raise I8LTError(f"{what}: {tokens.dim()}-dimensional tokens, expected [tokens, features]")
    if A.dim() != 3 or B.dim() != 3:
        raise I8LTError(f"{what}: A and B are [adapters, rank, in] and [adapters, out, rank]")
    E, r, K = A.shape
    N, M = B.shape[1], tokens.shape[0]
    if plan.adapters != E or plan.tokens != M or plan.data.get_device() != dev:
        raise I8LTError(f"{what}: a plan of {plan.tokens} tokens and {plan.adapters} adapters on {plan.data.device} "
                        f"for {M} tokens and {E} adapters on {tokens.device}")
    A = _arg(f"{what} A", A, dev, A.shape, dtype)
    B = _arg(f"{what} B", B, dev, (E, N, r), dtype)
    return dev, M, K, E, r, N, A, B, _arg(f"{what} scale", scale, dev, (E,), torch.float32)


def adapters_forward(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor | None,
                     plan: AdapterPlan, base: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None):
    """(y, t) with t = x A[e]^T and y = base + scale[e] t B[e]^T for each
    token's adapter e (i8lt_adapters_forward): x [M, K] (f16 / bf16),
    A [E, r, K], B [E, N, r], scale fp32 [E] or None, base [M, N] or None.
    ``out`` may be base itself (not x).  t [2, M, r], two 16-bit parts of one
    value with the tokens in the plan's order, is what the backward needs.
    ``ws``: a workspace of i8lt_adapters_workspace_size bytes, for a caller
    that reads its ``device_status``."""
    what = "adapters_forward"
    dev, M, K, E, r, N, A, B, scale = _adapter_args(what, x, A, B, scale, plan)
    dtype, device = x.dtype, x.device
    x = _arg(what, x, dev, (M, K), None)
    base = _arg("adapters_forward base", base, dev, (M, N), dtype)
    if out is not None:
        y = _out("adapters_forward out", out, dev, (M, N), dtype)
    else:
        y = torch.empty((M, N), dtype=dtype, device=device) if base is None else torch.empty_like(base)
    t = torch.empty((2, M, r), dtype=dtype, device=device)
    ws = _workspace(what, ws, _lib.i8lt_adapters_workspace_size(M, K, N, E, r), device)
    _check(_lib.i8lt_adapters_forward(x.data_ptr(), _code(dtype), M, K, A.data_ptr(), B.data_ptr(), E, r, N,
                                      _ptr(scale), plan.data.data_ptr(), _ptr(base), y.data_ptr(), t.data_ptr(),
                                      ws.data_ptr(), ws.numel(), _stream(x)), "i8lt_adapters_forward")
    if out is not None:
        _written(out)
    return y, t


def adapters_backward(g: torch.Tensor, x: torch.Tensor | None, t: torch.Tensor | None, A: torch.Tensor,
                      B: torch.Tensor, scale: torch.Tensor | None, plan: AdapterPlan,
                      addend: torch.Tensor | None = None, need_x: bool = True, need_A: bool = True,
                      need_B: bool = True, ws: torch.Tensor | None = None):
    """(gx, gA, gB) of ``adapters_forward`` (None where not needed), gx with
    ``addend`` (the shared projection's input gradient) added.  x is used for
    gA only, t for gB only; ``ws`` as in ``adapters_forward``."""
    what = "adapters_backward"
    dev, M, K, E, r, N, A, B, scale = _adapter_args(what, g, A, B, scale, plan)
    if need_A and x is None or need_B and t is None:
        raise I8LTError("adapters_backward: gA needs x and gB needs t")
    dtype, device = g.dtype, g.device
    g = _arg("adapters_backward g", g, dev, (M, N), None)
    x = _arg("adapters_backward x", x, dev, (M, K), dtype)
    t = _arg("adapters_backward t", t, dev, (2, M, r), dtype)
    addend = _arg("adapters_backward addend", addend, dev, (M, K), dtype)
    if not (need_x or need_A or need_B):
        return None, None, None
    gx = None
    if need_x:
        like = addend if addend is not None else x
        gx = torch.empty((M, K), dtype=dtype, device=device) if like is None else torch.empty_like(like)
    gA = torch.empty_like(A) if need_A else None
    gB = torch.empty_like(B) if need_B else None
    ws = _workspace(what, ws, _lib.i8lt_adapters_workspace_size(M, K, N, E, r), device)
    _check(_lib.i8lt_adapters_backward(g.data_ptr(), _ptr(x), _ptr(t), _code(dtype), M, K, A.data_ptr(),
                                       B.data_ptr(), E, r, N, _ptr(scale), plan.data.data_ptr(), _ptr(addend),
                                       _ptr(gx), _ptr(gA), _ptr(gB), ws.data_ptr(), ws.numel(), _stream(g)),
           "i8lt_adapters_backward")
    return gx, gA, gB


class AdaptersFunction(torch.autograd.Function):
    """y = base + the low-rank adapters' product of x (the gradient passes to
    base unchanged; scale has none, and a backward pass that wants one is
    refused)."""

    @staticmethod
    def forward(ctx, x, base, A, B, scale, plan):
        x2 = x.reshape(-1, x.shape[-1])
        b2 = None if base is None else base.reshape(x2.shape[0], base.shape[-1])
        y, t = adapters_forward(x2, A, B, scale, plan, base=b2)
        ctx.save_for_backward(x2, t, A, B, scale)
        ctx.plan, ctx.x_shape = plan, x.shape
        return y.reshape(*x.shape[:-1], B.shape[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x2, t, A, B, scale = ctx.saved_tensors
        need = ctx.needs_input_grad
        if need[4]:
            raise I8LTError("AdaptersFunction: scale requires a gradient, which the adapters do not compute")
        gx = gA = gB = None
        if need[0] or need[2] or need[3]:
            gx, gA, gB = adapters_backward(gy.reshape(x2.shape[0], gy.shape[-1]), x2, t, A, B, scale, ctx.plan, need_x=need[0],
                                           need_A=need[2], need_B=need[3])
        if gx is not None:
            gx = gx.reshape(ctx.x_shape)
        return gx, (gy if need[1] else None), gA, gB, None, None


def adamw_state_size(params) -> int:
    """Elements of the flat AdamW states of ``params``: each tensor's start is
    a multiple of 256."""
    blk = _lib.I8LT_ADAMW_BLOCK
    return sum(-(-p.numel() // blk) * blk for p in params)


_data_ptr, _size, _get_device = torch.Tensor.data_ptr, torch.Tensor.size, torch.Tensor.get_device
_is_contiguous, _numel, _dtype_of = torch.Tensor.is_contiguous, torch.Tensor.numel, operator.attrgetter("dtype")


def adamw_counts(params) -> torch.Tensor:
    """Update counts of ``params`` for ``adamw_step`` and ``adamw_step_8bit``
    in place of a step number: zeros, int64 [len(params), 2] on their device,
    whose first column the calls keep."""
    return torch.zeros(len(params), 2, dtype=torch.int64, device=params[0].device)


def _adamw_counts(what, step, count, device) -> int:
    """The address of update counts after their checks."""
    if step.dtype != torch.int64 or step.shape != (count, 2) or not step.is_contiguous() or step.device != device:
        raise I8LTError(f"{what}: update counts of shape {tuple(step.shape)}, {step.dtype} on {step.device}, expected "
                        f"contiguous ({count}, 2), torch.int64 on {device}")
    return step.data_ptr()


def _adamw_lists(what, params, grads):
    """(the parameters with a gradient, what must outlive the call, count,
    addresses of the lists of device addresses and sizes, dtypes, elements of a
    state), checked.
    Called for hundreds of tensors per step: each property is read in one
    sweep, and the lists are plain arrays (128 tensors: 90 us; 119 us with
    ctypes arrays, which convert element by element)."""
    n = len(params)
    if n != len(grads):
        raise I8LTError(f"{what}: {n} parameters, {len(grads)} gradients")
    present = params, grads
    if any([g is None for g in grads]):
        pairs = [(p, g) for p, g in zip(params, grads) if g is not None]
        present = [p for p, _ in pairs], [g for _, g in pairs]
    if not present[1]:
        return None
    p0, g0 = params[0], present[1][0]
    _require_cuda(p0)
    if set(map(_dtype_of, params)) != {p0.dtype} or set(map(_dtype_of, present[1])) != {g0.dtype}:
        raise I8LTError(f"{what}: parameters of one dtype and gradients of one dtype are expected")
    if set(map(_get_device, params)) | set(map(_get_device, present[1])) != {p0.get_device()}:
        raise I8LTError(f"{what}: tensors on {p0.device} and another device")
    if not all(map(_is_contiguous, params)):
        raise I8LTError(f"{what}: a parameter is not contiguous")
    if list(map(_size, present[0])) != list(map(_size, present[1])):
        raise I8LTError(f"{what}: a gradient has another shape than its parameter")
    held = grads
    if not all(map(_is_contiguous, present[1])):
        held = [None if g is None else g.contiguous() for g in grads]
    sizes = list(map(_numel, params))
    blk = _lib.I8LT_ADAMW_BLOCK
    total = sum([(k + blk - 1) // blk for k in sizes]) * blk
    addresses = map(_data_ptr, held) if present[1] is grads else [0 if g is None else g.data_ptr() for g in held]
    lists = array.array("Q", map(_data_ptr, params)), array.array("Q", addresses), array.array("q", sizes)
    if len(set(lists[0])) != n:                       # equal addresses: of empty tensors, or of one given twice
        starts = [a for a, k in zip(lists[0], sizes) if k]
        if len(set(starts)) != len(starts):
            raise I8LTError(f"{what}: a parameter is given twice")
    at = [a.buffer_info()[0] for a in lists]
    return present[0], (held, lists), n, *at, _code(p0.dtype), _code(g0.dtype), total


def _adamw_state(what, size, dtype, device, *ts):
    for t in ts:
        if t.dtype != dtype or t.numel() != size or not t.is_contiguous() or t.device != device:
            raise I8LTError(f"{what}: a state of {t.numel()} {t.dtype} on {t.device}, expected {size} contiguous "
                            f"{dtype} on {device}")


def _adamw_scalar(what, t, device):
    if t is not None and (t.dtype != torch.float32 or t.numel() != 1 or t.device != device):
        raise I8LTError(f"{what}: grad_scale and found_inf are fp32 tensors of one element on {device}")


def adamw_step(params, grads, m: torch.Tensor, v: torch.Tensor, step: int | torch.Tensor, lr: float, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
               grad_scale: torch.Tensor | None = None, found_inf: torch.Tensor | None = None) -> None:
    """One AdamW step, in place, over all ``params`` at once (i8lt_adamw_step).
    m and v: flat fp32 states of ``adamw_state_size(params)`` elements.
    No two parameters may overlap.  A parameter whose gradient is None stays as
    it is.  grad_scale multiplies every gradient; a found_inf other than 0 makes
    the step change nothing (both fp32 CUDA tensors of one element).  ``step``:
    the number of updates, this one included, that m and v of every parameter
    will have seen; or ``adamw_counts(params)``, which counts them on the device
    for each parameter, without those that had no gradient or that found_inf
    skipped."""
    lists = _adamw_lists("adamw_step", params, grads)
    if lists is None:
        return
    changed, held, n, pp, gp, sizes, pt, gt, size = lists
    p0 = changed[0]
    _adamw_state("adamw_step", size, torch.float32, p0.device, m, v)
    _adamw_scalar("adamw_step", grad_scale, p0.device)
    _adamw_scalar("adamw_step", found_inf, p0.device)
    call = _lib.i8lt_adamw_step
    if isinstance(step, torch.Tensor):
        call, step = _lib.i8lt_adamw_step_counted, _adamw_counts("adamw_step", step, n, p0.device)
    _check(call(pp, pt, gp, gt, sizes, n, m.data_ptr(), v.data_ptr(), step, lr, beta1, beta2, eps, weight_decay,
                _ptr(grad_scale), _ptr(found_inf), _stream(p0)), "i8lt_adamw_step")
    _written((*changed, m, v))


def adamw_step_8bit(params, grads, m: torch.Tensor, m_absmax: torch.Tensor, r: torch.Tensor, r_absmax: torch.Tensor,
                    step: int | torch.Tensor, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                    weight_decay: float = 0.01, grad_scale: torch.Tensor | None = None,
                    found_inf: torch.Tensor | None = None) -> None:
    """``adamw_step`` with 8-bit states (i8lt_adamw_step_8bit): m and
    r = sqrt(v) as flat float8_e4m3fn tensors of ``adamw_state_size(params)``
    elements, m_absmax and r_absmax fp32, one per 256 elements."""
    lists = _adamw_lists("adamw_step_8bit", params, grads)
    if lists is None:
        return
    changed, held, n, pp, gp, sizes, pt, gt, size = lists
    p0 = changed[0]
    _adamw_state("adamw_step_8bit", size, torch.float8_e4m3fn, p0.device, m, r)
    _adamw_state("adamw_step_8bit", size // _lib.I8LT_ADAMW_BLOCK, torch.float32, p0.device, m_absmax, r_absmax)
    _adamw_scalar("adamw_step_8bit", grad_scale, p0.device)
    _adamw_scalar("adamw_step_8bit", found_inf, p0.device)
    call = _lib.i8lt_adamw_step_8bit
    if isinstance(step, torch.Tensor):
        call, step = _lib.i8lt_adamw_step_8bit_counted, _adamw_counts("adamw_step_8bit", step, n, p0.device)
    _check(call(pp, pt, gp, gt, sizes, n, m.data_ptr(), m_absmax.data_ptr(), r.data_ptr(), r_absmax.data_ptr(), step,
                lr, beta1, beta2, eps, weight_decay, _ptr(grad_scale), _ptr(found_inf), _stream(p0)),
           "i8lt_adamw_step_8bit")
    _written((*changed, m, m_absmax, r, r_absmax))
