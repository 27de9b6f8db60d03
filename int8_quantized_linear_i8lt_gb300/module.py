"""nn.Module front ends: Linear8bitLt and the two-layer SiLU MLP.

The int8 weight is never drawn at random (``normal_`` has no int8 kernel, as
the lit-gpt QLoRA PR notes for bnb.int8 training): a layer is built from a
float weight with ``from_float``, or loaded with its CB / SCB buffers.
"""
from __future__ import annotations

import torch

from . import functional as F


class Linear8bitLt(torch.nn.Module):
    """Memory-efficient int8 linear layer (bitsandbytes PR #33): int8
    row-major weight CB with per-row scales SCB, fp16 outlier decomposition
    above ``threshold``, input cast to fp16 and output cast back, backward
    to the input through fp16 weights rebuilt on the fly.  The weight takes
    no gradient; the bias does."""

    def __init__(self, in_features: int, out_features: int, bias: bool = True, threshold: float = 6.0,
                 device=None, bias_dtype: torch.dtype = torch.float16, max_outliers: int | None = None):
        super().__init__()
        self.in_features = in_features
        self.out_features = out_features
        self.threshold = float(threshold)
        self.max_outliers = max_outliers
        ld = F.weight_ld(in_features)
        self.register_buffer("CB", torch.zeros(out_features, ld, dtype=torch.int8, device=device))
        self.register_buffer("SCB", torch.zeros(out_features, dtype=torch.float32, device=device))
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(out_features, dtype=bias_dtype, device=device))
        else:
            self.register_parameter("bias", None)

    @classmethod
    def from_float(cls, weight: torch.Tensor, bias: torch.Tensor | None = None, threshold: float = 6.0,
                   max_outliers: int | None = None) -> "Linear8bitLt":
        """Quantize a float weight [out, in] on its CUDA device."""
        N, K = weight.shape
        layer = cls(K, N, bias=bias is not None, threshold=threshold, device=weight.device,
                    bias_dtype=bias.dtype if bias is not None else torch.float16, max_outliers=max_outliers)
        CB, SCB = F.quantize_weight(weight)
        layer.CB.copy_(CB)
        layer.SCB.copy_(SCB)
        if bias is not None:
            with torch.no_grad():
                layer.bias.copy_(bias)
        return layer

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return F.Int8LinearFunction.apply(x, self.CB, self.SCB, self.bias, self.threshold, self.max_outliers)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, threshold={self.threshold}")


class Linear8bitLtTrainable(torch.nn.Module):
    """The trainable-weight mode of the same layer (bitsandbytes'
    has_fp16_weights=True): the float weight is a parameter, quantized afresh
    on every forward; its gradient comes from the int8 column-wise product
    G^T A (i8lt_grad_weight)."""

    def __init__(self, in_features: int, out_features: int, bias: bool = True, threshold: float = 6.0,
                 device=None, dtype: torch.dtype = torch.float16, max_outliers: int | None = None):
        super().__init__()
        self.in_features = in_features
        self.out_features = out_features
        self.threshold = float(threshold)
        self.max_outliers = max_outliers
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, dtype=dtype, device=device))
        torch.nn.init.kaiming_uniform_(self.weight, a=5 ** 0.5)
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(out_features, dtype=dtype, device=device))
        else:
            self.register_parameter("bias", None)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return F.Int8LinearTrainableFunction.apply(x, self.weight, self.bias, self.threshold, self.max_outliers)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, threshold={self.threshold}, trainable weight")


class Int8MLP(torch.nn.Module):
    """y = fc2(silu(fc1(x))) (+ x when ``residual``), both layers int8."""

    def __init__(self, fc1: Linear8bitLt, fc2: Linear8bitLt, residual: bool = False):
        super().__init__()
        self.fc1, self.fc2, self.residual = fc1, fc2, residual

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return F.Int8MLPFunction.apply(x, self.fc1.CB, self.fc1.SCB, self.fc1.bias, self.fc2.CB, self.fc2.SCB,
                                       self.fc2.bias, self.fc1.threshold, self.residual, self.fc1.max_outliers)


class Linear4bit(torch.nn.Module):
    """Frozen 4-bit linear layer of QLoRA fine-tuning: the weight is stored
    as packed 4-bit codes (``fmt``: "nf4", 4-bit NormalFloat, or "fp4", the
    E2M1 floating-point format) with one fp32 absmax per 64 elements of a row
    and decoded to the 16-bit compute dtype (the input's: f16 or bf16) inside
    the tensor-core matmuls of the forward and of the input gradient.  The
    weight takes no gradient; the bias does (reduced inside the
    input-gradient GEMM).  ``materialized``: each matmul first writes the
    16-bit weight to a temporary workspace and reads it with a plain GEMM
    (faster, N * K * 2 bytes of transient memory); the results are the same
    bits.  ``double_quant`` (the ``bnb.nf4-dq`` / ``bnb.fp4-dq`` options): the
    absmax values are stored in 8 bits (FP8 E4M3 codes in blocks of 256 with
    an fp32 scale each, around their mean) and decoded by one kernel per
    call."""

    fmt = "nf4"

    def __init__(self, in_features: int, out_features: int, bias: bool = True, device=None,
                 bias_dtype: torch.dtype = torch.bfloat16, materialized: bool = False, fmt: str | None = None,
                 double_quant: bool = False):
        super().__init__()
        from . import _lib
        if fmt is not None:
            self.fmt = F._fmt4(fmt)
        self.in_features = in_features
        self.out_features = out_features
        self.materialized = bool(materialized)
        self.double_quant = bool(double_quant)
        nblk = _lib.i8lt_nf4_blocks(in_features)
        self.register_buffer("packed", torch.zeros(out_features, _lib.i8lt_nf4_row_bytes(in_features),
                                                   dtype=torch.uint8, device=device))
        if self.double_quant:
            self.register_buffer("absmax_q", torch.zeros(out_features, nblk, dtype=torch.uint8, device=device))
            self.register_buffer("absmax2", torch.zeros(_lib.i8lt_absmax8_blocks(out_features * nblk),
                                                        dtype=torch.float32, device=device))
            self.register_buffer("absmax_offset", torch.zeros(1, dtype=torch.float32, device=device))
        else:
            self.register_buffer("absmax", torch.zeros(out_features, nblk, dtype=torch.float32, device=device))
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(out_features, dtype=bias_dtype, device=device))
        else:
            self.register_parameter("bias", None)

    @classmethod
    def from_float(cls, weight: torch.Tensor, bias: torch.Tensor | None = None,
                   materialized: bool = False, **kw) -> "Linear4bit":
        N, K = weight.shape
        layer = cls(K, N, bias=bias is not None, device=weight.device,
                    bias_dtype=bias.dtype if bias is not None else torch.bfloat16, materialized=materialized, **kw)
        packed, absmax = F.quantize_4bit(weight, layer.fmt)
        layer.packed.copy_(packed)
        if layer.double_quant:
            q, a2, off = F.double_quantize_absmax(absmax)
            layer.absmax_q.copy_(q)
            layer.absmax2.copy_(a2)
            layer.absmax_offset.copy_(off)
        else:
            layer.absmax.copy_(absmax)
        if bias is not None:
            with torch.no_grad():
                layer.bias.copy_(bias)
        return layer

    def decoded_absmax(self) -> torch.Tensor:
        """The fp32 absmax [N, blocks per row] the matmuls use."""
        if self.double_quant:
            return F.dequantize_absmax(self.absmax_q, self.absmax2, self.absmax_offset)
        return self.absmax

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return F.Linear4bitFunction.apply(x, self.packed, self.decoded_absmax(), self.in_features, self.bias,
                                          self.materialized, self.fmt)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}, "
                f"fmt={self.fmt}, double_quant={self.double_quant}")


class LinearNF4(Linear4bit):
    """The 4-bit NormalFloat layer (bnb.nf4)."""
    fmt = "nf4"


class LinearFP4(Linear4bit):
    """The 4-bit floating-point (E2M1) layer (bnb.fp4)."""
    fmt = "fp4"


class _FP8Weight(torch.nn.Module):
    """A module with FP8 ``codes`` and fp32 ``scales``, which keep their types
    when the module's dtype is converted (``half()``, ``to(dtype)``): while
    the buffers are moved they are integers, as the codes of the int8 and 4-bit
    layers are."""

    def _apply(self, fn, recurse=True):
        types = {"codes": (torch.uint8, F.FP8), "scales": (torch.int32, torch.float32)}
        for name, (raw, own) in types.items():
            if self._buffers[name].dtype == own:
                self._buffers[name] = self._buffers[name].view(raw)
        try:
            return super()._apply(fn, recurse)
        finally:
            for name, (raw, own) in types.items():
                if self._buffers[name].dtype == raw:
                    self._buffers[name] = self._buffers[name].view(own)


class LinearFP8(_FP8Weight):
    """Frozen FP8 linear layer: E4M3 codes with one fp32 scale per 128 x 128
    block of the weight; tokens (f16 or bf16) and output gradients are rounded
    to FP8 in blocks of 128 columns inside the call and multiplied on the FP8
    tensor cores.  The weight takes no gradient; the bias does."""

    def __init__(self, in_features: int, out_features: int, bias: bool = True, device=None,
                 bias_dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        self.in_features, self.out_features = in_features, out_features
        codes, scales = F._fp8_shapes(out_features, in_features)
        self.register_buffer("codes", F._zeros_fp8(codes, device))
        self.register_buffer("scales", torch.zeros(scales, dtype=torch.float32, device=device))
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(out_features, dtype=bias_dtype, device=device))
        else:
            self.register_parameter("bias", None)

    @classmethod
    def from_float(cls, weight: torch.Tensor, bias: torch.Tensor | None = None) -> "LinearFP8":
        """Quantize a float weight [out, in] on its CUDA device."""
        N, K = weight.shape
        layer = cls(K, N, bias=bias is not None, device="meta",
                    bias_dtype=bias.dtype if bias is not None else torch.bfloat16)
        layer.codes, layer.scales = F.fp8_quantize_weight(weight.detach())
        if bias is not None:
            layer.bias = torch.nn.Parameter(bias.detach().to(weight.device, copy=True))
        return layer

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return F.LinearFP8Function.apply(x, self.codes, self.scales, self.in_features, self.bias)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}"


class ExpertsFP8(_FP8Weight):
    """``LinearFP8`` for ``experts`` weights at once, without bias: rows
    offsets[e] up to offsets[e + 1] of x [tokens, in_features], sorted by
    expert, take expert e's (``offsets``: int32 [experts + 1] on the device).
    Rows of no expert give zeros, and get a gradient of zero."""

    def __init__(self, experts: int, in_features: int, out_features: int, device=None):
        super().__init__()
        self.experts, self.in_features, self.out_features = experts, in_features, out_features
        codes, scales = F._fp8_shapes(out_features, in_features)
        self.register_buffer("codes", F._zeros_fp8((experts, *codes), device))
        self.register_buffer("scales", torch.zeros((experts, *scales), dtype=torch.float32, device=device))

    @classmethod
    def from_float(cls, weight: torch.Tensor) -> "ExpertsFP8":
        """Quantize float weights [experts, out, in] on their CUDA device."""
        E, N, K = weight.shape
        layer = cls(E, K, N, device="meta")
        layer.codes, layer.scales = F.fp8_quantize_weight(weight.detach())
        return layer

    def forward(self, x: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        return F.ExpertsFP8Function.apply(x, self.codes, self.scales, self.in_features, offsets)

    def extra_repr(self) -> str:
        return f"experts={self.experts}, in_features={self.in_features}, out_features={self.out_features}"


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension with trainable weight and bias."""

    def __init__(self, features: int, eps: float = 1e-5, bias: bool = True, device=None,
                 dtype: torch.dtype = torch.float32):
        super().__init__()
        self.features = features
        self.eps = float(eps)
        self.weight = torch.nn.Parameter(torch.ones(features, dtype=dtype, device=device))
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(features, dtype=dtype, device=device))
        else:
            self.register_parameter("bias", None)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return F.LayerNormFunction.apply(x, self.weight, self.bias, self.eps)

    def extra_repr(self) -> str:
        return f"{self.features}, eps={self.eps}, bias={self.bias is not None}"


class LowRankAdapters(torch.nn.Module):
    """``adapters`` low-rank adapters beside a shared, frozen layer ``base``
    (Linear8bitLt, LinearNF4, ...): y = base(x) + scale[e] (x A[e]^T) B[e]^T
    for each token's adapter e.  A starts as N(0, 1 / in_features), B as
    zeros; ``dtype`` (f16 or bf16) is the compute type of the tokens.
    ``forward`` takes the batch's ``plan`` (``adapter_plan(index, adapters)``,
    shared by the layers of a model); without one all tokens use adapter 0."""

    def __init__(self, base: torch.nn.Module, rank: int, adapters: int = 1, scale: float = 1.0, device=None,
                 dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        self.base = base
        self.rank, self.adapters = rank, adapters
        K, N = base.in_features, base.out_features
        self.A = torch.nn.Parameter((torch.randn(adapters, rank, K, device=device) * K ** -0.5).to(dtype))
        self.B = torch.nn.Parameter(torch.zeros(adapters, N, rank, dtype=dtype, device=device))
        self.register_buffer("scale", torch.full((adapters,), float(scale), dtype=torch.float32, device=device))

    def forward(self, x: torch.Tensor, plan: F.AdapterPlan | None = None) -> torch.Tensor:
        if plan is None:
            plan = F.adapter_plan(None, self.adapters, x.numel() // x.shape[-1], x.device)
        return F.AdaptersFunction.apply(x, self.base(x), self.A, self.B, self.scale, plan)

    def extra_repr(self) -> str:
        return f"rank={self.rank}, adapters={self.adapters}"


class AdamW:
    """AdamW over all its parameters at once per dtype, with the states
    in 32 bits or (``bits=8``) as FP8 E4M3 with one fp32 absmax per 256
    elements.  A parameter without a gradient is left as it is.  step() takes
    the optional device scalars of a loss scaler or a gradient clip:
    ``grad_scale`` multiplies every gradient, a ``found_inf`` other than 0
    makes the step change nothing.  ``steps`` counts the calls; the bias
    corrections of a parameter are those of its own updates, without steps in
    which it had no gradient or that were skipped (``counts``, on the
    device).  With ``max_norm`` the step clips: the gradients (times
    grad_scale) enter it scaled to at most that norm of all of them together,
    and a norm that is not finite skips it; nothing is copied to the host, the
    gradients stay as they are, and step() returns their norm."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 bits: int = 32):
        if bits not in (8, 32):
            raise F.I8LTError(f"AdamW: states in 8 or 32 bits, not {bits}")
        self.lr, self.betas, self.eps, self.weight_decay, self.bits = lr, betas, eps, weight_decay, bits
        self.steps = 0
        lists: dict = {}
        for p in params:
            lists.setdefault((p.dtype, p.device), []).append(p)
        self.params = list(lists.values())
        for ps in self.params:      # one launch updates them all at once
            spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size()) for p in ps if p.numel())
            if any(end > start for (_, end), (start, _) in zip(spans, spans[1:])):
                raise F.I8LTError("AdamW: a parameter is given twice, or overlaps another one")
        self.counts = [F.adamw_counts(ps) for ps in self.params]
        self.states = []
        for ps in self.params:
            n, dev = F.adamw_state_size(ps), ps[0].device
            if bits == 8:
                # codes are set as bytes: 0 is E4M3's zero
                q = [torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
                top = [torch.zeros(n // 256, dtype=torch.float32, device=dev) for _ in range(2)]
                self.states.append((q[0], top[0], q[1], top[1]))
            else:
                self.states.append(tuple(torch.zeros(n, dtype=torch.float32, device=dev) for _ in range(2)))

    @torch.no_grad()
    def step(self, grad_scale: torch.Tensor | None = None, found_inf: torch.Tensor | None = None,
             max_norm: float | None = None) -> torch.Tensor | None:
        norm = None
        if max_norm is not None:
            grads = [p.grad for ps in self.params for p in ps if p.grad is not None]
            if grads:
                norm, grad_scale, found_inf = F.grad_norm(grads, max_norm, grad_scale, found_inf)
        self.steps += 1
        call = F.adamw_step_8bit if self.bits == 8 else F.adamw_step
        for ps, st, counts in zip(self.params, self.states, self.counts):
            call(ps, [p.grad for p in ps], *st, step=counts, lr=self.lr, beta1=self.betas[0],
                 beta2=self.betas[1], eps=self.eps, weight_decay=self.weight_decay, grad_scale=grad_scale,
                 found_inf=found_inf)
        return norm

    def zero_grad(self) -> None:
        for ps in self.params:
            for p in ps:
                p.grad = None

    def state_dict(self) -> dict:
        return {"steps": self.steps, "bits": self.bits, "states": [tuple(t.clone() for t in st) for st in self.states],
                "counts": [c[:, 0].clone() for c in self.counts]}

    def load_state_dict(self, d: dict) -> None:
        if d["bits"] != self.bits or [[t.shape for t in st] for st in d["states"]] != \
                [[t.shape for t in st] for st in self.states] or \
                [len(c) for c in d.get("counts", self.counts)] != [len(c) for c in self.counts]:
            raise F.I8LTError("AdamW: the state was saved for other parameters")
        self.steps = d["steps"]
        for k, counts in enumerate(self.counts):
            # a state saved without counts: every step was an update
            counts[:, 0] = d["counts"][k] if "counts" in d else self.steps
        for st, src in zip(self.states, d["states"]):
            for t, v in zip(st, src):
                t.copy_(v)
