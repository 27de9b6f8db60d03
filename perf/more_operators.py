"""Block-scaled FP8 layers and gradient clipping as measured workloads: the
linear layer whose operands have one scale per block of 128, the same layer
for experts with ragged numbers of rows, and the norm of all gradients with
their scaling in place.

``run`` computes a case either in plain torch operations in 32 bits (``own``
false) or through the calls of int8_quantized_linear_i8lt_gb300 (``own``
true), on the same inputs and with the same outputs.

Sizes are those of the framework's workloads: 7B-style MLP layers 4096 ->
11008, the 8192 -> 28672 projections of 16384 tokens, the adapters of 32
layers, and the odd sizes of its parity tests.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
BLOCK = 128                      # columns (of a weight: columns and rows) per scale
E4M3_MAX = 448.0
TINY = 2.0 ** -100               # a block below it is a block of zeros
CLIP_EPS = 1e-6                  # of the clip factor max_norm / (norm + CLIP_EPS)


def listed():
    return [
        # a single decoded token through the MLP's first layer: latency
        {"name": "linear decode 1", "op": "linear", "dir": "fwd", "M": 1, "K": 4096, "N": 11008, "bias": 0, "dt": "bf16"},
        # 16 requests decode one token each through the large projection: the weight has to be read
        {"name": "linear decode 16", "op": "linear", "dir": "fwd", "M": 16, "K": 8192, "N": 28672, "bias": 1, "dt": "f16"},
        # 4096 tokens of a prompt through the MLP's first layer
        {"name": "linear prefill", "op": "linear", "dir": "fwd", "M": 4096, "K": 4096, "N": 11008, "bias": 1, "dt": "bf16"},
        # a training step of the large projection: forward, input and bias gradients
        {"name": "linear train", "op": "linear", "dir": "train", "M": 16384, "K": 8192, "N": 28672, "bias": 1, "dt": "bf16"},
        # odd sizes in both directions, no row on a 16-byte boundary of its own
        {"name": "linear train odd", "op": "linear", "dir": "train", "M": 777, "K": 1100, "N": 519, "bias": 1, "dt": "f16"},
        # 64 requests decode one token each, two of 64 experts per token
        {"name": "experts decode", "op": "experts", "dir": "fwd", "M": 128, "K": 4096, "N": 2048, "E": 64, "behind": 0,
         "dt": "bf16"},
        # prompts over eight experts of the MLP's first layer
        {"name": "experts prefill", "op": "experts", "dir": "fwd", "M": 8192, "K": 4096, "N": 11008, "E": 8, "behind": 0,
         "dt": "bf16"},
        # forward and input gradient at odd sizes, an expert without rows, rows behind the last expert's
        {"name": "experts train odd", "op": "experts", "dir": "train", "M": 1333, "K": 1100, "N": 519, "E": 5,
         "behind": 21, "dt": "f16"},
        # the gradients of one rank-16 adapter: latency
        {"name": "norm one adapter", "op": "norm", "layers": 1, "r": 16, "K": 4096, "N": 11008, "odd": 0, "dt": "f32"},
        # rank-64 adapters of all the MLP layers of a 32-layer model: 128 tensors
        {"name": "norm 32 layers", "op": "norm", "layers": 32, "r": 64, "K": 4096, "N": 11008, "odd": 0, "dt": "bf16"},
        # the two full weights of a trainable MLP
        {"name": "norm mlp weights", "op": "norm", "layers": 1, "r": 0, "K": 4096, "N": 11008, "odd": 0, "dt": "f32"},
        # gradients scaled in place (a loss scale taken out), every tensor of odd length
        {"name": "scale 32 layers odd", "op": "scale", "layers": 32, "r": 64, "K": 4096, "N": 11008, "odd": 1,
         "dt": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "experts", "experts", "norm", "scale"))
    if op in ("linear", "experts"):
        K, N = _log(rng, 64, 28672), _log(rng, 64, 28672)
        if rng.random() < 0.6:
            K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
        M = _log(rng, 1, min(16384, 16384 * 8192 * 28672 // (K * N)))
        dt, direction = rng.choice(("f16", "bf16")), rng.choice(("fwd", "train"))
        if op == "linear":
            return {"op": op, "dir": direction, "M": M, "K": K, "N": N, "bias": rng.choice((0, 1)), "dt": dt}
        E = max(1, min(_log(rng, 1, 64), 2 ** 30 // (K * N)))
        return {"op": op, "dir": direction, "M": M, "K": K, "N": N, "E": E,
                "behind": rng.choice((0, 0, M // 50)), "dt": dt}
    return {"op": op, "layers": _log(rng, 1, 32), "r": rng.choice((4, 8, 16, 32, 64)), "K": _log(rng, 256, 8192),
            "N": _log(rng, 256, 8192), "odd": rng.choice((0, 1)), "dt": rng.choice(("f16", "bf16", "f32"))}


# --- inputs -----------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dt):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(DTYPES[dt])


def _activation(g, M, K, dt):
    """N(0,1) with a thousandth of the columns 20 times as large."""
    x = torch.randn((M, K), generator=g, device=DEV)
    heavy = torch.rand(K, generator=g, device=DEV) < 0.001
    return x.mul_(torch.where(heavy, 20.0, 1.0)).to(DTYPES[dt])


def _code_scale(top):
    return torch.where(top >= TINY, torch.div(torch.full_like(top, E4M3_MAX), top), 0.0)


def _weight(g, E, N, K):
    """Codes [E, N, K rounded up to 16] and scales [E, N / 128, K / 128] of
    N(0, 0.02) weights, a scale per block of 128 x 128."""
    nb, kb, ld = -(-N // BLOCK), -(-K // BLOCK), -(-K // 16) * 16
    codes = torch.zeros(E, N, ld, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scales = torch.empty(E, nb, kb, device=DEV)
    for e in range(E):
        W = torch.zeros(nb * BLOCK, kb * BLOCK, device=DEV)
        W[:N, :K] = torch.randn((N, K), generator=g, device=DEV).mul_(0.02)
        B = W.view(nb, BLOCK, kb, BLOCK)
        top = B.abs().amax((1, 3))
        B.mul_(_code_scale(top)[:, None, :, None])
        codes[e].view(torch.uint8)[:, :K] = W[:N, :K].to(torch.float8_e4m3fn).view(torch.uint8)
        scales[e] = top * (1 / E4M3_MAX)
    return codes, scales


def _tensor_shapes(case):
    K, N, r = case["K"], case["N"], case["r"]
    one = [(r, K), (N, r), (r, N), (K, r)] if r else [(N, K), (K, N)]
    if r and case["layers"] == 1:
        one = one[:2]
    return [(a * b - 3 * case["odd"],) if case["odd"] else (a, b) for a, b in one] * case["layers"]


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] in ("linear", "experts"):
        M, K, N, dt = (case[k] for k in ("M", "K", "N", "dt"))
        E = case.get("E", 1)
        s["x"] = _activation(g, M, K, dt)
        s["codes"], s["scales"] = _weight(g, E, N, K)
        if case["op"] == "linear":
            s["codes"], s["scales"] = s["codes"][0], s["scales"][0]
            s["bias"] = _normal(g, (N,), 0.01, dt) if case["bias"] else None
        else:
            # unequal shares; one expert of five or more has no rows
            share = torch.rand(E, generator=g, device=DEV) + 0.25
            if E > 4:
                share[torch.randint(E, (1,), generator=g, device=DEV)] = 0
            pick = torch.multinomial(share, M - case["behind"], replacement=True, generator=g)
            s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
            s["offsets"][1:] = torch.bincount(pick, minlength=E).cumsum(0)
            # the row ranges as numbers, for the plain form
            s["ranges"] = s["offsets"].tolist()
        if case["dir"] == "train":
            s["g"] = _normal(g, (M, N), 1.0, dt)
        return s
    # the gradients back to back in one buffer, as a flattened one holds them
    shapes = _tensor_shapes(case)
    s["flat"] = _normal(g, (sum(math.prod(shape) for shape in shapes),), 1e-3, case["dt"])
    s["grads"], at = [], 0
    for shape in shapes:
        s["grads"].append(s["flat"][at:at + math.prod(shape)].view(shape))
        at += math.prod(shape)
    if case["op"] == "norm":
        s["max_norm"] = 0.5 * 1e-3 * math.sqrt(at)           # about half the norm
        s["grad_scale"] = torch.ones(1, device=DEV)
    else:
        # there and back again, so that the values of a repeated pass stay in range
        s["factors"] = [torch.full((1,), f, device=DEV) for f in (2.0, 0.5)]
        s["pass"] = 0
    return s


# --- one pass ---------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        import int8_quantized_linear_i8lt_gb300 as I
        return {"linear": _own_linear, "experts": _own_experts, "norm": _own_norm, "scale": _own_scale}[case["op"]](I, case, s)
    return {"linear": _linear, "experts": _experts, "norm": _norm, "scale": _scale}[case["op"]](case, s)


def _own_linear(I, case, s):
    K = case["K"]
    y = I.fp8_forward(s["x"], s["codes"], s["scales"], K, s["bias"])
    if case["dir"] == "fwd":
        return {"y": y}
    gx, gb = I.fp8_backward_input(s["g"], s["codes"], s["scales"], K,
                                  bias_dtype=None if s["bias"] is None else s["bias"].dtype)
    return {"y": y, "gx": gx} if gb is None else {"y": y, "gx": gx, "gb": gb}


def _own_experts(I, case, s):
    K = case["K"]
    y = I.fp8_experts_forward(s["x"], s["codes"], s["scales"], K, s["offsets"])
    if case["dir"] == "fwd":
        return {"y": y}
    return {"y": y, "gx": I.fp8_experts_backward_input(s["g"], s["codes"], s["scales"], K, s["offsets"])}


def _rounded(x):
    """x [M, C] as its E4M3 codes times the scales of its blocks, in 32 bits."""
    M, C = x.shape
    cb = -(-C // BLOCK)
    X = torch.zeros(M, cb * BLOCK, device=DEV)
    X[:, :C] = x
    B = X.view(M, cb, BLOCK)
    top = B.abs().amax(2, keepdim=True)
    q = (B * _code_scale(top)).to(torch.float8_e4m3fn).float()
    return (q * (top * (1 / E4M3_MAX))).view(M, -1)[:, :C]


def _expanded(codes, scales, K):
    """The weight [N, K] that codes and scales stand for, in 32 bits."""
    N = codes.shape[0]
    s = scales.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return codes[:, :K].float() * s


def _linear(case, s):
    dt = s["x"].dtype
    W = _expanded(s["codes"], s["scales"], case["K"])
    y = _rounded(s["x"]) @ W.T
    if s["bias"] is not None:
        y += s["bias"].float()
    out = {"y": y.to(dt)}
    if case["dir"] == "train":
        del y
        out["gx"] = (_rounded(s["g"]) @ W).to(dt)
        if s["bias"] is not None:
            out["gb"] = s["g"].float().sum(0).to(s["bias"].dtype)
    return out


def _experts(case, s):
    M, K, N, E = (case[k] for k in ("M", "K", "N", "E"))
    dt, at = s["x"].dtype, s["ranges"]
    train = case["dir"] == "train"
    y = torch.zeros(M, N, dtype=dt, device=DEV)
    gx = torch.zeros(M, K, dtype=dt, device=DEV) if train else None
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        W = _expanded(s["codes"][e], s["scales"][e], K)
        y[rows] = (_rounded(s["x"][rows]) @ W.T).to(dt)
        if train:
            gx[rows] = (_rounded(s["g"][rows]) @ W).to(dt)
    return {"y": y, "gx": gx} if train else {"y": y}


def _own_norm(I, case, s):
    norm, scale, found_inf = I.grad_norm(s["grads"], max_norm=s["max_norm"], grad_scale=s["grad_scale"])
    return {"norm": norm, "scale": scale, "found_inf": found_inf}


def _norm(case, s):
    c = s["grad_scale"][0]
    total = torch.zeros((), dtype=torch.float64, device=DEV)     # long sums
    for t in s["grads"]:
        d = t.double()
        total += (d * d).sum()
    norm = torch.sqrt(total).float() * c
    scale = c * torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
    return {"norm": norm, "scale": scale, "found_inf": (~torch.isfinite(norm)).float()}


def _own_scale(I, case, s):
    I.scale_grads_(s["grads"], s["factors"][s["pass"] & 1])
    s["pass"] += 1
    return {"grads": s["flat"]}


def _scale(case, s):
    f = s["factors"][s["pass"] & 1]
    s["pass"] += 1
    for t in s["grads"]:
        t.copy_(t.float() * f)
    return {"grads": s["flat"]}


# --- what a pass cannot do without ------------------------------------------

def work(case):
    if case["op"] in ("linear", "experts"):
        M, K, N = case["M"], case["K"], case["N"]
        # experts that can have rows: no more than there are rows
        E = min(case.get("E", 1), M - case.get("behind", 0))
        weight = E * (N * K + 4 * (-(-N // BLOCK)) * (-(-K // BLOCK)))
        rows = M - case.get("behind", 0)
        extra = 2 * N if case.get("bias") else 0
        fwd = {"bytes": 2 * rows * K + 2 * M * N + weight + extra, "flops": 2 * rows * K * N}
        if case["dir"] == "fwd":
            return fwd
        # x, g and the weight in; y, gx and the bias gradient out
        return {"bytes": fwd["bytes"] + 2 * rows * N + 2 * M * K + extra, "flops": 2 * fwd["flops"]}
    n = sum(math.prod(shape) for shape in _tensor_shapes(case))
    if case["op"] == "norm":
        return {"bytes": n * SIZE[case["dt"]] + 16, "flops": 2 * n}
    return {"bytes": 2 * n * SIZE[case["dt"]] + 4, "flops": n}


# --- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "experts": _exact_experts, "norm": _exact_norm, "scale": _exact_scale}[case["op"]](case, s)


def _exact_codes(v):
    """E4M3 values nearest to v (which came from 32 bits), ties to even: steps
    of an eighth of the binade, 2^-9 below 2^-6."""
    e = torch.frexp(v)[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rounded(x):
    """Block by block of 128 columns: codes of the 32-bit product of x and
    the 32-bit 448 / max, times the 32-bit max / 448."""
    out = []
    for part in x.double().split(BLOCK, dim=1):
        top = part.abs().max(1, keepdim=True).values
        r = torch.where(top >= TINY, E4M3_MAX / top, 0.0).float().double()
        out.append(_exact_codes((part * r).float().double()) * (top * torch.tensor(1 / E4M3_MAX).double().item()).float().double())
    return torch.cat(out, 1)


def _exact_weight(codes, scales, K):
    W = codes[:, :K].double()
    for i, rows in enumerate(W.split(BLOCK, dim=0)):
        for j, block in enumerate(rows.split(BLOCK, dim=1)):
            block.mul_(scales[i, j].double())
    return W


def _too_long(case):
    return work(case)["flops"] > 4e12 or case.get("E", 1) * case["K"] * case["N"] > 2 ** 30


def _exact_linear(case, s):
    if _too_long(case):
        return None
    W = _exact_weight(s["codes"], s["scales"], case["K"])
    y = torch.einsum("mk,nk->mn", _exact_rounded(s["x"]), W)
    if s["bias"] is not None:
        y = y + s["bias"].double()
    if case["dir"] == "fwd":
        return {"y": y}
    out = {"y": y, "gx": torch.einsum("mn,nk->mk", _exact_rounded(s["g"]), W)}
    if s["bias"] is not None:
        out["gb"] = s["g"].double().sum(0)
    return out


def _exact_experts(case, s):
    if _too_long(case):
        return None
    x = _exact_rounded(s["x"])
    y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEV)
    train = case["dir"] == "train"
    if train:
        g, gx = _exact_rounded(s["g"]), torch.zeros_like(x)
    which = torch.bucketize(torch.arange(case["M"], device=DEV), s["offsets"][1:].long(), right=True)
    for e in range(case["E"]):
        rows = (which == e).nonzero()[:, 0]
        if not len(rows):
            continue
        W = _exact_weight(s["codes"][e], s["scales"][e], case["K"])
        y[rows] = torch.einsum("mk,nk->mn", x[rows], W)
        if train:
            gx[rows] = torch.einsum("mn,nk->mk", g[rows], W)
    return {"y": y, "gx": gx} if train else {"y": y}


def _exact_norm(case, s):
    c = float(s["grad_scale"])
    norm = c * math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"]))
    scale = c * min(1.0, s["max_norm"] / (norm + CLIP_EPS))
    return {k: torch.tensor(v, dtype=torch.float64, device=DEV)
            for k, v in (("norm", norm), ("scale", scale), ("found_inf", 0.0 if math.isfinite(norm) else 1.0))}


def _exact_scale(case, s):
    f = float(s["factors"][0])
    return {"grads": torch.cat([t.double().flatten() * f for t in s["grads"]])}
