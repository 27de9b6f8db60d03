"""The adapter fine-tuning operators as measured workloads: low-rank adapters
beside a shared projection, layer norm, and AdamW over many tensors.

``run`` computes a case either in plain torch operations in 32 bits (``own``
false) or through the calls of int8_quantized_linear_i8lt_gb300 (``own``
true), on the same inputs and with the same outputs.

Sizes are those of the framework's workloads: 7B-style MLP layers 4096 ->
11008 and 11008 -> 4096, the 8192-wide projections of 16384 tokens, and the
odd sizes of its parity tests.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5                       # layer norm
LR, B1, B2, AEPS, WD = 2e-4, 0.9, 0.999, 1e-8, 0.01
BLOCK = 256                      # elements per absmax of the 8-bit states; tensors start at multiples of it
E4M3_MAX = 448.0


def listed():
    return [
        # a single decoded token through a 4096-wide norm: latency
        {"name": "norm fwd 1 token", "op": "norm", "dir": "fwd", "M": 1, "N": 4096, "dt": "f16"},
        # the norm before the 8192-wide projections, 16384 tokens
        {"name": "norm fwd 16384x8192", "op": "norm", "dir": "fwd", "M": 16384, "N": 8192, "dt": "bf16"},
        # the norm before the 7B-style MLP in training, 8192 tokens
        {"name": "norm bwd 8192x4096", "op": "norm", "dir": "bwd", "M": 8192, "N": 4096, "dt": "f16"},
        # rows of odd length, none of them on a 16-byte boundary of its own
        {"name": "norm bwd odd", "op": "norm", "dir": "bwd", "M": 1333, "N": 4099, "dt": "bf16"},
        # 64 requests decode one token each, every one with an adapter of its own
        {"name": "adapters decode", "op": "adapters", "dir": "fwd", "M": 64, "K": 4096, "N": 4096, "r": 16, "E": 64,
         "order": "mixed", "dt": "f16"},
        # prompts of several requests in one batch, eight adapters and some tokens without one
        {"name": "adapters prefill", "op": "adapters", "dir": "fwd", "M": 2048, "K": 4096, "N": 11008, "r": 16, "E": 8,
         "order": "runs", "dt": "bf16"},
        # fine-tuning one rank-64 adapter of the MLP's first layer: forward and backward
        {"name": "adapters train", "op": "adapters", "dir": "train", "M": 8192, "K": 4096, "N": 11008, "r": 64, "E": 1,
         "order": "runs", "dt": "bf16"},
        # three adapters trained together at odd sizes, tokens interleaved
        {"name": "adapters train odd", "op": "adapters", "dir": "train", "M": 777, "K": 1100, "N": 519, "r": 12, "E": 3,
         "order": "mixed", "dt": "f16"},
        # the two matrices of one rank-16 adapter: latency
        {"name": "adamw one adapter", "op": "adamw", "bits": 32, "layers": 1, "r": 16, "K": 4096, "N": 11008,
         "odd": 0, "dt": "f32"},
        # the two full weights of a trainable 7B-style MLP, 32-bit states
        {"name": "adamw mlp weights", "op": "adamw", "bits": 32, "layers": 1, "r": 0, "K": 4096, "N": 11008,
         "odd": 0, "dt": "f32"},
        # rank-64 adapters of all the MLP layers of a 32-layer model, 8-bit states: 128 tensors
        {"name": "adamw8 32 layers", "op": "adamw", "bits": 8, "layers": 32, "r": 64, "K": 4096, "N": 11008,
         "odd": 0, "dt": "bf16"},
        # the trainable MLP weights with 8-bit states, every tensor with a part of a block at its end
        {"name": "adamw8 mlp weights", "op": "adamw", "bits": 8, "layers": 1, "r": 0, "K": 4096, "N": 11008,
         "odd": 1, "dt": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "adapters", "adapters", "adamw"))
    if op == "norm":
        N = _log(rng, 64, 28672)
        if rng.random() < 0.6:
            N = max(64, N // 64 * 64)
        M = _log(rng, 1, min(32768, 16384 * 8192 // N))
        return {"op": op, "dir": rng.choice(("fwd", "bwd")), "M": M, "N": N, "dt": rng.choice(("f16", "bf16", "f32"))}
    if op == "adapters":
        M, E = _log(rng, 1, 8192), _log(rng, 1, 64)
        r = rng.choice((4, 8, 12, 16, 24, 32, 64))
        K, N = _log(rng, 256, 8192), _log(rng, 256, 8192)
        if rng.random() < 0.7:
            K, N = K // 64 * 64, N // 64 * 64
        E = max(1, min(E, 2 * M, 16384 // M))
        return {"op": op, "dir": rng.choice(("fwd", "train")), "M": M, "K": K, "N": N, "r": r, "E": E,
                "order": rng.choice(("runs", "mixed")), "dt": rng.choice(("f16", "bf16"))}
    K, N = _log(rng, 256, 8192), _log(rng, 256, 8192)
    return {"op": op, "bits": rng.choice((32, 8)), "layers": _log(rng, 1, 32), "r": rng.choice((4, 8, 16, 32, 64)),
            "K": K, "N": N, "odd": rng.choice((0, 1)), "dt": rng.choice(("f16", "bf16", "f32"))}


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


def _tensor_shapes(case):
    K, N, r = case["K"], case["N"], case["r"]
    one = [(r, K), (N, r), (r, N), (K, r)] if r else [(N, K), (K, N)]
    if r and case["layers"] == 1:
        one = one[:2]
    return [(a * b - 3 * case["odd"],) if case["odd"] else (a, b) for a, b in one] * case["layers"]


def _layout(shapes):
    sizes = [math.prod(s) for s in shapes]
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    return sizes, starts, at


def _quantize8(x, floor):
    """E4M3 codes of x in blocks of 256 and the blocks' absmax; ``floor``: the
    smallest code a value above zero may take."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    y = b * torch.where(top > 0, E4M3_MAX / torch.where(top > 0, top, 1.0), 0.0)
    if floor:
        y = torch.where(b > 0, y.clamp(min=2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn).view(-1), top.view(-1)


def _dequantize8(q, top):
    return (q.view(-1, BLOCK).float() * (top * (1.0 / E4M3_MAX))[:, None]).view(-1)


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "norm":
        M, N, dt = case["M"], case["N"], case["dt"]
        s["x"] = _activation(g, M, N, dt)
        s["x"] += torch.randn((M, 1), generator=g, device=DEV).to(s["x"].dtype)
        s["w"] = (1 + 0.1 * torch.randn(N, generator=g, device=DEV)).to(DTYPES[dt])
        s["b"] = _normal(g, (N,), 0.1, dt)
        if case["dir"] == "bwd":
            s["g"] = _normal(g, (M, N), 1.0, dt)
            x = s["x"].float()
            s["mean"] = x.mean(1)                      # what the forward pass kept
            s["rstd"] = (x.var(1, correction=0) + EPS).rsqrt()
    elif case["op"] == "adapters":
        M, K, N, r, E, dt = (case[k] for k in ("M", "K", "N", "r", "E", "dt"))
        s["x"] = _activation(g, M, K, dt)
        s["A"] = _normal(g, (E, r, K), K ** -0.5, dt)
        s["B"] = _normal(g, (E, N, r), 0.02, dt)
        s["scale"] = 0.5 + torch.rand(E, generator=g, device=DEV)
        s["base"] = _normal(g, (M, N), 1.0, dt)
        none = 1 if E > 1 else 0                       # with several adapters, some tokens use none (-1)
        if case["order"] == "mixed" and M <= E:
            s["index"] = torch.randperm(E, generator=g, device=DEV)[:M].int()
        elif case["order"] == "mixed":
            s["index"] = torch.randint(-none, E, (M,), generator=g, device=DEV).int()
        else:                                          # whole requests, one after another
            cuts = torch.rand(M, generator=g, device=DEV) < (2.0 * E / M if E > 1 else 0.0)
            which = torch.randint(-none, E, (M,), generator=g, device=DEV)
            s["index"] = which[torch.cumsum(cuts, 0).clamp(max=M - 1)].int()
        if case["dir"] == "train":
            s["g"] = _normal(g, (M, N), 1.0, dt)
            s["addend"] = _normal(g, (M, K), 1.0, dt)  # the shared projection's input gradient
    else:
        shapes = _tensor_shapes(case)
        sizes, starts, total = _layout(shapes)
        dt = DTYPES[case["dt"]]
        inside = torch.zeros(total, dtype=torch.bool, device=DEV)
        for n, at in zip(sizes, starts):
            inside[at:at + n] = True

        def flat(std):
            return torch.randn(total, generator=g, device=DEV).mul_(std).mul_(inside)

        s["p"], s["grad"] = flat(0.02).to(dt), flat(1e-3).to(dt)
        m, r = flat(3e-4), flat(1e-3).abs_()
        del inside
        s["params"] = [s["p"][at:at + n].view(sh) for n, at, sh in zip(sizes, starts, shapes)]
        s["grads"] = [s["grad"][at:at + n].view(sh) for n, at, sh in zip(sizes, starts, shapes)]
        s["step"] = 10                                 # steps made so far
        if case["bits"] == 8:
            s["m"], s["m_absmax"] = _quantize8(m, False)
            s["r"], s["r_absmax"] = _quantize8(r, True)
        else:
            s["m"], s["v"] = m, r * r
    return s


# --- one pass ---------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        import int8_quantized_linear_i8lt_gb300 as I
        return {"norm": _own_norm, "adapters": _own_adapters, "adamw": _own_adamw}[case["op"]](I, case, s)
    return {"norm": _norm, "adapters": _adapters, "adamw": _adamw}[case["op"]](case, s)


def _own_norm(I, case, s):
    if case["dir"] == "fwd":
        y, mean, rstd = I.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    gx, gw, gb = I.layer_norm_backward(s["g"], s["x"], s["mean"], s["rstd"], s["w"])
    return {"gx": gx, "gw": gw, "gb": gb}


def _norm(case, s):
    x = s["x"].float()
    if case["dir"] == "fwd":
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
        y = d * rstd[:, None] * s["w"].float() + s["b"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    g, rstd = s["g"].float(), s["rstd"][:, None]
    h = (x - s["mean"][:, None]) * rstd
    gw, gb = (g * h).sum(0), g.sum(0)
    g = g * s["w"].float()
    gx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    dt = s["x"].dtype
    return {"gx": gx.to(dt), "gw": gw.to(dt), "gb": gb.to(dt)}


def _own_adapters(I, case, s):
    plan = I.adapter_plan(s["index"], case["E"])
    y, t = I.adapters_forward(s["x"], s["A"], s["B"], s["scale"], plan, base=s["base"])
    if case["dir"] == "fwd":
        return {"y": y}
    gx, gA, gB = I.adapters_backward(s["g"], s["x"], t, s["A"], s["B"], s["scale"], plan, addend=s["addend"])
    return {"y": y, "gx": gx, "gA": gA, "gB": gB}


def _adapters(case, s):
    E, r, dt = case["E"], case["r"], s["x"].dtype
    x, A = s["x"].float(), s["A"].float().flatten(0, 1)                       # [E r, K]
    B = s["B"].float().transpose(1, 2).flatten(0, 1)                          # [E r, N]
    # each token's scale in its own adapter's columns, 0 in the others'
    pick = (s["index"][:, None] == torch.arange(E, device=DEV)) * s["scale"]  # [M, E]
    pick = pick.repeat_interleave(r, 1)
    t = (x @ A.T) * pick
    y = s["base"].float() + t @ B
    if case["dir"] == "fwd":
        return {"y": y.to(dt)}
    g = s["g"].float()
    u = (g @ B.T) * pick
    gx = s["addend"].float() + u @ A
    gA = (u.T @ x).view(E, r, -1)
    gB = (t.T @ g).view(E, r, -1).transpose(1, 2).contiguous()
    return {"y": y.to(dt), "gx": gx.to(dt), "gA": gA.to(dt), "gB": gB.to(dt)}


def _own_adamw(I, case, s):
    s["step"] += 1
    kw = dict(step=s["step"], lr=LR, beta1=B1, beta2=B2, eps=AEPS, weight_decay=WD)
    if case["bits"] == 8:
        I.adamw_step_8bit(s["params"], s["grads"], s["m"], s["m_absmax"], s["r"], s["r_absmax"], **kw)
        return {k: s[k] for k in ("p", "m", "m_absmax", "r", "r_absmax")}
    I.adamw_step(s["params"], s["grads"], s["m"], s["v"], **kw)
    return {k: s[k] for k in ("p", "m", "v")}


def _adamw(case, s):
    s["step"] += 1
    p, g = s["p"].float(), s["grad"].float()
    bits8 = case["bits"] == 8
    if bits8:
        m, r = _dequantize8(s["m"], s["m_absmax"]), _dequantize8(s["r"], s["r_absmax"])
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * B1 + g * (1 - B1)
    v = v * B2 + g * g * (1 - B2)
    r = torch.sqrt(v)
    size, root = LR / (1 - B1 ** s["step"]), 1 / math.sqrt(1 - B2 ** s["step"])
    s["p"].copy_(p * (1 - LR * WD) - m * size / (r * root + AEPS))
    if bits8:
        (q, top), (q2, top2) = _quantize8(m, False), _quantize8(r, True)
        s["m"].copy_(q), s["m_absmax"].copy_(top), s["r"].copy_(q2), s["r_absmax"].copy_(top2)
        return {k: s[k] for k in ("p", "m", "m_absmax", "r", "r_absmax")}
    s["m"].copy_(m), s["v"].copy_(v)
    return {k: s[k] for k in ("p", "m", "v")}


# --- what a pass cannot do without ------------------------------------------

def work(case):
    if case["op"] == "norm":
        M, N, e = case["M"], case["N"], SIZE[case["dt"]]
        if case["dir"] == "fwd":
            return {"bytes": 2 * M * N * e + 2 * N * e + 8 * M, "flops": 8 * M * N}
        return {"bytes": 3 * M * N * e + 3 * N * e + 8 * M, "flops": 14 * M * N}
    if case["op"] == "adapters":
        M, K, N, r, E = (case[k] for k in ("M", "K", "N", "r", "E"))
        weights = 2 * min(E, M) * r * (K + N)
        fwd = 2 * M * (K + 2 * N) + weights + 4 * M + 4 * E
        if case["dir"] == "fwd":
            return {"bytes": fwd, "flops": 2 * M * r * (K + N)}
        return {"bytes": fwd + 2 * M * (N + 3 * K) + weights + 2 * E * r * (K + N), "flops": 6 * M * r * (K + N)}
    sizes, _, total = _layout(_tensor_shapes(case))
    e, n = SIZE[case["dt"]], sum(sizes)
    if case["bits"] == 8:
        return {"bytes": n * (3 * e + 4) + total // BLOCK * 16, "flops": 25 * n}
    return {"bytes": n * (3 * e + 16), "flops": 15 * n}


# --- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "adapters": _exact_adapters, "adamw": _exact_adamw}[case["op"]](case, s)


def _exact_norm(case, s):
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    N = case["N"]
    if case["dir"] == "fwd":
        mean = x.sum(1) / N
        x = x.sub_(mean[:, None])
        rstd = ((x * x).sum(1) / N + EPS) ** -0.5
        return {"y": x.mul_(rstd[:, None]).mul_(w).add_(b), "mean": mean, "rstd": rstd}
    g, rstd = s["g"].double(), s["rstd"].double()
    h = x.sub_(s["mean"].double()[:, None]).mul_(rstd[:, None])
    gb, gw = g.sum(0), torch.einsum("mn,mn->n", g, h)
    first, second = (g @ w) / N, torch.einsum("mn,mn,n->m", g, h, w) / N
    gx = g.mul_(w).sub_(first[:, None]).sub_(h.mul_(second[:, None])).mul_(rstd[:, None])
    return {"gx": gx, "gw": gw, "gb": gb}


def _exact_adapters(case, s):
    E = case["E"]
    if case["M"] * (case["K"] + case["N"]) * case["r"] > 2 ** 34:
        return None
    x, A, B = s["x"].double(), s["A"].double(), s["B"].double()
    train = case["dir"] == "train"
    y = s["base"].double()
    if train:
        g, gx = s["g"].double(), s["addend"].double()
        gA, gB = torch.zeros_like(A), torch.zeros_like(B)
    for e in range(E):
        rows = (s["index"] == e).nonzero()[:, 0]
        if not len(rows):
            continue
        scale = s["scale"][e].double()
        t = x[rows] @ A[e].T
        y[rows] += scale * (t @ B[e].T)
        if train:
            u = scale * (g[rows] @ B[e])
            gx[rows] += u @ A[e]
            gA[e], gB[e] = u.T @ x[rows], scale * (g[rows].T @ t)
    return {"y": y, "gx": gx, "gA": gA, "gB": gB} if train else {"y": y}


def _exact_adamw(case, s):
    """The 8-bit codes depend on the rounding of single values and have no
    value in 64 bits; the parameters and the blocks' absmax have one."""
    step = s["step"] + 1
    p, g = s["p"].double(), s["grad"].double()
    if case["bits"] == 8:
        m = (s["m"].double().view(-1, BLOCK) * s["m_absmax"].double()[:, None] / E4M3_MAX).view(-1)
        v = (s["r"].double().view(-1, BLOCK) * s["r_absmax"].double()[:, None] / E4M3_MAX).view(-1) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * g * g
    p = p - LR * WD * p - LR * (m / (1 - B1 ** step)) / ((v / (1 - B2 ** step)) ** 0.5 + AEPS)
    if case["bits"] == 8:
        return {"p": p, "m": None, "m_absmax": m.abs().view(-1, BLOCK).amax(1), "r": None,
                "r_absmax": v.sqrt().view(-1, BLOCK).amax(1)}
    return {"p": p, "m": m, "v": v}
