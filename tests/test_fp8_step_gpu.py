"""The FP8 layers, adapters, layer norm, clipping and AdamW together: a step
that fine-tunes on frozen FP8 layers, and the same model serving."""
import pytest
import torch

import int8_quantized_linear_i8lt_gb300 as I

pytestmark = pytest.mark.gpu


class Block(torch.nn.Module):
    """norm -> FP8 layer with adapters -> experts of the sorted tokens."""

    def __init__(self, width=256, hidden=384, experts=3, seed=0):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5
        self.norm = I.LayerNorm(width, device="cuda", dtype=torch.bfloat16)
        self.up = I.LowRankAdapters(I.LinearFP8.from_float(w(hidden, width), torch.zeros(hidden, device="cuda")),
                                    rank=8, adapters=2, device="cuda")
        with torch.no_grad():
            self.up.B.copy_(torch.randn(self.up.B.shape, generator=g, device="cuda") * 0.1)
        self.experts = I.ExpertsFP8.from_float(w(experts, width, hidden))

    def forward(self, x, plan, order, offsets):
        h = self.up(self.norm(x), plan)
        y = self.experts(h.index_select(0, order), offsets)
        return x + torch.zeros_like(x).index_copy(0, order, y)


def batch(tokens, seed, width=256, experts=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
    plan = I.adapter_plan(torch.randint(-1, 2, (tokens,), generator=g, device="cuda").int(), 2)
    pick = torch.randint(0, experts, (tokens,), generator=g, device="cuda")
    order = torch.argsort(pick, stable=True)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(pick, minlength=experts).cumsum(0)
    return x, plan, order, offsets


def plain(block, x, order, offsets, index):
    """The block in 64 bits with the weights that the codes stand for and
    without FP8 rounding of tokens."""
    xd = x.double()
    n = torch.nn.functional.layer_norm(xd, (xd.shape[1],), block.norm.weight.double(), block.norm.bias.double(), 1e-5)
    base = block.up.base
    W = I.fp8_dequantize_weight(base.codes, base.scales, base.in_features, torch.float32).double()
    h = n @ W.T
    for e in range(2):
        rows = (index == e).nonzero()[:, 0]
        h[rows] += (n[rows] @ block.up.A[e].double().T) @ block.up.B[e].double().T
    E = I.fp8_dequantize_weight(block.experts.codes, block.experts.scales, block.experts.in_features, torch.float32).double()
    out = xd.clone()
    at = offsets.tolist()
    for e in range(len(at) - 1):
        rows = order[at[e]:at[e + 1]]
        out[rows] += h[rows] @ E[e].T
    return out


def test_block_against_64_bits():
    block = Block()
    x, plan, order, offsets = batch(200, 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    torch.randn(200, 256, generator=g, device="cuda")
    index = torch.randint(-1, 2, (200,), generator=g, device="cuda")
    with torch.no_grad():
        y = block(x, plan, order, offsets)
    with torch.no_grad():
        ref = plain(block, x, order, offsets, index)
    # every product's tokens are rounded by at most 2^-4 of a value; a sum of
    # many such errors of random signs stays far below their bound, 2^-4 of
    # the magnitudes: the 2-norm of the whole is held to it
    err, size = (y.double() - ref).norm(), (ref - x.double()).norm()
    assert float(err) <= 2 * 2.0 ** -4 * float(size) + 2.0 ** -8 * float(ref.norm())


def test_step_changes_what_trains_and_clips():
    block = Block()
    params = [p for p in block.parameters() if p.requires_grad]
    assert {p.shape for p in params} >= {block.up.A.shape, block.up.B.shape, block.norm.weight.shape}
    frozen = [b.clone() for b in (block.up.base.codes.view(torch.uint8), block.experts.codes.view(torch.uint8))]
    opt = I.AdamW(params, lr=1e-2)
    x, plan, order, offsets = batch(300, 2)
    x.requires_grad_(True)
    gy = torch.randn(300, 256, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    block(x, plan, order, offsets).backward(gy)
    assert torch.isfinite(x.grad).all() and all(torch.isfinite(p.grad).all() for p in params)
    total = torch.sqrt(sum((p.grad.double() ** 2).sum() for p in params))
    before = [p.detach().clone() for p in params]
    norm = opt.step(max_norm=0.5)
    assert abs(float(norm) - float(total)) <= float(total) * 18 * 2.0 ** -24
    assert all(not torch.equal(p, b) for p, b in zip(params, before))
    assert torch.equal(frozen[0], block.up.base.codes.view(torch.uint8))
    assert torch.equal(frozen[1], block.experts.codes.view(torch.uint8))
    # a gradient that is not finite: the step changes nothing
    held = [p.detach().clone() for p in params]
    opt.zero_grad()
    gy[7, 7] = float("inf")
    block(x, plan, order, offsets).backward(gy)
    assert not torch.isfinite(opt.step(max_norm=0.5))
    assert all(torch.equal(p, h) for p, h in zip(params, held))


def test_single_tokens_give_the_rows_of_the_batch():
    """Decoding one token at a time takes other kernels than the batch: each
    sums a row's blocks in its own order, 2^-24 a step, before the one rounding
    to 16 bits."""
    g = torch.Generator(device="cuda").manual_seed(5)
    W = torch.randn(384, 1024, generator=g, device="cuda") * 0.03
    layer = I.LinearFP8.from_float(W)
    x = torch.randn(300, 1024, generator=g, device="cuda").half()
    many = layer(x)
    size = x.abs().double() @ W.abs().double().T
    for rows in (slice(0, 1), slice(7, 20), slice(100, 140), slice(200, 264)):
        few = layer(x[rows])
        # sums: as the layer's own bound; two roundings to fp16
        lim = size[rows] * (1 + 2.0 ** -3) * 2 * (128 * 2.0 ** -23 + 12 * 2.0 ** -24) + many[rows].double().abs() * 2.0 ** -10 + 2.0 ** -24
        assert bool(((few.double() - many[rows].double()).abs() <= lim).all())


def test_forward_and_backward_in_a_graph():
    """The functional calls of one layer's step captured once, replayed on new tokens."""
    g = torch.Generator(device="cuda").manual_seed(6)
    codes, scales = I.fp8_quantize_weight(torch.randn(512, 640, generator=g, device="cuda"))
    params = [torch.nn.Parameter(torch.zeros(512, device="cuda"))]
    grads = [torch.empty(512, device="cuda")]
    m, v = (torch.zeros(I.adamw_state_size(params), device="cuda") for _ in range(2))
    counts = I.adamw_counts(params)
    x = torch.zeros(700, 640, device="cuda").bfloat16()

    def step():
        y = I.fp8_forward(x, codes, scales, 640, params[0].detach())
        gx, gb = I.fp8_backward_input(y, codes, scales, 640, bias_dtype=torch.float32)
        grads[0].copy_(gb)
        norm, scale, inf = I.grad_norm(grads, 1.0)
        I.adamw_step(params, grads, m, v, counts, 1e-2, grad_scale=scale, found_inf=inf)
        return y, gx, norm

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.no_grad():
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        outs = step()
    state = [t.clone() for t in (params[0].detach(), m, v, counts)]
    for seed in (1, 2):
        g.manual_seed(seed)
        x.copy_(torch.randn(700, 640, generator=g, device="cuda"))
        graph.replay()
        got = [o.clone() for o in outs] + [t.clone() for t in (params[0].detach(), m, v, counts)]
        with torch.no_grad():
            for t, s in zip((params[0], m, v, counts), state):
                t.copy_(s)
            expect = [*step(), params[0].detach(), m, v, counts]
            assert all(torch.equal(a[..., :1] if a is got[-1] else a, b[..., :1] if a is got[-1] else b) for a, b in zip(got, expect))
            state = [t.clone() for t in (params[0].detach(), m, v, counts)]
