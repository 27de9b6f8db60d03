"""The block-scaled FP8 layers on a GB300 against their definition in 64 bits."""
import pytest
import torch

import _fp8 as R
import int8_quantized_linear_i8lt_gb300 as I
from int8_quantized_linear_i8lt_gb300 import _lib

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def tokens(M, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, C, generator=g)
    x *= torch.where(torch.rand(C, generator=g) < 0.01, 20.0, 1.0)
    if M > 2:
        x[1] = 0                                     # a row of zeros
        x[2, : C // 2] *= 2.0 ** -12                 # blocks of very different size
    return x.to(dtype)


def weights(N, K, seed, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(N, K, generator=g) * 0.02).to(dtype)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("M,C", [(1, 1), (1, 128), (3, 129), (5, 16), (2, 130), (33, 1100), (7, 8192), (300, 519)])
def test_quantize(M, C, dtype):
    x = tokens(M, C, dtype, M + C)
    q, s = I.fp8_quantize(x.cuda())
    rq, rs = R.rows(x)
    assert torch.equal(q[:, :C].cpu().double(), rq)
    assert not q[:, C:].float().any()
    assert torch.equal(s.cpu().double(), rs)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 127), (200, 300), (519, 1100)])
def test_quantize_weight(N, K, dtype):
    W = weights(N, K, N + K, dtype)
    W[0, 0] = 3.0
    both = torch.stack([W, W * 0.25])
    q, s = I.fp8_quantize_weight(both.cuda())
    assert q.shape == (2, N, (K + 15) // 16 * 16) and s.shape == (2, -(-N // 128), -(-K // 128))
    for e in range(2):
        rq, rs = R.weight(both[e])
        assert torch.equal(q[e, :, :K].cpu().double(), rq) and not q[e, :, K:].float().any()
        assert torch.equal(s[e].cpu().double(), rs)
    one = I.fp8_quantize_weight(both[1].cuda())
    assert torch.equal(one[0].view(torch.uint8), q[1].view(torch.uint8)) and torch.equal(one[1], s[1])
    back = I.fp8_dequantize_weight(q, s, K, F32)
    expect = torch.stack([R.expand_weight(*R.weight(both[e])) for e in range(2)])
    assert torch.equal(back.cpu(), expect.float())


SIZES = [(1, 1, 1), (1, 128, 128), (2, 130, 127), (3, 16, 8), (1, 4096, 520), (17, 300, 200), (128, 256, 128),
         (129, 384, 257), (64, 2048, 1024), (300, 1000, 1000), (513, 640, 640), (777, 1100, 519), (1025, 512, 1536),
         (2300, 300, 2600), (2600, 2310, 280),
         (40, 520, 260), (64, 256, 8200), (33, 8200, 130), (200, 130, 9001)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_forward(M, K, N, dtype):
    x, W = tokens(M, K, dtype, 1), weights(N, K, 2)
    bias = None if N % 2 else torch.randn(N, generator=torch.Generator().manual_seed(3)).to(dtype if N % 4 else F32)
    q, s = I.fp8_quantize_weight(W.cuda())
    y = I.fp8_forward(x.cuda(), q, s, K, None if bias is None else bias.cuda())
    ref, size = R.product(x, R.expand_weight(*R.weight(W)), bias)
    assert y.shape == (M, N) and y.dtype == dtype
    R.check(y, ref, size, K, "y")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_backward_input(M, K, N, dtype):
    G, W = tokens(M, N, dtype, 4), weights(N, K, 5)
    q, s = I.fp8_quantize_weight(W.cuda())
    gx, gb = I.fp8_backward_input(G.cuda(), q, s, K, bias_dtype=F32)
    ref, size = R.product(G, R.expand_weight(*R.weight(W)), transposed=True)
    R.check(gx, ref, size, N, "gx")
    total = G.double().sum(0)
    # sums of M terms in 32 bits, in any order
    assert bool(((gb.cpu().double() - total).abs() <= G.double().abs().sum(0) * M * 2.0 ** -24 + 1e-30).all())
    only = I.fp8_backward_input(G.cuda(), q, s, K, need_grad_A=False, bias_dtype=F32)
    assert only[0] is None and torch.equal(only[1], gb)
    assert torch.equal(I.fp8_backward_input(G.cuda(), q, s, K)[0], gx)


def clamped(offsets, M):
    """The row ranges that offsets stand for."""
    out, top = [], 0
    for o in offsets:
        top = max(top, min(max(o, 0), M))
        out.append(top)
    return out


GROUPS = [
    (1, [0, 1], 128, 128), (5, [0, 0, 0, 5, 5], 300, 200), (40, [0, 7, 7, 19, 40], 256, 384),
    (300, [0, 130, 131, 290], 640, 257), (520, [3, 260, 511], 130, 520), (64, [0, 0], 128, 16),
    (200, list(range(0, 201, 2)), 144, 136), (1333, [0, 300, 300, 811, 1000, 1312], 1100, 519),
    (0, [0, 0, 0], 64, 64), (2650, [11, 700, 700, 1500, 2640], 200, 2100), (2600, [0, 255, 513, 1300, 2600], 2200, 136),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,offsets,K,N", GROUPS)
def test_experts(M, offsets, K, N, dtype):
    E = len(offsets) - 1
    W = torch.stack([weights(N, K, 10 + e) for e in range(E)])
    q, s = I.fp8_quantize_weight(W.cuda())
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    for transposed in (False, True):
        C, Rn = (N, K) if transposed else (K, N)
        call = I.fp8_experts_backward_input if transposed else I.fp8_experts_forward
        t = tokens(M, C, dtype, 6)
        y = call(t.cuda(), q, s, K, off)
        kept = torch.full((M, Rn), 7.0, dtype=dtype).cuda()
        assert call(t.cuda(), q, s, K, off, out=kept) is kept
        inside = torch.zeros(M, dtype=torch.bool)
        for e in range(E):
            a, b = offsets[e], offsets[e + 1]
            inside[a:b] = True
            if b > a:
                ref, size = R.product(t[a:b], R.expand_weight(*R.weight(W[e])), transposed=transposed)
                R.check(y[a:b], ref, size, C, f"expert {e}")
        assert not y.cpu()[~inside].float().any()
        assert torch.equal(kept.cpu()[inside], y.cpu()[inside]) and bool((kept.cpu()[~inside] == 7).all())


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [-5, 10, 500, 600], [90, 10, 0, 100], [2 ** 31 - 1, 0, -2 ** 31, 5]])
def test_experts_offsets_out_of_order(offsets):
    """Ranges never overlap and never leave the tokens."""
    M, K, N, E = 100, 128, 64, 3
    W = torch.stack([weights(N, K, 20 + e) for e in range(E)])
    q, s = I.fp8_quantize_weight(W.cuda())
    x = tokens(M, K, F16, 7).cuda()
    got = I.fp8_experts_forward(x, q, s, K, torch.tensor(offsets, dtype=torch.int32).cuda())
    expect = I.fp8_experts_forward(x, q, s, K, torch.tensor(clamped(offsets, M), dtype=torch.int32).cuda())
    assert torch.equal(got, expect)


def test_experts_neighbours_do_not_mix():
    """A NaN in one expert's weight, or in rows of none, reaches no other's outputs."""
    M, K, N, E = 260, 200, 150, 3
    W = torch.stack([weights(N, K, 30 + e) for e in range(E)])
    x = tokens(M, K, BF16, 8)
    off = torch.tensor([0, 100, 120, 250], dtype=torch.int32).cuda()
    q, s = I.fp8_quantize_weight(W.cuda())
    for transposed in (False, True):
        call = I.fp8_experts_backward_input if transposed else I.fp8_experts_forward
        t = tokens(M, N, BF16, 8) if transposed else x
        clean = call(t.cuda(), q, s, K, off)
        bad, tb = W.clone(), t.clone()
        bad[1] = float("nan")
        tb[250:] = float("inf")
        tb[119] = float("nan")
        qb, sb = I.fp8_quantize_weight(bad.cuda())
        y = call(tb.cuda(), qb, sb, K, off)
        assert y[100:120].isnan().all()
        assert torch.equal(y[:100], clean[:100]) and torch.equal(y[120:], clean[120:])


def test_not_finite():
    M, K, N = 140, 256, 200
    x, W = tokens(M, K, F16, 9), weights(N, K, 11)
    q, s = I.fp8_quantize_weight(W.cuda())
    clean = I.fp8_forward(x.cuda(), q, s, K)
    x[5, 3], x[130, 255] = float("nan"), float("inf")
    y = I.fp8_forward(x.cuda(), q, s, K)
    rest = [m for m in range(M) if m not in (5, 130)]
    assert y[5].isnan().all() and y[130].isnan().all() and torch.equal(y[rest], clean[rest])
    W[150, 7] = float("inf")                         # its block is rows 128 to 199
    q, s = I.fp8_quantize_weight(W.cuda())
    y = I.fp8_forward(x.cuda(), q, s, K)
    assert y[:, 128:].isnan().all() and torch.equal(y[rest][:, :128], clean[rest][:, :128])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,N", [(1, 300, 39200), (16, 9001, 130), (7, 1111, 520), (16, 2056, 4100), (5, 136, 40001)])
def test_few_tokens(M, K, N, dtype):
    """Several tiles a CTA, many blocks a CTA, rows on no 16 bytes; a bias gradient
    beside it changes no bit of the product."""
    x, W = tokens(M, K, dtype, 31), weights(N, K, 32)
    q, s = I.fp8_quantize_weight(W.cuda())
    y = I.fp8_forward(x.cuda(), q, s, K)
    ref, size = R.product(x, R.expand_weight(*R.weight(W)))
    R.check(y, ref, size, K, "y")
    G = tokens(M, N, dtype, 33).cuda()
    assert torch.equal(I.fp8_backward_input(G, q, s, K)[0], I.fp8_backward_input(G, q, s, K, bias_dtype=F32)[0])


def test_few_rows_of_an_uneven_share():
    M, K, N, E = 500, 200, 130, 64
    W = torch.stack([weights(N, K, 40 + e) for e in range(E)])
    q, s = I.fp8_quantize_weight(W.cuda())
    cuts = [0, 0, 3] + [403] * 20 + list(range(404, 404 + 40)) + [450, 490]
    off = torch.tensor(cuts, dtype=torch.int32)
    assert len(cuts) == E + 1
    for transposed in (False, True):
        x = tokens(M, N if transposed else K, F16, 34)
        call = I.fp8_experts_backward_input if transposed else I.fp8_experts_forward
        y = call(x.cuda(), q, s, K, off.cuda())
        assert not y[490:].any()
        for e in range(E):
            a, b = cuts[e], cuts[e + 1]
            if a < b:
                ref, size = R.product(x[a:b], R.expand_weight(*R.weight(W[e])), transposed=transposed)
                R.check(y[a:b], ref, size, x.shape[1], f"expert {e}")


def test_few_tokens_in_two_graphs():
    K, N = 1024, 640
    q, s = I.fp8_quantize_weight(weights(N, K, 37).cuda())
    x = torch.zeros(4, K, dtype=F16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        I.fp8_forward(x, q, s, K)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.add_(1)                                # the product sees what the kernel before it wrote
            outs.append(I.fp8_forward(x, q, s, K))
    x.copy_(tokens(4, K, F16, 38))
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            graph.replay()
            assert torch.equal(out, I.fp8_forward(x, q, s, K))


def test_linear_on_the_grid_has_exact_differences():
    """Values the codes hold exactly: the layer is linear between them, and
    <g, f(x + e) - f(x)> = <gx, e>."""
    g = torch.Generator().manual_seed(12)
    M, K, N = 30, 260, 140
    grid = lambda *shape: torch.randint(-6, 7, shape, generator=g).double()
    x, e, G, W = grid(M, K), torch.randint(-1, 2, (M, K), generator=g).double(), grid(M, N), grid(N, K)
    for t in (x, G):                                 # every block's maximum is 7, with or without e
        t[:, ::128] = 7
        t[:, -1] = 7
    e[:, ::128] = 0
    e[:, -1] = 0
    W[::128, ::128] = 7
    W[-1, ::128] = W[::128, -1] = W[-1, -1] = 7
    layer = I.LinearFP8.from_float(W.float().cuda())
    assert torch.equal(layer.codes[:, :K].cpu().double(), W * 64)
    xa = x.half().cuda().requires_grad_(True)
    ya = layer(xa)
    yb = layer((x + e).half().cuda())
    ya.backward(G.half().cuda())
    # y and gx are sums below 2^11 * 7^2 of exact products: half's step decides
    size = x.abs() @ W.abs().T
    assert bool(((ya.detach().cpu().double() - x @ W.T).abs() <= (x @ W.T).abs() * 2.0 ** -11 + size * 2.0 ** -16).all())
    left, right = float((G * (yb - ya).detach().cpu().double()).sum()), float((xa.grad.cpu().double() * e).sum())
    slack = float(((x @ W.T).abs() * 2 + 60) .mul(2.0 ** -10).mul(G.abs()).sum() + ((G @ W).abs().mul(2.0 ** -10) * e.abs()).sum())
    assert abs(left - float((G * (e @ W.T)).sum())) <= slack and abs(left - right) <= 2 * slack


def test_modules_and_autograd():
    g = torch.Generator(device="cuda").manual_seed(13)
    W = torch.randn(200, 300, generator=g, device="cuda") * 0.05
    b = torch.randn(200, generator=g, device="cuda").bfloat16()
    layer = I.LinearFP8.from_float(W, b)
    x = torch.randn(4, 9, 300, generator=g, device="cuda").bfloat16().requires_grad_(True)
    y = layer(x)
    gy = torch.randn(y.shape, generator=g, device="cuda").bfloat16()
    y.backward(gy)
    assert torch.equal(y.detach().reshape(-1, 200), I.fp8_forward(x.detach().reshape(-1, 300), layer.codes, layer.scales, 300, b))
    gx, gb = I.fp8_backward_input(gy.reshape(-1, 200), layer.codes, layer.scales, 300, bias_dtype=b.dtype)
    assert torch.equal(x.grad.reshape(-1, 300), gx) and torch.equal(layer.bias.grad, gb)
    other = I.LinearFP8(300, 200, device="cuda")
    other.load_state_dict(layer.state_dict())
    assert torch.equal(other(x), y)
    experts = I.ExpertsFP8.from_float(torch.stack([W, -W]))
    off = torch.tensor([0, 10, 30], dtype=torch.int32, device="cuda")
    t = x.detach().reshape(-1, 300).clone().requires_grad_(True)
    z = experts(t, off)
    z.backward(gy.reshape(-1, 200))
    assert not z[30:].any() and not t.grad[30:].any()
    assert torch.equal(t.grad[:10], gx[:10]) and torch.equal(t.grad[10:30], -gx[10:30])
    with pytest.raises(RuntimeError):                # differentiating twice
        t2 = t.detach().clone().requires_grad_(True)
        (a,) = torch.autograd.grad(experts(t2, off).sum(), t2, create_graph=True)
        a.sum().backward()


def test_views_streams_and_workspaces():
    g = torch.Generator(device="cuda").manual_seed(14)
    W = torch.randn(96, 160, generator=g, device="cuda")
    q, s = I.fp8_quantize_weight(W)
    base = torch.randn(70, 161, generator=g, device="cuda").half()
    x = base[1:, 1:]                                 # neither contiguous nor aligned
    y = I.fp8_forward(x, q, s, 160)
    assert torch.equal(y, I.fp8_forward(x.contiguous(), q, s, 160))
    flat = torch.empty(69 * 160 + 1, dtype=F16, device="cuda")[1:].view(69, 160).copy_(x)
    assert torch.equal(y, I.fp8_forward(flat, q, s, 160))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = I.fp8_forward(flat, q, s, 160)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, z)
    ws = torch.empty(_lib.i8lt_fp8_workspace_size(69, 160), dtype=torch.uint8, device="cuda").fill_(255)
    assert torch.equal(y, I.fp8_forward(flat, q, s, 160, ws=ws)) and I.device_status(ws)[0] == 0


def test_offsets_beyond_32_bits():
    """Tokens of 2^31 elements and more, forward and back, and experts' codes of
    as many bytes: the last rows and the last expert."""
    M, K, N = 265000, 8192, 160
    q, s = I.fp8_quantize_weight(weights(N, K, 50).cuda())
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[-200:] = tokens(200, K, BF16, 51).cuda()
    y = I.fp8_forward(x, q, s, K)
    assert torch.equal(y[-200:], I.fp8_forward(x, q, s, K)[-200:]) and not y[:-200].any()
    ref, size = R.product(x[-200:].cpu(), R.expand_weight(*R.weight(weights(N, K, 50))))
    R.check(y[-200:], ref, size, K, "y")
    del x
    G = torch.zeros(M, N, dtype=BF16, device="cuda")
    G[-200:] = tokens(200, N, BF16, 52).cuda()
    gx = I.fp8_backward_input(G, q, s, K)[0]
    ref, size = R.product(G[-200:].cpu(), R.expand_weight(*R.weight(weights(N, K, 50))), transposed=True)
    R.check(gx[-200:], ref, size, N, "gx")
    assert not gx[:100].any() and not gx[-300:-200].any()
    del gx, G
    E, N, K = 130, 4096, 4200                        # 130 x 4096 x 4208 codes
    last = weights(N, K, 53)
    W = torch.zeros(E, N, K, dtype=BF16, device="cuda")
    W[-1] = last.cuda()
    q, s = I.fp8_quantize_weight(W)
    assert q.numel() > 2 ** 31
    for rows in (3, 200):
        x = tokens(rows, K, BF16, 54)
        off = torch.tensor([0] * E + [rows], dtype=torch.int32).cuda()
        y = I.fp8_experts_forward(x.cuda(), q, s, K, off)
        ref, size = R.product(x, R.expand_weight(*R.weight(last.to(BF16))))
        R.check(y, ref, size, K, f"{rows} rows")


def test_two_threads_at_once():
    """Calls from two threads on streams of their own share nothing."""
    import threading
    sizes = [(5, 2048, 1500), (300, 640, 900), (2600, 512, 1800), (40, 1100, 260)]
    work = []
    for i, (M, K, N) in enumerate(sizes):
        q, s = I.fp8_quantize_weight(weights(N, K, 60 + i).cuda())
        x, G = tokens(M, K, F16, 70 + i).cuda(), tokens(M, N, F16, 80 + i).cuda()
        call = lambda x=x, G=G, q=q, s=s, K=K: (I.fp8_forward(x, q, s, K),
                                                *I.fp8_backward_input(G, q, s, K, bias_dtype=F32),
                                                *I.grad_norm([x, G], 1.0))
        work.append((call, call()))
    torch.cuda.synchronize()
    wrong = []

    def run(order):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                for i in order:
                    call, expect = work[i]
                    if not all(torch.equal(a, b) for a, b in zip(call(), expect)):
                        wrong.append(i)
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(order,)) for order in ([0, 1, 2, 3], [2, 3, 1, 0])]
    for thread in threads:
        thread.start()
    for thread in threads:
        thread.join()
    assert not wrong


def test_captured_and_replayed():
    g = torch.Generator(device="cuda").manual_seed(15)
    W = torch.randn(2, 256, 384, generator=g, device="cuda")
    q, s = I.fp8_quantize_weight(W)
    x = torch.zeros(300, 384, device="cuda").half()
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    G = torch.zeros(300, 256, device="cuda").half()
    call = lambda: (I.fp8_forward(x, q[0], s[0], 384), I.fp8_experts_forward(x, q, s, 384, off),
                    I.fp8_experts_backward_input(G, q, s, 384, off), *I.fp8_backward_input(G, q[1], s[1], 384, bias_dtype=F32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for seed, cuts in ((1, [0, 100, 300]), (2, [0, 0, 220]), (3, [40, 290, 300])):
        g.manual_seed(seed)
        x.copy_(torch.randn(300, 384, generator=g, device="cuda"))
        G.copy_(torch.randn(300, 256, generator=g, device="cuda"))
        off.copy_(torch.tensor(cuts, dtype=torch.int32))
        graph.replay()
        for a, b in zip(outs, call()):
            assert torch.equal(a, b)


def test_refusals():
    W = torch.randn(64, 96, device="cuda")
    q, s = I.fp8_quantize_weight(W)
    x = torch.randn(8, 96, device="cuda").half()
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    q2, s2 = I.fp8_quantize_weight(torch.stack([W, W]))
    calls = [
        lambda: I.fp8_forward(x.float(), q, s, 96),                                 # f32 is no compute type
        lambda: I.fp8_forward(x[:, :95], q, s, 96), lambda: I.fp8_forward(x[0], q, s, 96),
        lambda: I.fp8_forward(x, q.view(torch.uint8), s, 96), lambda: I.fp8_forward(x, q, s.half(), 96),
        lambda: I.fp8_forward(x, q, s[:, :0], 96), lambda: I.fp8_forward(x, q, s, 96, torch.zeros(63, device="cuda")),
        lambda: I.fp8_forward(x, q, s, 96, out=torch.empty(8, 64, device="cuda")),
        lambda: I.fp8_forward(x, q, s, 96, out=torch.empty(64, 8, device="cuda").half().T),
        lambda: I.fp8_forward(x, q, s, 96, ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: I.fp8_forward(x, q.cpu(), s, 96), lambda: I.fp8_forward(x, q2, s2, 96),
        lambda: I.fp8_experts_forward(x, q, s, 96, off), lambda: I.fp8_experts_forward(x, q2, s2, 96, off.long()),
        lambda: I.fp8_experts_forward(x, q2, s2, 96, off[:2]), lambda: I.fp8_experts_forward(x, q2, s2, 96, off.cpu()),
        lambda: I.fp8_backward_input(x, q, s, 96), lambda: I.fp8_quantize_weight(W[0]),
        lambda: I.fp8_quantize_weight(W.long()), lambda: I.fp8_quantize(x[0]),
        lambda: I.fp8_quantize_weight(torch.zeros(1025, 1, 1, device="cuda")),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(I.I8LTError):
            call()
            pytest.fail(f"call {i} was not refused")
    empty = I.fp8_forward(x[:0], q, s, 96)
    assert empty.shape == (0, 64)
    gx, gb = I.fp8_backward_input(torch.zeros(0, 64, device="cuda").half(), q, s, 96, bias_dtype=F16)
    assert gx.shape == (0, 96) and not gb.any()
