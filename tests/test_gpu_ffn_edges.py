"""The feed-forward operators at the edges of what their calls allow: rows that pass the registers, values
far from one, zeros and non-finite rows in the backward products, offsets past 32 bits, captured backward
passes, workspaces and operands that are refused."""
import pytest
import torch

import ffn_ref as ref
import w4a16_gemm_awq_b200 as w4

pytestmark = pytest.mark.gpu


def cuda(layer):
    return tuple(t.cuda() for t in layer)


def bits(t):
    return t.view(torch.int16)


def run_gated_backward(M, K, F, name="silu"):
    gate, wg = ref.pack_layer(M, F, K)
    up, wu = ref.pack_layer(M + 1, F, K)
    dh, g, u = ref.bf(1, M, F), ref.bf(2, M, F, spread=2.0), ref.bf(3, M, F, spread=2.0)
    dx = w4.w4a16_gated_backward(dh.cuda(), g.cuda(), u.cuda(), cuda(gate), cuda(up), activation=name)
    w4.check_device_status()
    ref.check(dx, *ref.gated_backward(dh, g, u, wg, wu, name), "dx", norm2=ref.ONE_ROUNDING)


@pytest.mark.parametrize("M,F", [(3, 16384), (3, 16512), (700, 16512), (900, 128), (400, 2176)])
def test_gated_backward_rows(M, F):
    """Rows in the ring (several per block), the longest that fit there, and longer ones, read twice."""
    run_gated_backward(M, 1024, F)


@pytest.mark.parametrize("M", [20, 3000])
def test_long_operand_rows(M):
    """Rows past the 8192 channels that the conversion to fp16 keeps in registers; more rows than blocks."""
    K, N = 10240, 128
    gate, wg = ref.pack_layer(1, N, K)
    up, wu = ref.pack_layer(2, N, K)
    x = ref.bf(3, M, K)
    h, e, _, _ = ref.gated(x, wg, wu, gate, up, 128, "silu")
    ref.check(w4.w4a16_gated(x.cuda(), cuda(gate), cuda(up)), h, e, "h", norm2=ref.ONE_ROUNDING)
    layer, w = ref.pack_layer(4, K, 1024)
    dx, db = w4.w4a16_linear_fused_backward(x.cuda(), *cuda(layer), bias_grad=False)
    assert db is None
    want, e, _, _ = ref.linear_backward(x, None, w, "none")
    ref.check(dx, want, e, "dx", norm2=ref.ONE_ROUNDING)
    w4.check_device_status()


@pytest.mark.parametrize("M,N", [(1, 128), (17, 384), (2000, 128), (5000, 1152), (513, 8320), (40, 4224), (200, 16384),
                                 (40, 16512), (700, 17536)])
def test_bias_gradient_runs(M, N):
    """Column sums over one run of rows and over many, rows within the registers and longer ones."""
    layer, w = ref.pack_layer(N, N, 1024)
    dy, pre = ref.bf(1, M, N), ref.bf(2, M, N, spread=2.0)
    dx, db = w4.w4a16_linear_fused_backward(dy.cuda(), *cuda(layer), pre=pre.cuda(), activation="gelu", bias_grad=True)
    w4.check_device_status()
    want, e, b, eb = ref.linear_backward(dy, pre, w, "gelu")
    ref.check(dx, want, e, "dx", norm2=ref.ONE_ROUNDING)
    ref.check(db, b, eb, "dbias", norm2=2.0 ** -16)


def products(M, K=1024, N=256):
    """The products without an activation as functions of one operand that they are linear in (the gated
    block: of degree 2), with that operand's width."""
    layer, up = (cuda(ref.pack_layer(s, N, K)[0]) for s in (1, 2))
    g, u = ref.bf(8, M, N).cuda(), ref.bf(9, M, N).cuda()
    return [(lambda x: w4.w4a16_linear_fused(x, *layer), K, 1),
            (lambda x: w4.w4a16_gated(x, layer, up, activation="none"), K, 2),
            (lambda dy: w4.w4a16_linear_fused_backward(dy, *layer)[0], N, 1),
            (lambda dy: w4.w4a16_linear_fused_backward(dy, *layer, bias_grad=True)[0], N, 1),
            (lambda dh: w4.w4a16_gated_backward(dh, g, u, layer, up, activation="none"), N, 1)]


@pytest.mark.parametrize("M", [7, 60])
def test_rows_far_from_one(M):
    """Rows times a power of two give the output times its power, to the bit: sums in 32 bits take it along,
    and an operand in 16 bits has its row's scale."""
    e = torch.tensor([(-50, -20, 0, 20, 50)[m % 5] for m in range(M)])
    for f, width, degree in products(M):
        x = ref.bf(5, M, width)
        base = f(x.cuda()).cpu()
        got = f(torch.ldexp(x.float(), e[:, None]).to(torch.bfloat16).cuda()).cpu()
        want = torch.ldexp(base.double(), degree * e[:, None]).to(torch.bfloat16)
        assert torch.equal(bits(got), bits(want))
    w4.check_device_status()


def test_small_values_beside_a_large_one():
    """Values 2^-26 of their row's largest keep all their bits in the 16-bit operand: the large one meets a
    weight of zero, so the others are all that is seen."""
    M, K, N = 40, 1024, 256
    (qw, sc, z), w = ref.pack_layer(3, N, K)
    zeros = (z[0].view(-1, 1) >> torch.arange(0, 32, 4)) & 15
    qw[:, 0] = (qw[:, 0] & ~15) | zeros.reshape(-1).to(torch.int32)
    w[:, 0] = 0
    x = ref.bf(4, M, K).clamp(-3, 3) * 2.0 ** -26
    x[:, 0] = 1.5
    layer = cuda((qw, sc, z))
    up, wu = ref.pack_layer(5, N, K)
    _, g, u = w4.w4a16_gated(x.cuda(), layer, cuda(up), save=True)
    small = x.clone()
    small[:, 0] = 0
    p, e = ref.projection(small, w, (qw, sc, z), 128, half=True)
    ref.check(g, p, e + ref.STEP * (p.abs() + e) + 2.0 ** -38 * 1.5 * w.abs().sum(1), "g", norm2=ref.ONE_ROUNDING)
    p, e = ref.projection(x, wu, up, 128, half=True)
    ref.check(u, p, e + ref.STEP * (p.abs() + e), "u", norm2=ref.ONE_ROUNDING)


@pytest.mark.parametrize("M", [6, 90])
def test_zero_and_non_finite_rows(M):
    """A row of zeros gives zeros; a NaN or an infinity reaches its own row only."""
    for f, width, _ in products(M):
        x = ref.bf(6, M, width)
        base = f(x.cuda()).cpu()
        x[1] = 0
        x[2, 17] = float("nan")
        x[4, 100] = float("-inf")
        got = f(x.cuda()).cpu()
        assert not got[1].any()
        assert torch.isnan(got[2]).all()
        assert not torch.isfinite(got[4]).any()
        keep = [m for m in range(M) if m not in (1, 2, 4)]
        assert torch.equal(bits(got[keep]), bits(base[keep]))
    w4.check_device_status()


@pytest.mark.parametrize("name", ref.ACTS)
def test_activations_of_large_values(name):
    """Values past the range of the exponential: the activations and their derivatives saturate."""
    M, K, N = 20, 1024, 128
    layer, w = ref.pack_layer(1, N, K)
    d = cuda(layer)
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 9.0, -9.0, 40.0, -40.0, 100.0, -100.0, 1e6, -1e6, 1e15, -1e15, 1e25, -1e25,
                      3e38, -3e38]).to(torch.bfloat16)
    bias = v.repeat(8)[:N].contiguous()
    for m in (3, M):
        x = torch.zeros(m, K, dtype=torch.bfloat16)
        y = w4.w4a16_linear_fused(x.cuda(), *d, bias=bias.cuda(), activation=name)
        want, e, _, _ = ref.linear(x, w, layer, 128, bias=bias, name=name)
        ref.check(y, want, e, "y", norm2=ref.ONE_ROUNDING)
    pre = bias.repeat(M, 1)
    dy = ref.bf(2, M, N)
    dx, db = w4.w4a16_linear_fused_backward(dy.cuda(), *d, pre=pre.cuda(), activation=name, bias_grad=True)
    da = ref.act(pre.double(), name)[1]
    dp = dy.double() * da
    # saturated derivatives are exact; the others here have |p| <= 100
    slack = ref.FAST * dy.double().abs() * (1 + pre.double().abs().clamp(max=100.0))
    want, e = ref._back(dp, dy.double().abs().amax(1, True), slack, w, N)
    ref.check(dx, want, e, "dx", norm2=ref.ONE_ROUNDING)
    ref.check(db, dp.sum(0), slack.sum(0) + M * 2.0 ** -24 * dp.abs().sum(0), "dbias", norm2=2.0 ** -16)


def test_offsets_past_32_bits():
    """More than 2^31 elements in an operand or an output: the last rows are right."""
    M, last = 131072 + 5, 6
    layer, w = ref.pack_layer(1, 16512, 1024)
    x = torch.randn(M, 1024, device="cuda").to(torch.bfloat16)
    y = w4.w4a16_linear_fused(x, *cuda(layer))
    w4.check_device_status()
    # with the rows beside them, for the bound of the product of many tokens
    p, e, _, _ = ref.linear(x[-20:].cpu(), w, layer, 128)
    ref.check(y[-last:], p[-last:], e[-last:], "y")
    del y
    F = 8320
    (gate, wg), (up, wu) = ref.pack_layer(2, F, 1024), ref.pack_layer(3, F, 1024)
    dh, g, u = (torch.empty(M, F, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(3))
    dx = w4.w4a16_gated_backward(dh, g, u, cuda(gate), cuda(up))
    w4.check_device_status()
    ref.check(dx[-last:], *ref.gated_backward(dh[-last:].cpu(), g[-last:].cpu(), u[-last:].cpu(), wg, wu, "silu"), "dx",
              norm2=ref.ONE_ROUNDING)
    del dx, g, u
    M, K = 70001, 32768
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_()
    nw = ref.bf(5, K)
    y, _ = w4.awq_rmsnorm(x, nw.cuda())
    w4.check_device_status()
    _, v = ref.norm(x[-last:].cpu(), None, nw, None, 1e-6)
    ref.check(y[-last:], v, (ref.STEP + 2.0 ** -16) * v.abs(), "norm")


@pytest.mark.parametrize("M", [3, 150])
def test_captured_backward(M):
    """The backward calls captured once, replayed on new values, with eager calls in between."""
    K, F = 1024, 2048
    gate, up, down = cuda(ref.pack_layer(1, F, K)[0]), cuda(ref.pack_layer(2, F, K)[0]), cuda(ref.pack_layer(3, K, F)[0])
    nw, s = ref.bf(4, K).cuda(), (ref.bf(5, K).float().abs() + 0.5).cuda()

    def step(do, h, g, u, pre):
        da, db = w4.w4a16_linear_fused_backward(do, *down, pre=pre, activation="gelu", bias_grad=True)
        dy = w4.w4a16_gated_backward(da, g, u, gate, up)
        dx, dw = w4.awq_rmsnorm_backward(dy, h, nw, s=s, dh=do)
        return dx, dw, db

    def values(seed):
        return [ref.bf(seed + i, M, n).cuda() for i, n in enumerate((K, K, F, F, K))]
    held = values(10)
    eager = step(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*held)
    for seed in (10, 20, 30):
        new = values(seed)
        for a, b in zip(held, new):
            a.copy_(b)
        want = step(*new)
        graph.replay()
        again = step(*new)
        for a, b, c in zip(out, want, again):
            assert torch.equal(a, b) and torch.equal(b, c)
    assert all(torch.equal(a, b) for a, b in zip(eager, step(*values(10))))
    w4.check_device_status()


def test_refused_operands():
    M, K, N = 20, 1024, 128
    layer = cuda(ref.pack_layer(1, N, K)[0])
    x = ref.bf(1, M, K + 8).cuda()
    flat = ref.bf(2, 1, M * K + 8).cuda().reshape(-1)
    nw = ref.bf(3, K).cuda()
    h = ref.bf(4, M, N).cuda()
    for bad in (x[:, :K], x[:, :K].float().contiguous(), x[:0, :K], x[0, :K], x[:, :K].cpu().contiguous()):
        for f in (lambda v: w4.w4a16_linear_fused(v, *layer), lambda v: w4.w4a16_gated(v, layer, layer),
                  lambda v: w4.awq_rmsnorm(v, nw), lambda v: w4.awq_rmsnorm_e4m3(v, nw),
                  lambda v: w4.awq_rmsnorm_backward(v, v, nw)):
            with pytest.raises((ValueError, w4.W4A16Error)):
                f(bad)
    odd = flat[1:1 + M * K].view(M, K)  # not on a 16-byte boundary
    for f in (lambda v: w4.w4a16_linear_fused(v, *layer), lambda v: w4.w4a16_gated(v, layer, layer),
              lambda v: w4.awq_rmsnorm(v, nw), lambda v: w4.awq_rmsnorm_backward(v, v, nw)):
        with pytest.raises(w4.W4A16Error):
            f(odd)
    x = x[:, :K].contiguous()
    with pytest.raises(ValueError):
        w4.w4a16_linear_fused_backward(h, *layer, activation="silu")  # no pre
    with pytest.raises(ValueError):
        w4.w4a16_linear_fused(x, *layer, residual=h[:, :64])
    with pytest.raises(ValueError):
        w4.w4a16_gated(x, layer, cuda(ref.pack_layer(2, 2 * N, K)[0]))
    with pytest.raises(ValueError):
        w4.w4a16_linear_fused(x, *layer, group_size=256)


def test_small_workspaces_are_refused():
    M, K, N = 40, 8192, 256
    layer = cuda(ref.pack_layer(1, N, K)[0])
    x, dy = ref.bf(1, M, K).cuda(), ref.bf(2, M, N).cuda()
    nw = ref.bf(3, K).cuda()
    for op, f, n in ((w4.OP_LINEAR, lambda ws: w4.w4a16_linear_fused(x, *layer, workspace=ws), N),
                     (w4.OP_GATED, lambda ws: w4.w4a16_gated(x, layer, layer, workspace=ws), N),
                     (w4.OP_LINEAR_BACKWARD, lambda ws: w4.w4a16_linear_fused_backward(dy, *layer, workspace=ws), N),
                     (w4.OP_GATED_BACKWARD, lambda ws: w4.w4a16_gated_backward(dy, dy, dy, layer, layer, workspace=ws), N),
                     (w4.OP_RMSNORM_BACKWARD, lambda ws: w4.awq_rmsnorm_backward(x, x, nw, workspace=ws), 0)):
        need = w4.w4a16_fused_workspace_bytes(op, M, n, K)
        assert need > 0
        f(torch.zeros(need, dtype=torch.uint8, device="cuda"))
        for size in (need - 16, 16):
            with pytest.raises(w4.W4A16Error):
                f(torch.zeros(size, dtype=torch.uint8, device="cuda"))
    w4.check_device_status()


def test_cut_tiles_repeat():
    """Tiles cut along the contraction, few wide ones joined by halves, many narrow ones whole: the bits of
    fifty calls agree, two streams at once included, and the counters are zero afterwards."""
    one = [(cuda(ref.pack_layer(1, 384, 14336)[0]), 14336, 384), (cuda(ref.pack_layer(2, 4096, 1024)[0]), 1024, 4096),
           (cuda(ref.pack_layer(3, 256, 8192)[0]), 8192, 256)]
    up = cuda(ref.pack_layer(4, 256, 8192)[0])
    calls = []
    for M in (20, 64, 100, 130, 250, 300):
        for layer, K, N in one:
            x, dy = ref.bf(M, M, K).cuda(), ref.bf(M + 1, M, N).cuda()
            calls.append((w4.OP_LINEAR, M, N, K, lambda ws, x=x, w=layer: w4.w4a16_linear_fused(x, *w, workspace=ws)))
            calls.append((w4.OP_LINEAR_BACKWARD, M, N, K,
                          lambda ws, dy=dy, w=layer: w4.w4a16_linear_fused_backward(dy, *w, workspace=ws)[0]))
        calls.append((w4.OP_GATED, M, N, K, lambda ws, x=x, w=layer: w4.w4a16_gated(x, w, up, workspace=ws)))
    need = max(w4.w4a16_fused_workspace_bytes(*c[:4]) for c in calls)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in streams]
    for *_, f in calls:
        want = f(spaces[0]).clone()
        torch.cuda.synchronize()
        outs = []
        for _ in range(25):
            for st, ws in zip(streams, spaces):
                with torch.cuda.stream(st):
                    outs.append(f(ws))
        torch.cuda.synchronize()
        assert all(torch.equal(bits(o), bits(want)) for o in outs)
    w4.check_device_status()
    assert not any(ws[:131072].any() for ws in spaces)
