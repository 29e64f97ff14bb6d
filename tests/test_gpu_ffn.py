"""The feed-forward products on the GPU against 64-bit references: the W4A16 linear layer with its
fused epilogue, the gated block, and their backward passes."""
import pytest
import torch

import ffn_ref as ref
import w4a16_gemm_awq_b200 as w4

pytestmark = pytest.mark.gpu


def cuda(layer):
    return tuple(t.cuda() for t in layer)


def c(t):
    return t.cuda() if t is not None else None


def run_linear(seed, M, K, N, gs, name, bias, residual, pre):
    layer, w = ref.pack_layer(seed, N, K, gs)
    x = ref.bf(seed + 1, M, K)
    b = ref.bf(seed + 2, N) if bias else None
    r = ref.bf(seed + 3, M, N, spread=4.0) if residual else None
    po = torch.empty(M, N, dtype=torch.bfloat16, device="cuda") if pre else None
    y = w4.w4a16_linear_fused(x.cuda(), *cuda(layer), bias=c(b), residual=c(r), activation=name, group_size=gs, pre_out=po)
    w4.check_device_status()
    want, e, p, ep = ref.linear(x, w, layer, gs, b, r, name)
    ref.check(y, want, e, "y")
    if pre:
        ref.check(po, p, ep, "pre")


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300])
def test_linear_tokens(M):
    run_linear(M, M, 1024, 384, 128, "silu", True, True, True)


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("M", [3, 40, 260])
def test_linear_activations(name, M):
    run_linear(7 * M, M, 1024, 256, 128, name, False, False, True)
    run_linear(7 * M, M, 1024, 256, 128, name, True, True, False)


@pytest.mark.parametrize("K,N,gs", [(1024, 128, 1024), (2048, 128, 256), (5120, 640, 1024), (3 * 2048, 256, 2048),
                                    (14336, 128, 128), (1024, 4224, 512)])
@pytest.mark.parametrize("M", [1, 12, 50, 270])
def test_linear_sizes(K, N, gs, M):
    run_linear(K + N + M, M, K, N, gs, "none", False, True, False)


def test_linear_many_tiles():
    """More output tiles than the GPU has SMs, ragged in tokens."""
    run_linear(5, 1100, 1024, 5120, 128, "gelu_tanh", True, True, True)


def test_linear_equals_plain_product():
    """Without an epilogue the decode call gives the bits of w4a16_gemv."""
    layer, _ = ref.pack_layer(3, 512, 4096)
    d = cuda(layer)
    for M in (1, 8, 16):
        x = ref.bf(M, M, 4096).cuda()
        a, b = w4.w4a16_linear_fused(x, *d), w4.w4a16_gemv(x, *d)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17, 33, 64, 65, 128, 129, 256, 257, 300])
def test_gated_tokens(M):
    run_gated(M, M, 1024, 384, 128, "silu", M % 2 == 0)


def run_gated(seed, M, K, F, gs, name, save):
    gate, wg = ref.pack_layer(seed, F, K, gs)
    up, wu = ref.pack_layer(seed + 1, F, K, gs)
    x = ref.bf(seed + 2, M, K)
    out = w4.w4a16_gated(x.cuda(), cuda(gate), cuda(up), activation=name, group_size=gs, save=save)
    w4.check_device_status()
    h, e, g, u = ref.gated(x, wg, wu, gate, up, gs, name)
    if save:
        ref.check(out[1], *g, "g")
        ref.check(out[2], *u, "u")
        out = out[0]
    ref.check(out, h, e, "h", norm2=ref.ONE_ROUNDING)


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("M", [4, 70])
def test_gated_activations(name, M):
    run_gated(11 * M, M, 1024, 256, 128, name, True)


@pytest.mark.parametrize("K,F,gs", [(1024, 128, 1024), (4096, 256, 256), (8192, 128, 128), (1024, 2176, 128)])
@pytest.mark.parametrize("M", [1, 16, 60, 300])
def test_gated_sizes(K, F, gs, M):
    run_gated(K + F + M, M, K, F, gs, "silu", False)


def run_linear_backward(seed, M, K, N, gs, name, bias):
    layer, w = ref.pack_layer(seed, N, K, gs)
    dy = ref.bf(seed + 1, M, N)
    pre = ref.bf(seed + 2, M, N, spread=2.0) if name != "none" else None
    dx, db = w4.w4a16_linear_fused_backward(dy.cuda(), *cuda(layer), pre=c(pre), activation=name, group_size=gs,
                                            bias_grad=bias)
    w4.check_device_status()
    want, e, b, eb = ref.linear_backward(dy, pre, w, name)
    ref.check(dx, want, e, "dx", norm2=ref.ONE_ROUNDING)
    if bias:
        ref.check(db, b, eb, "dbias", norm2=2.0 ** -16)
    else:
        assert db is None


@pytest.mark.parametrize("M", [1, 2, 16, 17, 31, 64, 65, 100, 128, 129, 200, 256, 257, 300])
def test_linear_backward_tokens(M):
    run_linear_backward(M, M, 1024, 384, 128, "gelu", True)


@pytest.mark.parametrize("name", ref.ACTS)
def test_linear_backward_activations(name):
    run_linear_backward(1, 70, 1024, 256, 128, name, True)
    run_linear_backward(2, 70, 1024, 256, 128, name, False)


@pytest.mark.parametrize("K,N,gs", [(1024, 128, 1024), (2048, 128, 256), (5120, 640, 1024), (4096, 1152, 512),
                                    (1024, 5120, 128)])
@pytest.mark.parametrize("M", [3, 50, 270])
def test_linear_backward_sizes(K, N, gs, M):
    run_linear_backward(K + N + M, M, K, N, gs, "none", True)


@pytest.mark.parametrize("M,K,F,gs,name", [(1, 1024, 128, 128, "silu"), (16, 1024, 256, 256, "silu"),
                                           (33, 2048, 128, 2048, "gelu"), (130, 1024, 640, 128, "gelu_tanh"),
                                           (300, 1024, 256, 1024, "relu"), (257, 4096, 384, 128, "none")])
def test_gated_backward(M, K, F, gs, name):
    gate, wg = ref.pack_layer(M, F, K, gs)
    up, wu = ref.pack_layer(M + 1, F, K, gs)
    dh, g, u = ref.bf(1, M, F), ref.bf(2, M, F, spread=2.0), ref.bf(3, M, F, spread=2.0)
    dx = w4.w4a16_gated_backward(dh.cuda(), g.cuda(), u.cuda(), cuda(gate), cuda(up), activation=name, group_size=gs)
    w4.check_device_status()
    ref.check(dx, *ref.gated_backward(dh, g, u, wg, wu, name), "dx", norm2=ref.ONE_ROUNDING)


# ------------------------------------------------------------------ what calls may do

@pytest.mark.parametrize("M", [5, 100])
def test_residual_in_place(M):
    layer, _ = ref.pack_layer(9, 256, 1024)
    d = cuda(layer)
    x, r = ref.bf(1, M, 1024).cuda(), ref.bf(2, M, 256).cuda()
    want = w4.w4a16_linear_fused(x, *d, residual=r)
    y = r.clone()
    got = w4.w4a16_linear_fused(x, *d, residual=y, out=y)
    assert got is y and torch.equal(want.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("M", [3, 37, 261])
def test_rows_behind_the_last_stay(M):
    """Outputs are views of larger buffers: nothing behind row M - 1 is written."""
    K, N, extra = 1024, 256, 300
    layer, _ = ref.pack_layer(1, N, K)
    up, _ = ref.pack_layer(2, N, K)
    d, du = cuda(layer), cuda(up)
    x, dy = ref.bf(1, M, K).cuda(), ref.bf(2, M, N).cuda()

    def buf(cols):
        b = torch.full((M + extra, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        return b, b[:M]
    outs = []
    for run, cols in ((lambda o: w4.w4a16_linear_fused(x, *d, out=o), N),
                      (lambda o: w4.w4a16_linear_fused(x, *d, activation="silu", pre_out=o), N),
                      (lambda o: w4.w4a16_gated(x, d, du, out=o), N),
                      (lambda o: w4.w4a16_linear_fused_backward(dy, *d, out=o), K),
                      (lambda o: w4.w4a16_gated_backward(dy, dy, dy, d, du, out=o), K)):
        b, o = buf(cols)
        run(o)
        outs.append(b)
    w4.check_device_status()
    for b in outs:
        assert (b[M:] == 7.0).all() and not (b[:M] == 7.0).all()


@pytest.mark.parametrize("M", [6, 90])
def test_non_finite_rows_stay_their_own(M):
    """A NaN or an infinity in a token's row reaches that token's outputs only."""
    layer, w = ref.pack_layer(4, 256, 1024)
    up, wu = ref.pack_layer(5, 256, 1024)
    x = ref.bf(1, M, 1024)
    y0 = w4.w4a16_linear_fused(x.cuda(), *cuda(layer), activation="silu").cpu()
    h0 = w4.w4a16_gated(x.cuda(), cuda(layer), cuda(up)).cpu()
    x[2, 17] = float("nan")
    x[4, 1000] = float("inf")
    y = w4.w4a16_linear_fused(x.cuda(), *cuda(layer), activation="silu").cpu()
    h = w4.w4a16_gated(x.cuda(), cuda(layer), cuda(up)).cpu()
    keep = [m for m in range(M) if m not in (2, 4)]
    for a, b in ((y, y0), (h, h0)):
        assert torch.isnan(a[2]).all()
        assert not torch.isfinite(a[4]).all()
        assert torch.equal(a[keep].view(torch.int16), b[keep].view(torch.int16))


def chain(x, r, nw, s, gate, up, down, ws=None):
    """One feed-forward half layer: norm, gated block, down projection and residual."""
    y, h = w4.awq_rmsnorm(x, nw, residual=r, s=s)
    a = w4.w4a16_gated(y, gate, up, workspace=ws)
    return w4.w4a16_linear_fused(a, *down, residual=h, workspace=ws)


def chain_inputs(M, K, F, seed=0):
    gate, wg = ref.pack_layer(seed, F, K, scale=0.003)
    up, wu = ref.pack_layer(seed + 1, F, K, scale=0.003)
    down, wd = ref.pack_layer(seed + 2, K, F, scale=0.003)
    x, r = ref.bf(seed + 3, M, K), ref.bf(seed + 4, M, K)
    nw = (1 + 0.1 * ref.bf(seed + 5, K).float()).to(torch.bfloat16)
    s = ref.bf(seed + 6, K).float().abs() + 0.5
    return (x, r, nw, s, gate, up, down), (wg, wu, wd)


def to_cuda(v):
    return tuple(t.cuda() for t in v) if isinstance(v, tuple) else v.cuda()


@pytest.mark.parametrize("M", [1, 5, 16, 17, 140, 300])
def test_half_layer(M):
    """The three operators one after another against 64 bits (each rounding of an operand in between
    is a further independent one of 2^-8 / sqrt 3, and the output's residual only dilutes them)."""
    K, F = 1024, 2048
    inp, (wg, wu, wd) = chain_inputs(M, K, F)
    out = chain(*map(to_cuda, inp)).double().cpu()
    w4.check_device_status()
    x, r, nw, s = inp[:4]
    h, y = ref.norm(x, r, nw, s, 1e-6)
    want = (ref.act(y @ wg.t(), "silu")[0] * (y @ wu.t())) @ wd.t() + h
    assert float((out - want).norm() / want.norm()) < 2 * ref.STEP


@pytest.mark.parametrize("M", [2, 80])
def test_half_layer_backward(M):
    """The gradients of the half layer, put together from the backward calls, against autograd in 64 bits."""
    K, F = 1024, 2048
    inp, (wg, wu, wd) = chain_inputs(M, K, F, seed=20)
    x, r, nw, s, gate, up, down = map(to_cuda, inp)
    dout = ref.bf(77, M, K)
    y, h = w4.awq_rmsnorm(x, nw, residual=r, s=s)
    a, g, u = w4.w4a16_gated(y, gate, up, save=True)
    do = dout.cuda()
    da, _ = w4.w4a16_linear_fused_backward(do, *down)
    dy = w4.w4a16_gated_backward(da, g, u, gate, up)
    dx, dnw = w4.awq_rmsnorm_backward(dy, h, nw, s=s, dh=do)
    w4.check_device_status()
    hd = (inp[0].float() + inp[1].float()).to(torch.bfloat16).double().requires_grad_()
    nd = inp[2].double().requires_grad_()
    yd = hd * torch.rsqrt(hd.square().mean(1, keepdim=True) + 1e-6) * nd / inp[3].double()
    out = (torch.nn.functional.silu(yd @ wg.t()) * (yd @ wu.t())) @ wd.t() + hd
    out.backward(dout.double())
    for got, want in ((dx, hd.grad), (dnw, nd.grad)):
        # about ten roundings of 2^-8 / sqrt 3 lie between dout and dx
        assert float((got.double().cpu() - want).norm() / want.norm()) < 3 * ref.STEP


@pytest.mark.parametrize("M", [4, 150])
def test_captured_and_replayed(M):
    """Two graphs of the half layer captured one after the other and replayed at the same time on two
    streams: each owns its workspace."""
    K, F = 1024, 2048
    runs = []
    for seed in (0, 40):
        inp, _ = chain_inputs(M, K, F, seed=seed)
        args = tuple(map(to_cuda, inp))
        want = chain(*args)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = chain(*args)
        runs.append((graph, out, want, args))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (graph, out, _, _) in zip(streams, runs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    w4.check_device_status()
    for _, out, want, _ in runs:
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("M", [4, 150])
def test_two_streams_at_once(M):
    K, F = 1024, 2048
    inp, _ = chain_inputs(M, K, F)
    args = tuple(map(to_cuda, inp))
    want = chain(*args)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(chain(*args))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


def test_repeatable_and_workspace_left_clean():
    """Split sums are added in a fixed order; the counters are zero after every call."""
    K, N, M = 8192, 256, 40
    layer, _ = ref.pack_layer(2, N, K)
    up, _ = ref.pack_layer(3, N, K)
    d, du = cuda(layer), cuda(up)
    big, _ = ref.pack_layer(6, 4096, 1024)
    db = cuda(big)
    nbytes = max(w4.w4a16_fused_workspace_bytes(op, m, n, k) for op in range(4)
                 for m, n, k in ((M, N, K), (4, N, K), (M, 4096, 1024)))
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    x, x4, dy, dyb = (ref.bf(i, *s).cuda() for i, s in enumerate(((M, K), (4, K), (M, N), (M, 4096))))
    calls = [lambda: w4.w4a16_linear_fused(x, *d, workspace=ws), lambda: w4.w4a16_linear_fused(x4, *d, workspace=ws),
             lambda: w4.w4a16_gated(x, d, du, workspace=ws), lambda: w4.w4a16_gated(x4, d, du, workspace=ws),
             lambda: w4.w4a16_linear_fused_backward(dy, *d, workspace=ws)[0],
             lambda: w4.w4a16_linear_fused_backward(dyb, *db, workspace=ws)[0],
             lambda: w4.w4a16_gated_backward(dy, dy, dy, d, du, workspace=ws)]
    first = [f() for f in calls]
    for _ in range(3):
        for f, want in zip(calls, first):
            assert torch.equal(f().view(torch.int16), want.view(torch.int16))
            assert not ws[:131072].any()
    w4.check_device_status()


def test_quantized_layer_end_to_end():
    """awq_quantize's own output through the fused call, against its dequantized weights."""
    torch.manual_seed(0)
    W = torch.randn(256, 2048, device="cuda") * 0.02
    a = torch.rand(2048, device="cuda") + 0.5
    qw, sc, z, s = w4.awq_quantize(W, a, 0.5, 256)
    shifts = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device="cuda")
    q = ((qw.unsqueeze(-1).long() >> shifts) & 15).reshape(256, 8, 256).double()
    zz = ((z.unsqueeze(-1).long() >> torch.arange(0, 32, 4, device="cuda")) & 15).reshape(8, 256).t().double()
    w = ((q - zz.unsqueeze(-1)) * sc.view(torch.float16).t().double().unsqueeze(-1)).reshape(256, 2048).cpu()
    for M in (4, 200):
        x = ref.bf(M, M, 2048)
        y = w4.w4a16_linear_fused(x.cuda(), qw, sc, z, activation="gelu", group_size=256)
        want, e, _, _ = ref.linear(x, w, (qw.cpu(), sc.cpu(), z.cpu()), 256, name="gelu")
        ref.check(y, want, e, "y")
