"""Calls of the feed-forward products one after another on different operands and weights, with nothing waited
for in between: what a call leaves in shared memory, tensor memory and the workspace is wrong for the next one, so
a stage, an accumulator or a partial tile that is used before it is written shows.  Every output is compared in
full: each set's first one with 64 bits, all later ones with the first, to the bit (every sum has a fixed order)."""
import pytest
import torch

import ffn_ref as ref
import w4a16_gemm_awq_b200 as w4

pytestmark = pytest.mark.gpu


def gpu(t):
    return tuple(v.cuda() for v in t) if isinstance(t, tuple) else t.cuda()


def host(*ts):
    return tuple(t.cpu() for t in ts)


def make(op, seed, M, K, N, gs=128):
    """(call, check of its output) of one product on operands of its own; N is F for the gated ones."""
    layer, w = ref.pack_layer(seed, N, K, gs)
    d, wd = gpu(layer), w.cuda()
    if op == "linear":
        x, r = ref.bf(seed + 1, M, K).cuda(), ref.bf(seed + 2, M, N).cuda()
        y, e, _, _ = ref.linear(x, wd, d, gs, residual=r, name="silu")
        return (lambda: w4.w4a16_linear_fused(x, *d, residual=r, activation="silu", group_size=gs),
                lambda got: ref.check(got, *host(y, e), "y"))
    if op == "linear backward":
        dy, pre = ref.bf(seed + 1, M, N).cuda(), ref.bf(seed + 2, M, N, spread=2.0).cuda()
        dx, e, b, eb = ref.linear_backward(dy, pre, wd, "gelu")

        def check(got):
            ref.check(got[0], *host(dx, e), "dx", norm2=ref.ONE_ROUNDING)
            ref.check(got[1], *host(b, eb), "dbias", norm2=2.0 ** -16)
        return (lambda: w4.w4a16_linear_fused_backward(dy, *d, pre=pre, activation="gelu", group_size=gs, bias_grad=True),
                check)
    up, wu = ref.pack_layer(seed + 3, N, K, gs)
    du, wud = gpu(up), wu.cuda()
    if op == "gated":
        x = ref.bf(seed + 1, M, K).cuda()
        h, e, g, u = ref.gated(x, wd, wud, d, du, gs, "silu")

        def check(got):
            ref.check(got[0], *host(h, e), "h", norm2=ref.ONE_ROUNDING)
            ref.check(got[1], *host(*g), "g")
            ref.check(got[2], *host(*u), "u")
        return lambda: w4.w4a16_gated(x, d, du, group_size=gs, save=True), check
    dh, g, u = ref.bf(seed + 1, M, N).cuda(), ref.bf(seed + 2, M, N, spread=2.0).cuda(), ref.bf(seed + 4, M, N, spread=2.0).cuda()
    dx, e = ref.gated_backward(dh, g, u, wd, wud, "silu")
    return (lambda: w4.w4a16_gated_backward(dh, g, u, d, du, group_size=gs),
            lambda got: ref.check(got, *host(dx, e), "dx", norm2=ref.ONE_ROUNDING))


def flat(out):
    return [t.view(torch.int32 if t.dtype == torch.float32 else torch.int16) for t in (out if isinstance(out, tuple) else (out,))]


def alternate(calls, rounds, batch=10):
    """calls: (call, check) pairs, called in turn."""
    first = []
    for call, check in calls:
        out = call()
        check(out)
        first.append(flat(out))
    torch.cuda.synchronize()
    wrong = 0
    for _ in range(0, rounds, batch):
        outs = [[flat(call()) for call, _ in calls] for _ in range(batch)]
        for turn in outs:
            wrong += sum(not torch.equal(a, b) for got, want in zip(turn, first) for a, b in zip(got, want))
        del outs
    w4.check_device_status()
    assert wrong == 0, f"{wrong} outputs differ from their set's first one"


# tokens, K, N: tiles of 256 channels x 256 tokens (or all of fewer) on 74 pairs of CTAs
SHAPES = {
    "linear": [(700, 1024, 18944), (1100, 1024, 14336), (64, 1024, 57344), (1000, 14336, 4096), (300, 4096, 4096),
               (77, 8192, 8192), (3000, 5120, 5120)],
    "linear backward": [(9472, 2048, 512), (1100, 14336, 512), (64, 57344, 512), (1023, 5120, 5120), (640, 5120, 4096),
                        (90, 5120, 7168), (3000, 5120, 5120), (33, 1024, 8192)],
    "gated": [(700, 1024, 9472), (1100, 1024, 7168), (64, 1024, 28672), (1000, 8192, 2048), (300, 4096, 2048), (1500, 4096, 5120)],
    "gated backward": [(9472, 2048, 512), (1100, 14336, 512), (64, 57344, 256), (1023, 5120, 2560), (700, 4096, 7168),
                       (90, 4096, 7168), (3000, 5120, 2560)],
}


@pytest.mark.parametrize("op,M,K,N", [(op, *s) for op, shapes in SHAPES.items() for s in shapes])
def test_two_sets(op, M, K, N):
    """One product on two sets: three and more tiles per pair and fewer than one, long and short contractions, whole
    tiles, cut ones, and cut ones that are joined by halves."""
    alternate([make(op, seed, M, K, N) for seed in (10, 50)], 100)


@pytest.mark.parametrize("M", [40, 200, 1023])
def test_products_in_turn(M):
    """All four products in turn, each on two sets and two group sizes."""
    calls = [make(op, seed, M, 4096, 2048, gs) for seed, gs in ((10, 128), (50, 1024)) for op in SHAPES]
    alternate(calls, 100)


@pytest.mark.parametrize("M", [100, 1023])
def test_two_sizes_in_turn(M):
    """A wide and a narrow tile, few and many tiles, with the workspace and the counters between them."""
    calls = [make("linear backward", 10, M, 5120, 5120), make("linear backward", 20, 33, 1024, 8192),
             make("gated backward", 30, M, 2048, 1024), make("linear", 40, 20, 14336, 384), make("linear", 60, 5, 4096, 4096),
             make("gated", 70, M, 2048, 640)]
    alternate(calls, 100)
