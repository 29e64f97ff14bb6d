"""Decode calls one after another on two sets of operands and weights, with nothing waited for in between: a ring
slot that is refilled before its codes were read, or read before they came, shows as an output of the wrong weights.
Each set's first output is compared with 64 bits, all later ones with the first, to the bit."""
import pytest
import torch

import ffn_ref as ref
import w4a16_gemm_awq_b200 as w4
from test_gpu_ffn_alternate import alternate, gpu, make

pytestmark = pytest.mark.gpu


def plain(seed, M, K, N, schedule):
    layer, w = ref.pack_layer(seed, N, K)
    d = gpu(layer)
    x = ref.bf(seed + 1, M, K).cuda()
    p, e = ref.projection(x, w.cuda(), d, 128)
    bound = (e + ref.STEP * (p.abs() + e)).cpu()
    return (lambda: w4.w4a16_gemv_ex(x, *d, schedule=schedule)), (lambda got: ref.check(got, p.cpu(), bound, "y"))


@pytest.mark.parametrize("schedule", [w4.GEMV_STREAM_K, w4.GEMV_CLUSTER])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 4096), (4, 14336, 4096), (8, 4096, 28672), (9, 4096, 6144), (16, 14336, 4096)])
def test_plain(schedule, M, K, N):
    alternate([plain(seed, M, K, N, schedule) for seed in (10, 50)], 400, batch=50)


@pytest.mark.parametrize("op,M,K,N", [("linear", 1, 4096, 4096), ("linear", 4, 14336, 4096), ("linear", 16, 8192, 8192),
                                      ("gated", 1, 4096, 14336), ("gated", 7, 8192, 2048), ("gated", 16, 4096, 14336)])
def test_epilogues(op, M, K, N):
    alternate([make(op, seed, M, K, N) for seed in (10, 50)], 400, batch=50)


@pytest.mark.parametrize("M", [2, 16])
def test_three_bits(M):
    """The 3-bit form against its own first outputs, each waited for."""
    K, N = 4096, 6144
    torch.manual_seed(M)
    calls = []
    for _ in range(2):
        W, a = torch.randn(N, K, device="cuda") * 0.02, torch.rand(K, device="cuda") + 0.5
        q = w4.awq_quantize3(W, a, 0.5)
        x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
        calls.append(((lambda x=x, q=q: w4.w3a16_gemv(x, *q[:3])), lambda got: torch.cuda.synchronize()))
    alternate(calls, 400, batch=50)


def test_mixed():
    """Plain, linear and gated calls of several sizes in turn, through one workspace."""
    calls = [plain(10, 1, 4096, 4096, w4.GEMV_AUTO), make("gated", 20, 1, 4096, 14336), make("linear", 30, 1, 14336, 4096),
             plain(40, 12, 4096, 6144, w4.GEMV_AUTO), make("linear", 50, 12, 4096, 4096), make("gated", 60, 12, 4096, 2048)]
    alternate(calls, 200, batch=20)
