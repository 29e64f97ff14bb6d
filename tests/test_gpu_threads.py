"""Two host threads that call the same operators at different widths, each on its own stream: what a launch sets for
its kernel must not take anything from the other thread's."""
import os
import shutil
import subprocess
import threading

import pytest
import torch

import ffn_ref as ref
import w4a16_gemm_awq_b200 as w4

pytestmark = pytest.mark.gpu


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def norm_calls(K):
    x, r, d = (ref.bf(i, 400, K).cuda() for i in range(3))
    nw = ref.bf(3, K).cuda()
    return [lambda: w4.awq_rmsnorm(x, nw, residual=r)[0], lambda: w4.awq_rmsnorm_e4m3(x, nw, residual=r)[1],
            lambda: w4.awq_rmsnorm_backward(x, r, nw, dh=d)[0]]


def layer_calls(N):
    M, K = 40, 1024
    layer, up = (tuple(t.cuda() for t in ref.pack_layer(s, N, K)[0]) for s in (1, 2))
    a, b, c = (ref.bf(i, M, N).cuda() for i in range(3))
    x = ref.bf(5, M, K).cuda()
    return [lambda: w4.w4a16_linear_fused_backward(a, *layer, pre=b, activation="gelu", bias_grad=True)[0],
            lambda: w4.w4a16_gated_backward(a, b, c, layer, up), lambda: w4.w4a16_gated(x, layer, up),
            lambda: w4.w4a16_linear_fused(x, *layer, residual=a)]


# widths whose launches are of the same kernel instances with different amounts of shared memory
@pytest.mark.parametrize("calls,widths", [(norm_calls, (8192, 4096)), (norm_calls, (16384, 14336)),
                                          (layer_calls, (8192, 5120)), (layer_calls, (14336, 2048))])
def test_two_widths(calls, widths):
    sets = [calls(n) for n in widths]
    want = [[f().clone() for f in fs] for fs in sets]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(2), []

    def work(fs, expected):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait(60)
                for _ in range(40):
                    outs = [[f() for f in fs] for _ in range(10)]
                    torch.cuda.current_stream().synchronize()
                    for turn in outs:
                        for got, w in zip(turn, expected):
                            if not torch.equal(got.view(torch.uint8), w.view(torch.uint8)):
                                raise AssertionError("an output differs from the one of a single thread")
        except BaseException as e:  # handed to the test's thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(sets, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads)
    assert not errors, errors
    w4.check_device_status()


@pytest.mark.parametrize("M", [40, 400])
def test_two_threads_on_one_stream(M):
    """The calls of two threads on the same stream, on different operands: each call is more than one launch, and the
    threads' launches may alternate."""
    N, K = 2048, 1024

    def calls(seed):
        layer, up = (tuple(t.cuda() for t in ref.pack_layer(seed + i, N, K)[0]) for i in (0, 1))
        a, b, c = (ref.bf(seed + i, M, N).cuda() for i in range(3))
        x = ref.bf(seed + 5, M, K).cuda()
        return [lambda: w4.w4a16_linear_fused_backward(a, *layer, pre=b, activation="gelu", bias_grad=True)[0],
                lambda: w4.w4a16_gated_backward(a, b, c, layer, up), lambda: w4.w4a16_gated(x, layer, up)]
    sets = [calls(10), calls(30)]
    want = [[f().clone() for f in fs] for fs in sets]
    torch.cuda.synchronize()
    stream, start, errors, outs = torch.cuda.Stream(), threading.Barrier(2), [], [[], []]

    def work(i):
        try:
            with torch.cuda.stream(stream):
                start.wait(60)
                for _ in range(200):
                    outs[i].append([f() for f in sets[i]])
        except BaseException as e:  # handed to the test's thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not errors, errors
    torch.cuda.synchronize()
    w4.check_device_status()
    for turns, expected in zip(outs, want):
        assert all(torch.equal(g.view(torch.int16), w.view(torch.int16)) for turn in turns for g, w in zip(turn, expected))


@pytest.mark.skipif(shutil.which("gcc") is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")),
                    reason="no host C compiler or no CUDA toolkit headers")
@pytest.mark.parametrize("what", ["operators", "quantize"])
def test_two_widths_from_c(tmp_path, what):
    """The same from a C program, whose threads are inside the library at the same time; and the quantizer, at two
    group sizes."""
    lib_dir = os.path.dirname(w4.build())
    out, lib64 = str(tmp_path / "two_threads"), os.path.join(CUDA, "lib64")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pthread", "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(CUDA, "include"), os.path.join(ROOT, "tests", "c_abi", "two_threads.c"),
                        "-L", lib_dir, "-lw4a16", "-L", lib64, "-lcudart", f"-Wl,-rpath,{lib_dir}", f"-Wl,-rpath,{lib64}",
                        "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([out, what], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
