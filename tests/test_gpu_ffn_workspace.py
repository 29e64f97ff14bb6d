"""The workspace query of the feed-forward operators: zero for what the calls refuse, and only for that."""
import pytest

import w4a16_gemm_awq_b200 as w4

pytestmark = pytest.mark.gpu

OPS = (w4.OP_LINEAR, w4.OP_LINEAR_BACKWARD, w4.OP_GATED, w4.OP_GATED_BACKWARD)
COUNTERS = (1 << 22) // 128 * 4


@pytest.mark.parametrize("op", OPS)
def test_products(op):
    gated = op in (w4.OP_GATED, w4.OP_GATED_BACKWARD)
    for M, N, K in ((0, 128, 1024), (-1, 128, 1024), ((1 << 24) + 1, 128, 1024), (4, 0, 1024), (4, 100, 1024), (4, 128, 0),
                    (4, 128, 1000), (4, 128, 512), (4, 128, 1 << 21), (4, (1 << 22) + 128, 1024)):
        assert w4.w4a16_fused_workspace_bytes(op, M, N, K) == 0, (M, N, K)
    for M, N, K in ((1, 128, 1024), (16, 384, 14336), (17, 128, 1024), (300, 5120, 5120), (1 << 24, 128, 1024), (20, 1 << 21, 1024)):
        assert w4.w4a16_fused_workspace_bytes(op, M, N, K) >= COUNTERS, (M, N, K)
    # two matrices of F rows: 2 F is at most the largest N
    for F in ((1 << 21) + 128, 1 << 22):
        assert (w4.w4a16_fused_workspace_bytes(op, 20, F, 1024) == 0) == gated, F


def test_norm_backward():
    op = w4.OP_RMSNORM_BACKWARD
    for M, K in ((0, 1024), ((1 << 24) + 1, 1024), (4, 0), (4, 4), (4, 1004), (4, 32776)):
        assert w4.w4a16_fused_workspace_bytes(op, M, 128, K) == 0, (M, K)
    for M, K in ((1, 8), (4, 1000), (5000, 32768), (1 << 24, 1024)):
        for N in (0, -5, 128):  # ignored
            assert w4.w4a16_fused_workspace_bytes(op, M, N, K) > COUNTERS, (M, K, N)


def test_unknown_operators():
    assert all(w4.w4a16_fused_workspace_bytes(op, 4, 128, 1024) == 0 for op in (-1, 5, 100))
