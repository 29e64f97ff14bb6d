"""The power of two per token that the gradients before an activation are scaled by in fp16: it goes by the largest
product dy act'(pre), not by the largest dy, whose unit may be a dead one."""
import pytest
import torch

import ffn_ref as ref
import w4a16_gemm_awq_b200 as w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("M,N", [(20, 384), (40, 8192), (20, 16384), (20, 16512), (700, 17536)])
def test_largest_gradient_on_a_dead_unit(M, N, bias):
    """Every row's largest dy, 2^30 times the others, meets a derivative of zero.  RELU's derivative is exact, so the
    bound is that of the roundings to fp16, relative to the largest product."""
    layer, w = ref.pack_layer(N, N, 1024)
    dy = ref.bf(1, M, N) * 2.0 ** -30
    pre = ref.bf(2, M, N).abs()
    at = torch.randint(0, N, (M, 4), generator=torch.Generator().manual_seed(3))
    dy.scatter_(1, at, 1.5)
    pre.scatter_(1, at, -1.0)
    dx, db = w4.w4a16_linear_fused_backward(dy.cuda(), *(t.cuda() for t in layer), pre=pre.cuda(), activation="relu",
                                            bias_grad=bias)
    w4.check_device_status()
    dp = dy.double() * (pre.double() > 0)
    want, e = ref._back(dp, dp.abs().amax(1, True), torch.zeros_like(dp), w, N)
    ref.check(dx, want, e, "dx", norm2=ref.ONE_ROUNDING)
    if bias:
        ref.check(db, dp.sum(0), M * 2.0 ** -24 * dp.abs().sum(0), "dbias", norm2=2.0 ** -16)


@pytest.mark.parametrize("M,F", [(20, 384), (20, 16384), (20, 16512)])
def test_gated_largest_gradient_on_a_dead_unit(M, F):
    gate, wg = ref.pack_layer(1, F, 1024)
    up, wu = ref.pack_layer(2, F, 1024)
    dh, g, u = ref.bf(3, M, F) * 2.0 ** -30, ref.bf(4, M, F).abs(), ref.bf(5, M, F)
    at = torch.randint(0, F, (M, 4), generator=torch.Generator().manual_seed(6))
    dh.scatter_(1, at, 1.5)
    g.scatter_(1, at, -1.0)
    dx = w4.w4a16_gated_backward(dh.cuda(), g.cuda(), u.cuda(), tuple(t.cuda() for t in gate), tuple(t.cuda() for t in up),
                                 activation="relu")
    w4.check_device_status()
    on = g.double() > 0
    dg, du = dh.double() * u.double() * on, dh.double() * g.double() * on
    largest = torch.maximum(dg.abs().amax(1, True), du.abs().amax(1, True))
    zero = torch.zeros_like(dg)
    d1, e1 = ref._back(dg, largest, zero, wg, 2 * F)
    d2, e2 = ref._back(du, largest, zero, wu, 2 * F)
    ref.check(dx, d1 + d2, e1 + e2 + ref.STEP * (d1 + d2).abs(), "dx", norm2=ref.ONE_ROUNDING)
