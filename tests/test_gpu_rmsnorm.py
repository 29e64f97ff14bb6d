"""RMS norm with the residual's addition, its 8-bit output and its backward pass, against 64 bits.

Bounds: v is computed in fp32 from exact bf16 values: the sum of K squares by at most 32 sequential
and 10 tree adds per value, rsqrt within 2 steps, three products and a division: below 64 * 2^-24
relative, then one rounding to bf16 (2^-8) or e4m3 (2^-4 of a normal value, 2^-10 absolute below)."""
import pytest
import torch

import ffn_ref as ref
import w4a16_gemm_awq_b200 as w4

pytestmark = pytest.mark.gpu

F32 = 64 * 2.0 ** -24
SIZES = [(1, 8), (3, 16), (2, 248), (5, 256), (7, 1000), (4, 1024), (300, 1032), (1, 4096), (33, 5120), (2000, 512),
         (9, 8192), (5, 8200), (6, 14336), (2, 16384), (3, 16392), (2, 28672), (3, 32768)]


def inputs(M, K, seed=0, scale=1.0):
    x, r = ref.bf(seed, M, K, spread=scale), ref.bf(seed + 1, M, K, spread=2 * scale)
    w = (1 + 0.2 * ref.bf(seed + 2, K).float()).to(torch.bfloat16)
    s = (ref.bf(seed + 3, K).float().abs() + 0.1)
    return x, r, w, s


def c(t):
    return t.cuda() if t is not None else None


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("residual,fold", [(True, True), (False, False), (True, False)])
def test_norm(M, K, residual, fold):
    x, r, w, s = inputs(M, K)
    r, s = r if residual else None, s if fold else None
    xc = x.cuda()
    y, h = w4.awq_rmsnorm(xc, w.cuda(), residual=c(r), s=c(s), eps=1e-5)
    hw, v = ref.norm(x, r, w, s, 1e-5)
    assert torch.equal(h.double().cpu(), hw)
    assert residual or h is xc
    ref.check(y, v, (ref.STEP + 2 * F32) * v.abs(), "y")


@pytest.mark.parametrize("scale", [1e-20, 1e-6, 1e4, 1e17])
def test_norm_scales(scale):
    """Rows far from one: eps decides for small ones; sums stay in range for large ones."""
    x, r, w, s = inputs(5, 1024, scale=scale)
    y, _ = w4.awq_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), s=s.cuda(), eps=1e-6)
    _, v = ref.norm(x, r, w, s, 1e-6)
    ref.check(y, v, (ref.STEP + 2 * F32) * v.abs() + 2.0 ** -126, "y")


def test_zero_rows():
    z = torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    y, h = w4.awq_rmsnorm(z, w, residual=z)
    assert not y.any() and not h.any()
    q, sc, _ = w4.awq_rmsnorm_e4m3(z, w, group_size=128)
    assert not q.float().any() and torch.equal(sc, torch.full_like(sc, 1e-12) / 448)


@pytest.mark.parametrize("M,K,gs", [(1, 128, 128), (4, 1024, 128), (3, 1024, 0), (5, 8, 0), (2, 1000, 0), (300, 5120, 256),
                                    (7, 8192, 1024), (3, 16384, 128), (2, 32768, 0), (2, 32768, 128), (2, 14336, 2048)])
@pytest.mark.parametrize("residual,fold", [(True, False), (False, True)])
def test_e4m3(M, K, gs, residual, fold):
    x, r, w, s = inputs(M, K)
    r, s = r if residual else None, s if fold else None
    q, sc, h = w4.awq_rmsnorm_e4m3(x.cuda(), w.cuda(), residual=c(r), s=c(s), eps=1e-5, group_size=gs)
    hw, v = ref.norm(x, r, w, s, 1e-5)
    assert torch.equal(h.double().cpu(), hw)
    parts = v.reshape(M, -1, gs or K)
    scale = parts.abs().amax(2).clamp(min=1e-12) / 448
    ref.check(sc, scale, 2 * F32 * scale, "scales", norm2=2 * F32)
    t = (parts / scale.unsqueeze(2)).reshape(M, K)  # the value each code stands for, up to 448
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 below 2^-6; the fp32 error moves a value
    # by 4 F32 of itself before it is rounded
    ref.check(q.float(), t, torch.clamp(2.0 ** -4 * t.abs(), min=2.0 ** -10) + 8 * F32 * t.abs(), "q", norm2=2.0 ** -4)


def test_e4m3_non_finite():
    """A NaN or an infinity spoils the groups that its row's statistics reach, and no other row."""
    x, _, w, _ = inputs(4, 512)
    q0, s0, _ = w4.awq_rmsnorm_e4m3(x.cuda(), w.cuda(), group_size=128)
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    q, s, _ = w4.awq_rmsnorm_e4m3(x.cuda(), w.cuda(), group_size=128)
    assert torch.isnan(s[1]).all() and torch.isnan(q[1].float()).all()
    # row 2: rstd = 0, so the infinity is 0 * inf = NaN in its group and the other groups are zero
    assert torch.isnan(s[2, 1]) and torch.isnan(q[2, 128:256].float()).all()
    assert not q[2, :128].float().any()
    for m in (0, 3):
        assert torch.equal(q[m].view(torch.uint8), q0[m].view(torch.uint8)) and torch.equal(s[m], s0[m])


@pytest.mark.parametrize("M,K", SIZES + [(1500, 1024)])
@pytest.mark.parametrize("dh,fold", [(True, True), (False, False)])
def test_backward(M, K, dh, fold):
    h, dy, w, s = inputs(M, K, seed=5)
    d = ref.bf(9, M, K) if dh else None
    s = s if fold else None
    dx, dw = w4.awq_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), s=c(s), dh=c(d), eps=1e-5)
    want, dww, rstd, v = ref.norm_backward(dy, h, w, s, d, 1e-5)
    xh = h.double() * rstd
    # the two terms in brackets cancel: their fp32 errors are relative to each of them
    mag = rstd * (v.abs() + xh.abs() * (v * xh).abs().mean(1, keepdim=True))
    ref.check(dx, want, ref.STEP * want.abs() + 4 * F32 * mag, "dx")
    # per row 8 * 2^-24, summed over M rows in fp32
    terms = (dy.double() * xh / (s.double() if fold else 1.0)).abs().sum(0)
    ref.check(dw, dww, (F32 + M * 2.0 ** -24) * terms, "dweight", norm2=2.0 ** -16 + F32 * 64)
    dx2, none = w4.awq_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), s=c(s), dh=c(d), eps=1e-5, weight_grad=False)
    assert none is None and torch.equal(dx.view(torch.int16), dx2.view(torch.int16))
    dx3, dw3 = w4.awq_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), s=c(s), dh=c(d), eps=1e-5)
    assert torch.equal(dw, dw3) and torch.equal(dx.view(torch.int16), dx3.view(torch.int16))


def test_in_place_and_rows_behind():
    M, K = 37, 1024
    x, r, w, s = (t.cuda() for t in inputs(M, K))
    y, h = w4.awq_rmsnorm(x, w, residual=r, s=s)
    big = torch.cat([r, torch.full((50, K), 3.0, dtype=torch.bfloat16, device="cuda")])
    y2, h2 = w4.awq_rmsnorm(x, w, residual=big[:M], s=s, sum_out=big[:M])
    assert h2.data_ptr() == big.data_ptr() and (big[M:] == 3.0).all()
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16)) and torch.equal(y.view(torch.int16), y2.view(torch.int16))
    xi = x.clone()
    y3, h3 = w4.awq_rmsnorm(xi, w, residual=r, s=s, out=xi)  # y over x
    assert y3 is xi and torch.equal(y3.view(torch.int16), y.view(torch.int16)) and torch.equal(h3, h)
    dy, dh = ref.bf(3, M, K).cuda(), ref.bf(4, M, K).cuda()
    dx, _ = w4.awq_rmsnorm_backward(dy, h, w, s=s, dh=dh)
    g = dh.clone()
    dx2, _ = w4.awq_rmsnorm_backward(dy, h, w, s=s, dh=g, out=g)
    assert torch.equal(dx.view(torch.int16), dx2.view(torch.int16))


# more rows than two per SM, with K where the ring's depth or the threads' share changes
MANY = [(300, 8), (1000, 16), (320, 248), (700, 2056), (400, 8200), (320, 16392), (310, 28672), (310, 32768)]


@pytest.mark.parametrize("M,K", MANY)
def test_many_rows(M, K):
    x, r, w, s = inputs(M, K, seed=30)
    y, h = w4.awq_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda(), s=s.cuda(), eps=1e-5)
    hw, v = ref.norm(x, r, w, s, 1e-5)
    assert torch.equal(h.double().cpu(), hw)
    ref.check(y, v, (ref.STEP + 2 * F32) * v.abs(), "y")
    q, sc, h = w4.awq_rmsnorm_e4m3(x.cuda(), w.cuda(), residual=r.cuda(), s=s.cuda(), eps=1e-5)
    assert torch.equal(h.double().cpu(), hw)
    scale = v.abs().amax(1, True) / 448
    ref.check(sc, scale, 2 * F32 * scale, "scales", norm2=2 * F32)
    t = v / scale
    ref.check(q.float(), t, torch.clamp(2.0 ** -4 * t.abs(), min=2.0 ** -10) + 8 * F32 * t.abs(), "q", norm2=2.0 ** -4)
    d = ref.bf(9, M, K)
    dx, dw = w4.awq_rmsnorm_backward(x.cuda(), r.cuda(), w.cuda(), s=s.cuda(), dh=d.cuda(), eps=1e-5)
    want, dww, rstd, v = ref.norm_backward(x, r, w, s, d, 1e-5)
    xh = r.double() * rstd
    mag = rstd * (v.abs() + xh.abs() * (v * xh).abs().mean(1, keepdim=True))
    ref.check(dx, want, ref.STEP * want.abs() + 4 * F32 * mag, "dx")
    terms = (x.double() * xh / s.double()).abs().sum(0)
    ref.check(dw, dww, (F32 + M * 2.0 ** -24) * terms, "dweight", norm2=2.0 ** -16 + F32 * 64)
    w4.check_device_status()


def test_non_finite_rows_in_the_backward_pass():
    """A NaN in a row's gradient spoils that row and, through the sum over rows, dweight; no other row."""
    h, dy, w, _ = inputs(400, 1024, seed=3)
    dx0, _ = w4.awq_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda())
    dy[5, 3] = float("nan")
    h[7, 9] = float("inf")
    dx, dw = w4.awq_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda())
    assert torch.isnan(dx[5]).all() and torch.isnan(dw[3])
    keep = [m for m in range(400) if m not in (5, 7)]
    assert torch.equal(dx[keep].view(torch.int16), dx0[keep].view(torch.int16))
