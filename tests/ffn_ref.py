"""64-bit reference of the feed-forward operators, and the error bounds of their kernels.

Bounds (every rounding to bf16 is off by at most 2^-8 of the value, to fp16 by 2^-11):
  projection, M <= 16  the decode GEMV's bound of parity.py (exact weights, fp32 sums);
  projection, M > 16   linear: 2^-8 sum |x w| (each weight rounded once to bf16); gated: 2^-11 sum |x w|
                       (weights rounded to fp16) and 2^-38 max |x| sum |w| (x over a power of two that
                       takes its row's maximum to 2^14 or more: an fp16 subnormal is off by 2^-25); both
                       + fp32 sums, whose chain is K / 16 adds in the tensor core and at most 64 outside,
                       2^-22 each;
  activations          |act'| <= 1.13 for every activation here (GELU's maximum is 1.129), and the
                       fast exponential and division are below 2^-18 |p| absolute;
  backward product     dp and the weight rounded to fp16, as above: 2 * 2^-11 + 2^-16 relative, 2^-37 of
                       the row's maximum, plus the error of act' (below 2^-18 (1 + |p|) of dy) on each term.
Such worst cases add up all signs alike, so the whole output is also held to a relative 2-norm: the
output's own rounding to bf16 is uniform with a root mean square of at most 2^-8 / sqrt 3; a second one of
that size (linear's weights) makes it sqrt(2 / 3) 2^-8 < 2^-8, two to fp16 beside it less than 0.6 * 2^-8.
"""
from __future__ import annotations

import numpy as np
import torch

from parity import GEMV_XS_COEF

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
LIPSCHITZ = 1.13
STEP = 2.0 ** -8
HALF_STEP = 2.0 ** -11
ONE_ROUNDING = 0.6 * STEP
FAST = 2.0 ** -18
TINY = 1e-30


def pack_layer(seed: int, N: int, K: int, gs: int = 128, scale: float = 0.006):
    """A random packed layer on the CPU: (qweight, scales, zeros) tensors and the fp64 weights.
    Codes and zero points cover 0..15; every nibble order step is done by hand."""
    r = np.random.default_rng(seed)
    q = r.integers(0, 16, (N, K), dtype=np.uint32)
    z = r.integers(0, 16, (K // gs, N), dtype=np.uint32)
    sc = (scale * np.exp(0.5 * r.standard_normal((K // gs, N)))).astype(np.float16)
    order = (0, 2, 4, 6, 1, 3, 5, 7)
    qw = np.zeros((N, K // 8), np.uint32)
    for j in range(8):
        qw |= q[:, order[j]::8] << np.uint32(4 * j)
    zw = np.zeros((K // gs, N // 8), np.uint32)
    for j in range(8):
        zw |= z[:, j::8] << np.uint32(4 * j)
    w = (q.astype(np.float64) - np.repeat(z.T, gs, 1)) * np.repeat(sc.astype(np.float64).T, gs, 1)
    return (torch.from_numpy(qw.view(np.int32)), torch.from_numpy(sc.view(np.int16)),
            torch.from_numpy(zw.view(np.int32))), torch.from_numpy(w)


def act(p, name):
    """(act(p), act'(p)) in fp64."""
    if name == "none":
        return p, torch.ones_like(p)
    if name == "relu":
        return torch.where(p > 0, p, torch.zeros_like(p)), (p > 0).to(p.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-p))
        return p * s, s * (1 + p * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(p / 2 ** 0.5))
        return p * c, c + p * torch.exp(-p * p / 2) / (2 * np.pi) ** 0.5
    a = (2 / np.pi) ** 0.5
    t = torch.tanh(a * (p + 0.044715 * p ** 3))
    return 0.5 * p * (1 + t), 0.5 * (1 + t) + 0.5 * p * (1 - t * t) * a * (1 + 3 * 0.044715 * p * p)


def bf(seed, *shape, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * spread).to(torch.bfloat16)


def projection(x, w, layer, gs, half=False):
    """(x W^T, its error bound before any output rounding) in fp64; x bf16."""
    x = x.double()
    p, mag = x @ w.t(), x.abs() @ w.abs().t()
    M, K = x.shape
    if M <= 16:
        sc = layer[1].view(torch.float16).double()  # [G][N]
        xs = x.abs().reshape(M, K // gs, gs).sum(-1) @ sc
        return p, GEMV_XS_COEF * xs + (K // 128 + 64) * 2.0 ** -22 * mag
    sums = (K // 16 + 64) * 2.0 ** -22
    if half:
        return p, (HALF_STEP + sums) * mag + 2.0 ** -38 * x.abs().amax(1, True) * w.abs().sum(1)
    return p, (STEP + sums) * mag


def linear(x, w, layer, gs, bias=None, residual=None, name="none"):
    """(y, bound of y, p, bound of p)."""
    p, e = projection(x, w, layer, gs)
    if bias is not None:
        p = p + bias.double()
    y, _ = act(p, name)
    if residual is not None:
        y = y + residual.double()
    ey = LIPSCHITZ * e + FAST * p.abs() + STEP * (y.abs() + LIPSCHITZ * e)
    return y, ey, p, e + STEP * (p.abs() + e) + 2.0 ** -22 * p.abs()


def gated(x, wg, wu, gate, up, gs, name):
    """(h, bound of h, (g, bound), (u, bound))."""
    g, eg = projection(x, wg, gate, gs, half=True)
    u, eu = projection(x, wu, up, gs, half=True)
    a, _ = act(g, name)
    ea = LIPSCHITZ * eg + FAST * g.abs()
    h = a * u
    e = ea * u.abs() + a.abs() * eu + ea * eu
    return h, e + STEP * (h.abs() + e), (g, eg + STEP * (g.abs() + eg)), (u, eu + STEP * (u.abs() + eu))


def _back(dp, largest, slack, w, depth):
    """dp W and its bound; largest: the rows' largest |dp|, over all the products that share its scale."""
    dx = dp @ w
    mag = dp.abs() @ w.abs()
    e = (2 * HALF_STEP + 2.0 ** -16 + (depth // 16 + 64) * 2.0 ** -22) * mag + slack @ w.abs()
    return dx, e + 2.0 ** -37 * largest * w.abs().sum(0) + STEP * (dx.abs() + e)


def linear_backward(dy, pre, w, name):
    """(dx, bound, dbias, bound)."""
    dy = dy.double()
    p = pre.double() if pre is not None else torch.zeros_like(dy)
    da = act(p, name)[1] if name != "none" else torch.ones_like(dy)
    slack = FAST * dy.abs() * (1 + p.abs()) if name != "none" else torch.zeros_like(dy)
    dp = dy * da
    dx, e = _back(dp, dy.abs().amax(1, True), slack, w, w.shape[0])
    M = dy.shape[0]
    return dx, e, dp.sum(0), slack.sum(0) + M * 2.0 ** -24 * dp.abs().sum(0)


def gated_backward(dh, g, u, wg, wu, name):
    dh, g, u = dh.double(), g.double(), u.double()
    a, da = act(g, name)
    k = FAST * dh.abs() * (1 + g.abs())
    dg, du = dh * u * da, dh * a
    largest = torch.maximum(dg.abs().amax(1, True), du.abs().amax(1, True))
    d1, e1 = _back(dg, largest, k * u.abs(), wg, 2 * wg.shape[0])
    d2, e2 = _back(du, largest, k, wu, 2 * wu.shape[0])
    return d1 + d2, e1 + e2 + STEP * (d1 + d2).abs()


def norm(x, residual, weight, s, eps):
    """(h as bf16 values, v) in fp64."""
    h = x.double()
    if residual is not None:
        h = (x.float() + residual.float()).to(torch.bfloat16).double()
    v = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * weight.double()
    return h, v if s is None else v / s.double()


def norm_backward(dy, h, weight, s, dh, eps):
    h, v = h.double(), dy.double()
    rstd = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    if s is not None:
        v = v / s.double()
    dw = (v * h * rstd).sum(0)
    v = v * weight.double()
    xh = h * rstd
    dx = rstd * (v - xh * (v * xh).mean(1, keepdim=True))
    return (dx if dh is None else dx + dh.double()), dw, rstd, v


def check(got, want, bound, what, norm2=STEP):
    """Every value within its bound, and all of them within norm2 in the 2-norm."""
    got = got.double().cpu()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    d = (got - want).abs()
    bad = d > bound + TINY
    assert not bad.any(), f"{what}: {int(bad.sum())} values beyond the bound, worst {float((d / (bound + TINY)).max()):.3g} times it"
    rel = float((got - want).norm() / want.norm().clamp(min=TINY))
    assert rel <= norm2, f"{what}: relative 2-norm {rel:.3g} > {norm2:.3g}"
