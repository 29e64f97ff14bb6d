"""The feed-forward operators without a GPU: refusals at the C boundary and in the binding, and the
64-bit reference's gradients against differences."""
import ctypes

import pytest
import torch

import ffn_ref as ref
import w4a16_gemm_awq_b200 as w4

FAKE = 1 << 20  # an aligned address that is never dereferenced: validation fails first
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    w4.build()
    return w4.lib()


def W(qw=FAKE, sc=FAKE, z=FAKE):
    return w4.Weights(qw, sc, z)


def linear(L, x=FAKE, w="W", bias=None, res=None, y=FAKE, pre=None, M=1, N=128, K=1024, gs=128, act=0, ws=FAKE, wsb=BIG):
    return L.w4a16_linear_fused(x, W() if w == "W" else w, bias, res, y, pre, M, N, K, gs, act, ws, wsb, None)


def linear_b(L, dy=FAKE, pre=FAKE, w="W", dx=FAKE, db=None, M=1, N=128, K=1024, gs=128, act=2, ws=FAKE, wsb=BIG):
    return L.w4a16_linear_fused_backward(dy, pre, W() if w == "W" else w, dx, db, M, N, K, gs, act, ws, wsb, None)


def gated(L, x=FAKE, w="W", up="W", h=FAKE, g=None, u=None, M=1, N=128, K=1024, gs=128, act=2, ws=FAKE, wsb=BIG):
    return L.w4a16_gated(x, W() if w == "W" else w, W() if up == "W" else up, h, g, u, M, N, K, gs, act, ws, wsb, None)


def gated_b(L, dh=FAKE, g=FAKE, u=FAKE, w="W", up="W", dx=FAKE, M=1, N=128, K=1024, gs=128, act=2, ws=FAKE, wsb=BIG):
    return L.w4a16_gated_backward(dh, g, u, W() if w == "W" else w, W() if up == "W" else up, dx, M, N, K, gs, act, ws,
                                  wsb, None)


@pytest.mark.parametrize("f", [linear, linear_b, gated, gated_b])
def test_product_refusals(L, f):
    for M, N, K in ((0, 128, 1024), (-1, 128, 1024), ((1 << 24) + 1, 128, 1024), (1, 0, 1024), (1, 64, 1024), (1, 130, 1024),
                    (1, 1 << 23, 1024), (1, 128, 0), (1, 128, 512), (1, 128, 1100), (1, 128, 1 << 21)):
        assert f(L, M=M, N=N, K=K) == w4.ERR_SHAPE, (M, N, K)
    for gs in (0, -128, 64, 192, 384, 2048):
        assert f(L, gs=gs) == w4.ERR_SHAPE, gs
    for act in (-1, 5, 100):
        assert f(L, act=act) == w4.ERR_VALUE
    assert f(L, w=None) == w4.ERR_NULL
    for bad in (W(qw=0), W(sc=0), W(z=0)):
        assert f(L, w=bad) == w4.ERR_NULL
    for bad in (W(qw=FAKE + 8), W(sc=FAKE + 2), W(z=FAKE + 4)):
        assert f(L, w=bad) == w4.ERR_ALIGN
    assert f(L, ws=None) == w4.ERR_NULL
    assert f(L, ws=FAKE + 8) == w4.ERR_ALIGN


@pytest.mark.parametrize("f,required,optional", [
    (linear, ("x", "y"), ("bias", "res", "pre")), (linear_b, ("dy", "pre", "dx"), ("db",)),
    (gated, ("x", "h"), ()), (gated_b, ("dh", "g", "u", "dx"), ())])
def test_product_pointers(L, f, required, optional):
    for name in required:
        assert f(L, **{name: None}) == w4.ERR_NULL, name
        assert f(L, **{name: FAKE + 8}) == w4.ERR_ALIGN, name
    for name in optional:
        assert f(L, **{name: FAKE + 8}) == w4.ERR_ALIGN, name


def test_gated_pairs(L):
    assert gated(L, g=FAKE) == w4.ERR_NULL and gated(L, u=FAKE) == w4.ERR_NULL
    assert gated(L, g=FAKE, u=FAKE + 2) == w4.ERR_ALIGN
    for f in (gated, gated_b):
        assert f(L, up=None) == w4.ERR_NULL
        assert f(L, up=W(sc=FAKE + 2)) == w4.ERR_ALIGN
        assert f(L, N=1 << 22) == w4.ERR_SHAPE  # 2 F rows pass the largest N


def test_norm_refusals(L):
    def fwd(x=FAKE, r=None, w=FAKE, s=None, eps=1e-6, h=None, y=FAKE, M=1, K=1024):
        return L.awq_rmsnorm(x, r, w, s, eps, h, y, M, K, None)

    def q8(x=FAKE, r=None, w=FAKE, s=None, eps=1e-6, h=None, y=FAKE, sc=FAKE, M=1, K=1024, gs=128):
        return L.awq_rmsnorm_e4m3(x, r, w, s, eps, h, y, sc, M, K, gs, None)

    def bwd(x=FAKE, r=None, w=FAKE, s=None, eps=1e-6, h=FAKE, y=FAKE, dw=FAKE, M=1, K=1024, ws=FAKE, wsb=BIG):
        return L.awq_rmsnorm_backward(x, h, w, s, r, eps, y, dw, M, K, ws, wsb, None)
    for f in (fwd, q8, bwd):
        for M, K in ((0, 1024), (-3, 1024), ((1 << 24) + 1, 1024), (1, 0), (1, 4), (1, 1004), (1, 32776)):
            assert f(M=M, K=K) == w4.ERR_SHAPE, (M, K)
        for eps in (-1e-6, float("nan"), float("inf")):
            assert f(eps=eps) == w4.ERR_VALUE
        for name in ("x", "w", "y"):
            assert f(**{name: None}) == w4.ERR_NULL
            assert f(**{name: FAKE + 8}) == w4.ERR_ALIGN
        for name in ("r", "s", "h"):
            assert f(**{name: FAKE + 4}) == w4.ERR_ALIGN
    assert q8(sc=None) == w4.ERR_NULL and q8(sc=FAKE + 4) == w4.ERR_ALIGN
    for gs in (0, 64, 192, 384, 2048, -128):
        assert q8(gs=gs) == w4.ERR_SHAPE, gs
    assert q8(K=1000, gs=128) == w4.ERR_SHAPE
    assert bwd(h=None) == w4.ERR_NULL and bwd(ws=None) == w4.ERR_NULL and bwd(ws=FAKE + 4) == w4.ERR_ALIGN
    assert bwd(dw=FAKE + 4) == w4.ERR_ALIGN


def test_workspace_query(L):
    for op in range(-1, 6):
        assert w4.w4a16_fused_workspace_bytes(op, 0, 128, 1024) == 0
        assert w4.w4a16_fused_workspace_bytes(op, 4, 100, 1000) == 0 or not torch.cuda.is_available()


def test_binding_refuses_before_the_library():
    x = torch.zeros(2, 1024, dtype=torch.bfloat16)
    layer = (torch.zeros(128, 128, dtype=torch.int32), torch.zeros(8, 128, dtype=torch.int16),
             torch.zeros(8, 16, dtype=torch.int32))
    y, w = torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(1024, dtype=torch.bfloat16)
    for f in (lambda: w4.w4a16_linear_fused(x, *layer), lambda: w4.w4a16_gated(x, layer, layer),
              lambda: w4.w4a16_linear_fused_backward(y, *layer), lambda: w4.w4a16_gated_backward(y, y, y, layer, layer),
              lambda: w4.awq_rmsnorm(x, w), lambda: w4.awq_rmsnorm_e4m3(x, w), lambda: w4.awq_rmsnorm_backward(x, x, w)):
        with pytest.raises(ValueError):  # CPU tensors never reach the library
            f()
    with pytest.raises(ValueError):
        w4._activation("swish")
    assert [w4._activation(a) for a in ref.ACTS] == list(range(5))


# ------------------------------------------------------------------ the reference itself

def test_packed_layer_matches_the_oracle(orc):
    """The hand-packed test layer read back by the oracle's own dequantization."""
    layer, w = ref.pack_layer(1, 128, 1024, 128)
    x = torch.eye(1024)[:64].to(torch.bfloat16)
    bits = x.view(torch.int16).numpy().view("uint16")
    got = orc.linear(bits, layer[0].numpy().view("uint32"), layer[1].numpy().view("uint16"),
                     layer[2].numpy().view("uint32"), 128)
    got = got[0] if isinstance(got, tuple) else got
    assert torch.allclose(torch.as_tensor(got).double(), w.t()[:64], rtol=0, atol=0)


@pytest.mark.parametrize("name", ref.ACTS)
def test_reference_gradients_against_differences(name):
    """The formulas of the backward passes against central differences in 64 bits (error of a
    difference with step d: d^2 / 6 |f'''| + 2^-52 / d |f|, below 1e-8 here)."""
    torch.manual_seed(3)
    d = 1e-5
    wg, wu = torch.randn(6, 5).double(), torch.randn(6, 5).double()
    x, dh = torch.randn(3, 5).double() + 0.05, torch.randn(3, 6).double()

    def loss(x):
        return (ref.act(x @ wg.t(), name)[0] * (x @ wu.t()) * dh).sum()

    def numeric(f, t):
        g = torch.zeros_like(t)
        for i in range(t.numel()):
            a, b = t.clone(), t.clone()
            a.view(-1)[i] += d
            b.view(-1)[i] -= d
            g.view(-1)[i] = (f(a) - f(b)) / (2 * d)
        return g
    g, u = x @ wg.t(), x @ wu.t()
    dx, _ = ref.gated_backward(dh, g, u, wg, wu, name)
    assert torch.allclose(dx, numeric(loss, x), rtol=1e-6, atol=1e-7)
    p = x @ wg.t()
    dx, _, db, _ = ref.linear_backward(dh, p, wg, name)
    assert torch.allclose(dx, numeric(lambda t: (ref.act(t @ wg.t(), name)[0] * dh).sum(), x), rtol=1e-6, atol=1e-7)
    b = torch.zeros(6).double()
    assert torch.allclose(db, numeric(lambda t: (ref.act(p + t, name)[0] * dh).sum(), b), rtol=1e-6, atol=1e-7)


def test_norm_reference_gradients_against_differences():
    torch.manual_seed(4)
    h, dy, dh = (torch.randn(3, 7).double() for _ in range(3))
    w, s = torch.randn(7).double(), torch.rand(7).double() + 0.5

    def loss(h, w):
        return (h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-5) * w / s * dy).sum() + (h * dh).sum()
    dx, dw, _, _ = ref.norm_backward(dy, h, w, s, dh, 1e-5)
    d = 1e-5
    for t, got, f in ((h, dx, lambda t: loss(t, w)), (w, dw, lambda t: loss(h, t))):
        for i in range(t.numel()):
            a, b = t.clone(), t.clone()
            a.view(-1)[i] += d
            b.view(-1)[i] -= d
            assert abs(float((f(a) - f(b)) / (2 * d)) - float(got.view(-1)[i])) < 1e-7
