"""Cases of the feed-forward operators around the W4A16 product: RMS norm with the residual's addition
(bf16 output with the 1/s fold, or e4m3 with scales) and its backward pass; the W4A16 linear layer with
bias, activation and residual in its epilogue and its backward pass; the gated feed-forward block (gate and
up projections, activation and product) and its backward pass.

`own` false: the operators in plain torch operations, in 32 bits, rounded once at the end.  `own` true: the
calls of w4a16_gemm_awq_b200.  Weights are packed as include/w4a16.h documents them.
"""
import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
TINY = 1e-12  # the least row maximum that a scale is made from
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one token through the norm before a 4096-wide layer: launch latency
        {"name": "norm one token", "op": "norm", "M": 1, "K": 4096, "fold": True, "residual": True},
        # a long prompt through the norm of an 8192-wide model
        {"name": "norm prompt", "op": "norm", "M": 8192, "K": 8192, "fold": True, "residual": True},
        # an odd batch of prompts, 8-bit output with a scale per 128 channels
        {"name": "norm e4m3 ragged", "op": "norm8", "M": 1999, "K": 5120, "group": 128, "fold": False, "residual": True},
        # a training step's gradient of the norm
        {"name": "norm backward", "op": "norm_bwd", "M": 4096, "K": 4096, "fold": True, "residual": True},
        # down projection of one decode step, residual added
        {"name": "linear decode", "op": "linear", "M": 4, "K": 14336, "N": 4096, "group": 128, "act": "none",
         "bias": False, "residual": True},
        # a batch between decode and prefill through a biased layer
        {"name": "linear batch gelu", "op": "linear", "M": 77, "K": 8192, "N": 8192, "group": 128, "act": "gelu_tanh",
         "bias": True, "residual": False},
        # down projection of a prompt, residual added
        {"name": "linear prompt", "op": "linear", "M": 2048, "K": 14336, "N": 4096, "group": 128, "act": "none",
         "bias": False, "residual": True},
        # gradient through a biased, activated layer with frozen weights, odd token count
        {"name": "linear backward", "op": "linear_bwd", "M": 1023, "K": 5120, "N": 5120, "group": 128, "act": "gelu",
         "bias": True},
        # gate and up projections of one decode step
        {"name": "gated one token", "op": "gated", "M": 1, "K": 4096, "F": 14336, "group": 128, "act": "silu", "save": False},
        # a decode batch of a large model
        {"name": "gated decode batch", "op": "gated", "M": 16, "K": 8192, "F": 28672, "group": 128, "act": "silu",
         "save": False},
        # gate and up projections of a long prompt
        {"name": "gated prompt", "op": "gated", "M": 4096, "K": 4096, "F": 14336, "group": 128, "act": "silu", "save": False},
        # gradient of the gated block in a training step
        {"name": "gated backward", "op": "gated_bwd", "M": 2048, "K": 4096, "F": 14336, "group": 128, "act": "silu"},
    ]


def _log(rng, lo, hi):
    """An integer between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("norm", "norm8", "norm_bwd", "linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd"))
    if op.startswith("norm"):
        K = 8 * _log(rng, 128, 1024)
        c = {"op": op, "M": _log(rng, 1, 8192), "K": K, "fold": rng.random() < 0.5, "residual": rng.random() < 0.7}
        if op == "norm8":
            c["K"] = 128 * max(1, K // 128)
            c["group"] = rng.choice((0, 128))
        return c
    K = 1024 * _log(rng, 1, 14)
    group = rng.choice((128, 128, 256, 1024))
    if op.startswith("linear"):
        c = {"op": op, "M": _log(rng, 1 if op == "linear" else 16, 4096), "K": K, "N": 128 * _log(rng, 4, 64),
             "group": group, "act": rng.choice(ACTS), "bias": rng.random() < 0.5}
        if op == "linear":
            c["residual"] = rng.random() < 0.5
        return c
    c = {"op": op, "M": _log(rng, 1 if op == "gated" else 16, 4096), "K": 1024 * _log(rng, 1, 4), "F": 128 * _log(rng, 4, 112),
         "group": group, "act": rng.choice(("silu", "gelu", "gelu_tanh", "relu"))}
    if op == "gated":
        c["save"] = rng.random() < 0.3
    return c


# ---------------------------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _weights(gen, N, K, group):
    """A quantized layer: codes of near-normal weights around a zero point near 7, packed."""
    qw = torch.zeros(N, K // 8, dtype=torch.int32, device="cuda")
    for nibble in range(8):
        q = (_randn(gen, N, K // 8) * 2.6 + 7.5).round_().clamp_(0, 15).to(torch.int32)
        qw |= q << (4 * nibble)
    G = K // group
    scales = (0.006 * torch.exp(0.3 * _randn(gen, G, N))).to(torch.float16).view(torch.int16)
    zeros = torch.zeros(G, N // 8, dtype=torch.int32, device="cuda")
    for nibble in range(8):
        z = (_randn(gen, G, N // 8) * 1.0 + 7.5).round_().clamp_(0, 15).to(torch.int32)
        zeros |= z << (4 * nibble)
    return qw, scales, zeros


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62))
    op, M, K = case["op"], case["M"], case["K"]
    bf = torch.bfloat16
    # per-channel spread of the activations, a few channels far out
    spread = torch.exp(0.5 * _randn(gen, K))
    spread[torch.randint(0, K, (8,), generator=gen, device="cuda")] *= 8.0
    d = {"case": dict(case)}
    if op.startswith("norm"):
        d["weight"] = (1.0 + 0.2 * _randn(gen, K)).to(bf)
        d["s"] = spread.sqrt().contiguous() if case["fold"] else None
        if op == "norm_bwd":
            d["h"] = (_randn(gen, M, K) * spread).to(bf)
            d["dy"] = _randn(gen, M, K).to(bf)
            d["dh"] = _randn(gen, M, K).to(bf) if case["residual"] else None
        else:
            d["x"] = _randn(gen, M, K).to(bf)
            d["residual"] = (_randn(gen, M, K) * spread).to(bf) if case["residual"] else None
        return d
    if op.startswith("linear"):
        N = case["N"]
        d["w"] = _weights(gen, N, K, case["group"])
        if op == "linear":
            d["x"] = (_randn(gen, M, K) * spread).to(bf)
            d["bias"] = _randn(gen, N).to(bf) if case["bias"] else None
            d["residual"] = _randn(gen, M, N).to(bf) if case["residual"] else None
        else:
            d["dy"] = _randn(gen, M, N).to(bf)
            d["pre"] = _randn(gen, M, N).to(bf) if case["act"] != "none" else None
        return d
    F = case["F"]
    d["gate"] = _weights(gen, F, K, case["group"])
    d["up"] = _weights(gen, F, K, case["group"])
    if op == "gated":
        d["x"] = (_randn(gen, M, K) * spread).to(bf)
    else:
        d["dh"] = _randn(gen, M, F).to(bf)
        d["g"] = _randn(gen, M, F).to(bf)
        d["u"] = _randn(gen, M, F).to(bf)
    return d


# ---------------------------------------------------------------------------------- plain forms

# element e of a word's 8 sits in the nibble at this bit
_ELEMENT_BIT = (0, 16, 4, 20, 8, 24, 12, 28)


def _dequant(w):
    """fp32 [N][K] of packed weights: (q - z) * scale."""
    qw, scales, zeros = w
    N, G = qw.shape[0], scales.shape[0]
    bits = torch.tensor(_ELEMENT_BIT, dtype=torch.int32, device=qw.device)
    q = ((qw.unsqueeze(-1) >> bits) & 15).reshape(N, G, -1).float()
    nib = torch.arange(0, 32, 4, dtype=torch.int32, device=qw.device)
    z = ((zeros.unsqueeze(-1) >> nib) & 15).reshape(G, N).t().float()
    sc = scales.view(torch.float16).t().float()
    return ((q - z.unsqueeze(-1)) * sc.unsqueeze(-1)).reshape(N, -1)


def _act(p, act):
    if act == "relu":
        return torch.where(p > 0, p, torch.zeros_like(p))
    if act == "silu":
        return p / (1.0 + torch.exp(-p))
    if act == "gelu":
        return 0.5 * p * (1.0 + torch.erf(p * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * p * (1.0 + torch.tanh(0.7978845608028654 * (p + 0.044715 * p * p * p)))
    return p


def _act_grad(p, act):
    if act == "relu":
        return (p > 0).to(p.dtype)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-p))
        return sg * (1.0 + p * (1.0 - sg))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(p * 0.7071067811865476)) + p * 0.3989422804014327 * torch.exp(-0.5 * p * p)
    if act == "gelu_tanh":
        t = torch.tanh(0.7978845608028654 * (p + 0.044715 * p * p * p))
        return 0.5 * (1.0 + t) + 0.5 * p * (1.0 - t * t) * 0.7978845608028654 * (1.0 + 0.134145 * p * p)
    return torch.ones_like(p)


def _plain_norm(d):
    h = d["x"].float()
    if d["residual"] is not None:
        h = (h + d["residual"].float()).to(torch.bfloat16).float()
    rstd = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    v = h * rstd * d["weight"].float()
    if d["s"] is not None:
        v = v / d["s"]
    return h.to(torch.bfloat16), v


def _plain(d):
    c = d["case"]
    op, bf = c["op"], torch.bfloat16
    if op == "norm":
        h, v = _plain_norm(d)
        return {"h": h, "y": v.to(bf)}
    if op == "norm8":
        h, v = _plain_norm(d)
        M, K = v.shape
        v = v.reshape(M, -1, c["group"] or K)
        scale = torch.clamp(v.abs().amax(dim=2, keepdim=True), min=TINY) / E4M3_MAX
        q = (v / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return {"h": h, "q": q.reshape(M, K), "scale": scale.reshape(M, -1)}
    if op == "norm_bwd":
        h, v = d["h"].float(), d["dy"].float()
        rstd = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        xhat = h * rstd
        if d["s"] is not None:
            v = v / d["s"]
        dweight = (v * xhat).double().sum(dim=0).float()
        v = v * d["weight"].float()
        dx = rstd * (v - xhat * (v * xhat).mean(dim=1, keepdim=True))
        if d["dh"] is not None:
            dx = dx + d["dh"].float()
        return {"dx": dx.to(bf), "dweight": dweight}
    if op == "linear":
        p = d["x"].float() @ _dequant(d["w"]).t()
        if d["bias"] is not None:
            p = p + d["bias"].float()
        y = _act(p, c["act"])
        if d["residual"] is not None:
            y = y + d["residual"].float()
        return {"y": y.to(bf)}
    if op == "linear_bwd":
        dp = d["dy"].float()
        if d["pre"] is not None:
            dp = dp * _act_grad(d["pre"].float(), c["act"])
        out = {"dx": (dp @ _dequant(d["w"])).to(bf)}
        if c["bias"]:
            out["dbias"] = dp.double().sum(dim=0).float()
        return out
    if op == "gated":
        x = d["x"].float()
        g, u = x @ _dequant(d["gate"]).t(), x @ _dequant(d["up"]).t()
        out = {"h": (_act(g, c["act"]) * u).to(bf)}
        if c["save"]:
            out["g"], out["u"] = g.to(bf), u.to(bf)
        return out
    g, u, dh = d["g"].float(), d["u"].float(), d["dh"].float()
    dg, du = dh * u * _act_grad(g, c["act"]), dh * _act(g, c["act"])
    return {"dx": (dg @ _dequant(d["gate"]) + du @ _dequant(d["up"])).to(bf)}


def _own(d):
    import w4a16_gemm_awq_b200 as w4
    c = d["case"]
    op = c["op"]
    if op == "norm":
        y, h = w4.awq_rmsnorm(d["x"], d["weight"], residual=d["residual"], s=d["s"], eps=EPS)
        return {"h": h, "y": y}
    if op == "norm8":
        q, scale, h = w4.awq_rmsnorm_e4m3(d["x"], d["weight"], residual=d["residual"], s=d["s"], eps=EPS,
                                          group_size=c["group"])
        return {"h": h, "q": q, "scale": scale}
    if op == "norm_bwd":
        dx, dweight = w4.awq_rmsnorm_backward(d["dy"], d["h"], d["weight"], s=d["s"], dh=d["dh"], eps=EPS)
        return {"dx": dx, "dweight": dweight}
    if op == "linear":
        return {"y": w4.w4a16_linear_fused(d["x"], *d["w"], bias=d["bias"], residual=d["residual"], activation=c["act"],
                                           group_size=c["group"])}
    if op == "linear_bwd":
        dx, dbias = w4.w4a16_linear_fused_backward(d["dy"], *d["w"], pre=d["pre"], activation=c["act"],
                                                   group_size=c["group"], bias_grad=c["bias"])
        return {"dx": dx, "dbias": dbias} if c["bias"] else {"dx": dx}
    if op == "gated":
        if not c["save"]:
            return {"h": w4.w4a16_gated(d["x"], d["gate"], d["up"], activation=c["act"], group_size=c["group"])}
        h, g, u = w4.w4a16_gated(d["x"], d["gate"], d["up"], activation=c["act"], group_size=c["group"], save=True)
        return {"h": h, "g": g, "u": u}
    return {"dx": w4.w4a16_gated_backward(d["dh"], d["g"], d["u"], d["gate"], d["up"], activation=c["act"],
                                          group_size=c["group"])}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------------- sizes

def _packed(N, K, group):
    return N * K // 2 + (K // group) * (2 * N + N // 2)


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    mk = 2 * M * K
    if op == "norm" or op == "norm8":
        r = 1 if case["residual"] else 0
        read = mk * (1 + r) + 2 * K + (4 * K if case["fold"] else 0)
        write = mk + (mk if op == "norm" else M * K + 4 * M * (K // (case["group"] or K)))
        return {"bytes": read + write, "flops": 8 * M * K}
    if op == "norm_bwd":
        read = mk * (3 if case["residual"] else 2) + 2 * K + (4 * K if case["fold"] else 0)
        return {"bytes": read + mk + 4 * K, "flops": 12 * M * K}
    if op == "linear":
        N = case["N"]
        return {"bytes": _packed(N, K, case["group"]) + mk + 2 * M * N * (2 if case["residual"] else 1)
                + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "linear_bwd":
        N = case["N"]
        return {"bytes": _packed(N, K, case["group"]) + mk + 2 * M * N * (1 if case["act"] == "none" else 2)
                + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    F = case["F"]
    w = 2 * _packed(F, K, case["group"])
    if op == "gated":
        return {"bytes": w + mk + 2 * M * F * (3 if case["save"] else 1), "flops": 4 * M * F * K}
    return {"bytes": w + mk + 6 * M * F, "flops": 4 * M * F * K}


# ---------------------------------------------------------------------------------- 64 bits

def _exact_weights(w):
    """fp64 [N][K]: the codes taken byte by byte, low nibble then high nibble, put in element order."""
    qw, scales, zeros = w
    N, words = qw.shape
    by = qw.contiguous().view(torch.uint8).reshape(N, words, 4)
    nibbles = torch.stack((by & 15, by >> 4), dim=3).reshape(N, words, 8)
    codes = torch.empty(N, words, 8, dtype=torch.float64, device=qw.device)
    codes[:, :, 0::2] = nibbles[:, :, 0:4].double()
    codes[:, :, 1::2] = nibbles[:, :, 4:8].double()
    zb = zeros.contiguous().view(torch.uint8)
    z = torch.stack((zb & 15, zb >> 4), dim=2).reshape(zeros.shape[0], N).double()
    sc = scales.view(torch.float16).double()
    group = words * 8 // zeros.shape[0]
    return (codes.reshape(N, -1) - z.t().repeat_interleave(group, dim=1)) * sc.t().repeat_interleave(group, dim=1)


def _exact_act(t, act):
    """(value, derivative) in fp64."""
    if act == "none":
        return t, torch.ones_like(t)
    if act == "relu":
        return t.clamp(min=0), (t > 0).double()
    if act == "silu":
        e = torch.sigmoid(t)
        return t * e, e + t * e * (1 - e)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-t / 2 ** 0.5)
        return t * cdf, cdf + t * torch.exp(-t * t / 2) / (2 * torch.pi) ** 0.5
    a = (2 / torch.pi) ** 0.5
    # 0.5 (1 + tanh z) = sigmoid(2 z)
    sg = torch.sigmoid(2 * a * (t + 0.044715 * t ** 3))
    return t * sg, sg + t * sg * (1 - sg) * 2 * a * (1 + 3 * 0.044715 * t ** 2)


def exact(case, seed):
    d = prepare(case, seed)
    op = case["op"]
    D = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    if op in ("norm", "norm8"):
        h = D["x"]
        if D["residual"] is not None:
            h = (h + D["residual"]).to(torch.bfloat16).double()
        v = h / torch.sqrt(h.square().mean(1, True) + EPS) * D["weight"]
        if D["s"] is not None:
            v = v / D["s"]
        if op == "norm":
            return {"h": h, "y": v}
        M, K = v.shape
        parts = v.reshape(M, -1, case["group"] or K)
        scale = parts.abs().amax(2).clamp(min=TINY) / E4M3_MAX
        return {"h": h, "q": (parts / scale.unsqueeze(2)).reshape(M, K), "scale": scale}
    if op == "norm_bwd":
        h, K = D["h"], case["K"]
        rstd = 1 / torch.sqrt(h.square().mean(1, True) + EPS)
        dv = D["dy"] if D["s"] is None else D["dy"] / D["s"]
        dweight = (dv * h * rstd).sum(0)
        dv = dv * D["weight"]
        dx = rstd * dv - h * rstd ** 3 * (dv * h).sum(1, True) / K
        if D["dh"] is not None:
            dx = dx + D["dh"]
        return {"dx": dx, "dweight": dweight}
    if op == "linear":
        p = D["x"] @ _exact_weights(d["w"]).t()
        if D["bias"] is not None:
            p = p + D["bias"]
        y = _exact_act(p, case["act"])[0]
        return {"y": y if D["residual"] is None else y + D["residual"]}
    if op == "linear_bwd":
        dp = D["dy"] if D["pre"] is None else D["dy"] * _exact_act(D["pre"], case["act"])[1]
        out = {"dx": dp @ _exact_weights(d["w"])}
        if case["bias"]:
            out["dbias"] = dp.sum(0)
        return out
    if op == "gated":
        g, u = D["x"] @ _exact_weights(d["gate"]).t(), D["x"] @ _exact_weights(d["up"]).t()
        out = {"h": _exact_act(g, case["act"])[0] * u}
        if case["save"]:
            out["g"], out["u"] = g, u
        return out
    a, da = _exact_act(D["g"], case["act"])
    return {"dx": (D["dh"] * D["u"] * da) @ _exact_weights(d["gate"]) + (D["dh"] * a) @ _exact_weights(d["up"])}
