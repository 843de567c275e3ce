"""The dense operators that stand beside the mixture-of-experts forward, as
workloads: 4-bit microscaling rounding (quantise, then read back), the linear
layer on 4-bit operands, the gated feed-forward block of a shared expert, and
its training step.

Sizes come from the named workloads of ``inputs.py`` (hidden 4096 / 2880 /
2048, inter 14336 / 2880 / 1408) or are generic. ``run`` computes either the
plain form (elementary torch operations in 32 bits) or, with ``own`` set, the
calls of ``weight_only_quantized_warp_b200.dense``; ``exact`` computes the
definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

ACT_GELU, ACT_SILU, ACT_SWIGLU = 1, 2, 3
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # -- quantise to 4 bits and read back
        # the activation rows of one decode step
        {"name": "mx4_round_tokens", "op": "mx4_round", "rows": 8, "K": 4096, "dtype": "bf16"},
        # a dense fp32 matrix of the 2880-wide model, row count odd
        {"name": "mx4_round_f32", "op": "mx4_round", "rows": 5761, "K": 2880, "dtype": "f32"},
        # one expert's dense gate and up projections, before they are bound
        {"name": "mx4_round_fc1", "op": "mx4_round", "rows": 28672, "K": 4096, "dtype": "bf16"},
        # -- linear layer, activations quantised in the call
        # a single token through a wide projection: weight bytes and latency
        {"name": "mx4_linear_token", "op": "mx4_linear", "T": 1, "N": 14336, "K": 4096, "dtype": "bf16", "bias": False},
        # a small ragged batch of decode tokens, with bias
        {"name": "mx4_linear_batch", "op": "mx4_linear", "T": 37, "N": 5760, "K": 2880, "dtype": "bf16", "bias": True},
        # fp32 activations and output, odd token and output counts
        {"name": "mx4_linear_f32", "op": "mx4_linear", "T": 1001, "N": 2817, "K": 1408, "dtype": "f32", "bias": True},
        # a long prompt
        {"name": "mx4_linear_prompt", "op": "mx4_linear", "T": 8192, "N": 14336, "K": 4096, "dtype": "bf16", "bias": False},
        # -- gated feed-forward block, forward only
        # a single token: every weight read once
        {"name": "gated_token", "op": "gated_forward", "T": 1, "H": 4096, "I": 14336, "act": ACT_SWIGLU, "fusion": 2,
         "alpha": 1.0, "beta": 0.0, "limit": 0.0, "bias": False},
        # a prompt through the 2880-wide block: interleaved, clamped, biased
        {"name": "gated_prompt", "op": "gated_forward", "T": 1024, "H": 2880, "I": 2880, "act": ACT_SWIGLU, "fusion": 1,
         "alpha": 1.702, "beta": 1.0, "limit": 7.0, "bias": True},
        # -- training step of the block: forward that keeps its projections, then backward
        # a small micro-batch of the fine-grained model's expert
        {"name": "gated_train_small", "op": "gated_train", "T": 64, "H": 2048, "I": 1408, "act": ACT_SILU, "fusion": 2,
         "alpha": 1.0, "beta": 0.0, "limit": 0.0, "bias": False},
        # a ragged batch, every option on
        {"name": "gated_train_ragged", "op": "gated_train", "T": 1023, "H": 2880, "I": 2880, "act": ACT_SWIGLU,
         "fusion": 1, "alpha": 1.702, "beta": 1.0, "limit": 7.0, "bias": True},
        # a full batch of the wide model
        {"name": "gated_train_wide", "op": "gated_train", "T": 4096, "H": 4096, "I": 14336, "act": ACT_SWIGLU,
         "fusion": 2, "alpha": 1.0, "beta": 0.0, "limit": 0.0, "bias": False},
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number in [lo, hi], even over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["mx4_round", "mx4_linear", "gated_forward", "gated_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "mx4_round":
        return {"op": op, "rows": _spread(rng, 1, 28672), "K": _spread(rng, 32, 4096, 32), "dtype": dtype}
    if op == "mx4_linear":
        return {"op": op, "T": _spread(rng, 1, 8192), "N": _spread(rng, 64, 14336), "K": _spread(rng, 32, 4096, 32),
                "dtype": dtype, "bias": rng.random() < 0.5}
    act = rng.choice([ACT_SWIGLU, ACT_SWIGLU, ACT_SILU, ACT_GELU])
    clamped = act == ACT_SWIGLU and rng.random() < 0.5
    return {"op": op, "T": _spread(rng, 1, 8192 if op == "gated_forward" else 4096), "H": _spread(rng, 64, 4096, 8),
            "I": _spread(rng, 64, 14336, 8), "act": act, "fusion": rng.choice([1, 2]),
            "alpha": 1.702 if clamped else 1.0, "beta": 1.0 if clamped else 0.0, "limit": 7.0 if clamped else 0.0,
            "bias": rng.random() < 0.5}


def work(case):
    if case["op"] == "mx4_round":
        n, s = case["rows"] * case["K"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * s, "flops": 12 * n}
    if case["op"] == "mx4_linear":
        T, N, K, s = case["T"], case["N"], case["K"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * K * s + N * K * 17 // 32 + T * N * s + (N * s if case["bias"] else 0), "flops": 2 * T * N * K}
    T, H, I = case["T"], case["H"], case["I"]
    bias = 2 * (2 * I + H) if case["bias"] else 0
    if case["op"] == "gated_forward":
        return {"bytes": 4 * T * H + 6 * H * I + bias, "flops": 6 * T * H * I}
    # x and dy in, y and dx out, each weight in and its gradient out
    return {"bytes": 8 * T * H + 12 * H * I + 2 * bias, "flops": 18 * T * H * I}


# ------------------------------------------------------------------ inputs

def _torch_dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _rows(g, rows, K, dtype):
    """Activation or weight rows: normal, every row of its own size, a few
    large channels, and some blocks that are zero."""
    x = torch.randn(rows, K, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(torch.randn(rows, 1, generator=g, device="cuda") * 0.5)
    x *= 1.0 + 7.0 * (torch.rand(1, K, generator=g, device="cuda") < 0.01)
    zero = torch.rand(rows, K // 32, 1, generator=g, device="cuda") < 0.002
    x.view(rows, K // 32, 32).masked_fill_(zero, 0.0)
    return x.to(dtype)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    dtype = _torch_dtype(case)
    if case["op"] == "mx4_round":
        return {"x": _rows(g, case["rows"], case["K"], dtype)}
    if case["op"] == "mx4_linear":
        T, N, K = case["T"], case["N"], case["K"]
        centre = 127 + int(round(math.log2(0.4 / math.sqrt(K))))
        s = {"x": _rows(g, T, K, dtype),
             "codes": torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
             "scales": torch.randint(centre - 2, centre + 3, (N, K // 32), generator=g, device="cuda",
                                     dtype=torch.uint8)}
        s["bias"] = n(N).mul_(0.1).to(dtype) if case["bias"] else None
        return s
    T, H, I = case["T"], case["H"], case["I"]
    bf = torch.bfloat16
    s = {"x": n(T, H).to(bf), "w1": n(2 * I, H).mul_(H ** -0.5).to(bf), "w2": n(H, I).mul_(I ** -0.5).to(bf)}
    s["b1"] = n(2 * I).mul_(0.1).to(bf) if case["bias"] else None
    s["b2"] = n(H).mul_(0.1).to(bf) if case["bias"] else None
    if case["op"] == "gated_train":
        s["dy"] = n(T, H).mul_(1e-2).to(bf)
    return s


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = dict(case)
    if own:
        from weight_only_quantized_warp_b200 import dense
        if case["op"] == "mx4_linear":
            # the layer that a program keeps
            state["layer"] = dense.MX4Linear(state["codes"], state["scales"], state["bias"])
        elif case["op"] != "mx4_round":
            state["layer"] = dense.GatedFFN(case["H"], case["I"], activation_type=case["act"],
                                            swiglu_fusion=case["fusion"], activation_alpha=case["alpha"],
                                            activation_beta=case["beta"], swiglu_limit=case["limit"])
    return state


# --------------------------------------------------------------- plain form

def _power(e):
    """2^e in fp32 for whole e in [-127, 127], from its bits."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).int().view(torch.float32)


def _plain_round(x):
    """Rows rounded to the 4-bit microscaling grid, as fp32 values."""
    f = x.float().view(x.shape[0], -1, 32)
    m = f.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(m)                                   # m = f * 2^e, f in [0.5, 1)
    e = torch.where(m > 0, e - 3, torch.full_like(e, -127)).clamp(-127, 127)
    v = f.abs() * _power(-e)
    code = ((v > 0.25).byte() + (v >= 0.75).byte() + (v > 1.25).byte() + (v >= 1.75).byte() + (v > 2.5).byte()
            + (v >= 3.5).byte() + (v > 5.0).byte())
    q = torch.tensor(GRID, device=x.device)[code.int()]
    return (torch.copysign(q, f) * _power(e)).view(x.shape)


def _plain_decode(codes, scales):
    """Packed codes (even element in the low half byte) and exponent bytes to fp32."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).view(codes.shape[0], -1)
    v = grid[c.int()].view(codes.shape[0], -1, 32)
    return (v * _power(scales.int().unsqueeze(-1) - 127)).view(codes.shape[0], -1)


def _split(gu, fusion):
    if fusion == 1:
        return gu[:, 0::2], gu[:, 1::2]
    half = gu.shape[1] // 2
    return gu[:, :half], gu[:, half:]


def _join(dg, du, fusion):
    if fusion == 1:
        return torch.stack((dg, du), -1).view(dg.shape[0], -1)
    return torch.cat((dg, du), 1)


def _plain_gate(c, g, u):
    """h, and its derivatives by g and u."""
    if c["act"] == ACT_SWIGLU:
        if c["limit"] > 0:
            gin, uin = (g <= c["limit"]).to(g.dtype), (u.abs() <= c["limit"]).to(g.dtype)
            g, u = g.clamp(max=c["limit"]), u.clamp(-c["limit"], c["limit"])
        else:
            gin = uin = 1.0
        sg = 1.0 / (1.0 + torch.exp(-c["alpha"] * g))
        a = g * sg
        return (u + c["beta"]) * a, gin * (u + c["beta"]) * (sg + c["alpha"] * a * (1.0 - sg)), uin * a
    if c["act"] == ACT_SILU:
        sg = 1.0 / (1.0 + torch.exp(-g))
        a = g * sg
        return a * u, u * (sg + a * (1.0 - sg)), a
    cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return g * cdf * u, u * (cdf + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5), g * cdf


def _plain_block(s, f):
    """The block in f's precision: y, and for a training step its gradients."""
    c = s["case"]
    x, w1, w2 = f(s["x"]), f(s["w1"]), f(s["w2"])
    gu = x @ w1.t()
    if s["b1"] is not None:
        gu += f(s["b1"])
    h, hg, hu = _plain_gate(c, *_split(gu, c["fusion"]))
    y = h @ w2.t()
    if s["b2"] is not None:
        y += f(s["b2"])
    if c["op"] == "gated_forward":
        return (y,)
    dy = f(s["dy"])
    dh = dy @ w2
    dgu = _join(dh * hg, dh * hu, c["fusion"])
    out = (y, dgu @ w1, dgu.t() @ x, dy.t() @ h)
    if c["bias"]:
        out += (dgu.sum(0), dy.sum(0))
    return out


# --------------------------------------------------------------------- run

def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    dtype = _torch_dtype(c)
    if c["op"] == "mx4_round":
        return _plain_round(state["x"]).to(dtype)
    if c["op"] == "mx4_linear":
        y = _plain_round(state["x"]) @ _plain_decode(state["codes"], state["scales"]).t()
        if state["bias"] is not None:
            y += state["bias"].float()
        return y.to(dtype)
    return tuple(t.to(torch.bfloat16) for t in _plain_block(state, torch.Tensor.float))


def _run_own(c, state):
    from weight_only_quantized_warp_b200 import dense
    if c["op"] == "mx4_round":
        codes, scales = dense.mx4_quantize(state["x"])
        return dense.mx4_dequantize(codes, scales, state["x"].dtype)
    if c["op"] == "mx4_linear":
        return state["layer"](state["x"])
    layer = state["layer"]
    w = (state["w1"], state["w2"], state["b1"], state["b2"])
    if c["op"] == "gated_forward":
        return (layer.forward(state["x"], *w),)
    y, gu = layer.forward_train(state["x"], *w)
    grads = layer.backward(state["dy"], state["x"], state["w1"], state["w2"], gu, bias=c["bias"])
    return (y, grads.dx, grads.dw1, grads.dw2) + ((grads.db1, grads.db2) if c["bias"] else ())


# ------------------------------------------------------------------- exact

def _exact_power(e):
    """2^e in fp64 for whole e, exactly (the bits of a normal number)."""
    return ((e.long() + 1023) * 2 ** 52).view(torch.float64)


def _exact_round(x):
    """The definition: 2^(floor(log2 max) - 2) per block, nearest grid value,
    a tie to the even code. The grid's spacing is 1/2 below 2, 1 below 4, 2 above."""
    f = x.double().reshape(x.shape[0], -1, 32)
    m = f.abs().amax(-1, keepdim=True)
    e = torch.frexp(torch.where(m > 0, m, torch.ones_like(m)))[1].double() - 3.0
    scale = torch.where(m > 0, _exact_power(e.clamp(-127, 127)), torch.ones_like(m))
    v = f / scale
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    return ((torch.round(a / step) * step).clamp(max=6.0) * torch.sign(v) * scale).reshape(x.shape)


def _exact_decode(codes, scales):
    K = codes.shape[1] * 2
    c = torch.empty(codes.shape[0], K, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes.long() % 16, codes.long() // 16
    ex, man = (c // 2) % 4, c % 2
    mag = torch.where(ex == 0, man * 0.5, (1.0 + 0.5 * man) * _exact_power(ex - 1))
    sign = 1.0 - 2.0 * (c // 8).double()
    return sign * mag.double() * _exact_power(scales.long() - 127).repeat_interleave(32, 1)


def _exact_gate(c, g, u):
    """The activation and its slope at g, and the factor beside it with its slope."""
    one = torch.ones_like(g)
    if c["act"] == ACT_GELU:
        phi = torch.special.ndtr(g)
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi), u, one
    alpha, beta, lim = (c["alpha"], c["beta"], c["limit"]) if c["act"] == ACT_SWIGLU else (1.0, 0.0, 0.0)
    gs = us = one
    if lim > 0:
        gs, us = torch.where(g > lim, 0.0, one), torch.where((u > lim) | (u < -lim), 0.0, one)
        g, u = torch.clamp_max(g, lim), torch.clamp(u, -lim, lim)
    s = torch.sigmoid(alpha * g)
    return g * s, gs * s * (1 + alpha * g * (1 - s)), u + beta, us


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "mx4_round":
        return _exact_round(s["x"])
    if case["op"] == "mx4_linear":
        y = torch.matmul(_exact_round(s["x"]), _exact_decode(s["codes"], s["scales"]).mT)
        return y if s["bias"] is None else y + s["bias"].double()
    x, w1, w2 = s["x"].double(), s["w1"].double(), s["w2"].double()
    I, rows = case["I"], torch.arange(case["I"], device="cuda")
    gi, ui = (2 * rows, 2 * rows + 1) if case["fusion"] == 1 else (rows, rows + I)
    g, u = torch.matmul(x, w1[gi].mT), torch.matmul(x, w1[ui].mT)
    if case["bias"]:
        g, u = g + s["b1"].double()[gi], u + s["b1"].double()[ui]
    a, slope, factor, fslope = _exact_gate(case, g, u)
    h = a * factor
    y = torch.matmul(h, w2.mT)
    if case["bias"]:
        y = y + s["b2"].double()
    if case["op"] == "gated_forward":
        return (y,)
    dy = s["dy"].double()
    dh = torch.matmul(dy, w2)
    dgu = torch.empty(case["T"], 2 * I, dtype=torch.float64, device="cuda")
    dgu[:, gi], dgu[:, ui] = dh * factor * slope, dh * a * fslope
    out = (y, torch.matmul(dgu, w1), torch.matmul(dgu.mT, x), torch.matmul(dy.mT, h))
    return out + (dgu.sum(0), dy.sum(0)) if case["bias"] else out
