"""64-bit references of the dense operators, with the bound of what a kernel
that follows the contract may be off.

Bounds count roundings: a value rounded to a type is off by at most
``finfo.eps / 2`` relative (bf16 2^-8, fp32 2^-24); an fp32 sum of n products
by at most n 2^-23 times the sum of their magnitudes (every addition off by
at most one unit of its partial sum, rounded or cut off); the activation's
fast exponential and division by 2^-18 relative to the sizes of their factors.
Errors travel through the activation by its largest slopes: |act'| <= 1.13 and
|act''| <= max(1, alpha) for every activation here (relu's kink and the
clamps, where a slope jumps, are bounded by the whole jump).
"""
from __future__ import annotations

import math

import torch

RELU, GELU, SILU, SWIGLU, IDENTITY = 0, 1, 2, 3, 4
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ADD = 2.0 ** -23
FAST = 2.0 ** -18


def power(e):
    """2^e for whole e, from the bits of a normal double (a device's pow need
    not be exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def mx4_quantize(x):
    """codes [rows, K/2] and scales [rows, K/32] of x's rows, by definition:
    the nearest of the eight magnitudes, a tie to the even code."""
    f = x.double().reshape(x.shape[0], -1, 32)
    bad = ~torch.isfinite(f).all(-1, keepdim=True)
    f = torch.where(bad, torch.zeros_like(f), f)
    m = f.abs().amax(-1, keepdim=True)
    E = torch.where(m > 0, torch.frexp(m)[1] - 3, torch.full_like(m, -127, dtype=torch.int32)).clamp(min=-127)
    v = f / power(E)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    dist = (v.abs().unsqueeze(-1) - grid).abs()
    odd = torch.tensor([0, 1] * 4, device=x.device) * 1e-12          # a tie goes to the even code
    code = (dist + odd).argmin(-1)
    code = torch.where(torch.signbit(f), code + 8, code)
    code = torch.where(bad, torch.zeros_like(code), code).reshape(x.shape)
    scales = torch.where(bad, torch.full_like(E, 255), E + 127).squeeze(-1).to(torch.uint8)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), scales


def mx4_values(codes, scales):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=codes.device)
    grid = torch.cat((grid, -grid))
    v = grid[torch.stack((codes % 16, codes // 16), -1).reshape(codes.shape[0], -1).long()]
    s = power(scales.long() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return v * s.repeat_interleave(32, 1)


def mx4_linear(xv, wv, bias, dtype):
    """(y, bound) for the values of two sets of MX4 rows."""
    y, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    err = xv.shape[1] * ADD * mag
    if bias is not None:
        y, err = y + bias.double(), err + ADD * (y.abs() + bias.double().abs())
    return y, err + HALF[dtype] * (y.abs() + err)


def act(kind, g, alpha, tanh):
    """Activation, slope."""
    if kind == RELU:
        return g.clamp(min=0), (g > 0).double()
    if kind == GELU and tanh:
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    if kind == GELU:
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if kind in (SILU, SWIGLU):
        s = torch.sigmoid(alpha * g)
        return g * s, s + alpha * g * s * (1 - s)
    return g, torch.ones_like(g)


class Block:
    """The gated block in 64 bits; ``bounds`` beside every value."""

    def __init__(self, x, w1, w2, b1=None, b2=None, kind=SWIGLU, fusion=2, alpha=0.0, beta=0.0, limit=0.0,
                 tanh=False):
        d = lambda t: None if t is None else t.double()  # noqa: E731
        self.x, self.w1, self.w2, self.b1, self.b2 = d(x), d(w1), d(w2), d(b1), d(b2)
        self.kind, self.fusion, self.tanh = kind, fusion, tanh
        self.alpha = (alpha or 1.0) if kind == SWIGLU else 1.0
        self.beta = beta if kind == SWIGLU else 0.0
        self.limit = limit if kind == SWIGLU and limit > 0 and math.isfinite(limit) else math.inf

    def split(self, t):
        return (t[:, 0::2], t[:, 1::2]) if self.fusion == 1 else t.chunk(2, 1)

    def join(self, g, u):
        return torch.stack((g, u), -1).flatten(1) if self.fusion == 1 else torch.cat((g, u), 1)

    def forward(self):
        H, I = self.x.shape[1], self.w2.shape[1]
        gu = self.x @ self.w1.t()
        self.egu = (H + 1) * ADD * (self.x.abs() @ self.w1.abs().t())
        if self.b1 is not None:
            gu = gu + self.b1
            self.egu = self.egu + ADD * gu.abs()
        self.gu = gu
        g, u = self.split(gu)
        eg, eu = self.split(self.egu)
        self.g, self.u = g.clamp(max=self.limit), u.clamp(-self.limit, self.limit) + self.beta
        a, slope = act(self.kind, self.g, self.alpha, self.tanh)
        h = a * self.u
        # slope's own size bounds the fast exponential's share
        self.fast_a = FAST * (a.abs() + self.g.abs() * 1.13)
        eh = 1.13 * self.u.abs() * eg + a.abs() * eu + 1.13 * eg * eu + self.fast_a * self.u.abs()
        self.a, self.slope, self.eg, self.eu = a, slope, eg, eu
        self.h, self.eh = h, eh + HALF[torch.bfloat16] * (h.abs() + eh)
        y = h @ self.w2.t()
        ey = self.eh @ self.w2.abs().t() + (I + 1) * ADD * ((h.abs() + self.eh) @ self.w2.abs().t())
        if self.b2 is not None:
            y = y + self.b2
            ey = ey + ADD * (y.abs() + ey)
        return y, ey + HALF[torch.bfloat16] * (y.abs() + ey)

    def backward(self, dy):
        """{name: (gradient, bound)} after ``forward``."""
        dy = dy.double()
        T, H = self.x.shape
        I, half = self.w2.shape[1], HALF[torch.bfloat16]
        dh = dy @ self.w2
        edh = H * ADD * (dy.abs() @ self.w2.abs())
        g0, u0 = self.split(self.gu)
        gin, uin = (g0 <= self.limit).double(), (u0.abs() <= self.limit).double()
        hg, hu = gin * self.slope * self.u, uin * self.a
        # by how much the slopes may move: smoothly, or by all of them where a jump is within reach
        curve = max(1.0, self.alpha)
        ehg = self.u.abs() * curve * self.eg + 1.13 * self.eu + curve * self.eg * self.eu + FAST * self.u.abs() * (
            1.13 + self.alpha * self.g.abs())
        ehu = 1.13 * self.eg + self.fast_a
        jump_g = (g0 - self.limit).abs() <= self.eg
        if self.kind == RELU:
            jump_g = jump_g | (g0.abs() <= self.eg)
        jump_u = (u0.abs() - self.limit).abs() <= self.eu
        ehg = ehg + jump_g * 1.13 * (self.u.abs() + self.eu)
        ehu = ehu + jump_u * (self.a.abs() + self.eg)
        out = {}
        dg, du = dh * hg, dh * hu
        eg_ = edh * (hg.abs() + ehg) + dh.abs() * ehg
        eu_ = edh * (hu.abs() + ehu) + dh.abs() * ehu
        dgu = self.join(dg, du)
        edgu = self.join(eg_, eu_) + 2 * ADD * dgu.abs()
        edgu = edgu + half * (dgu.abs() + edgu)

        def product(name, a, ea, b, eb, n):
            v = a @ b
            e = ea @ b.abs() if ea is not None else 0.0
            if eb is not None:
                e = e + a.abs() @ eb + (ea @ eb if ea is not None else 0.0)
            e = e + n * ADD * (a.abs() @ b.abs() + e)
            out[name] = (v, e + half * (v.abs() + e))

        product("dx", dgu, edgu, self.w1, None, 2 * I)
        product("dw1", dgu.t(), edgu.t(), self.x, None, T)
        product("dw2", dy.t(), None, self.h, self.eh, T)
        for name, v, e in (("db1", dgu, edgu), ("db2", dy, torch.zeros_like(dy))):
            s, es = v.sum(0), e.sum(0) + T * ADD * (v.abs() + e).sum(0)
            out[name] = (s, es + half * (s.abs() + es))
        return out
