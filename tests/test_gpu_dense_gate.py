"""The gated block's activation and its slopes, element by element over the
whole range of the gate: with x = 0 the projections are the bias exactly, with
w2 = 1 the output is h, and with one token's dy the bias gradient is the
gradient of the projections. So each value is held relative to its own size.
"""
from __future__ import annotations

import math

import pytest
import torch

import dense_reference as ref
from test_gpu_dense import BF, KINDS, SWIGLU_OPTS, dense  # noqa: F401

pytestmark = pytest.mark.gpu

# Kernel against formula, relative. The sigmoid's argument z carries up to five
# roundings (of 2^-24), which its exponential turns into |z| times as much, and
# the fast exponential is off by (2 + 1.17 |z|) 2^-23 by itself; beyond |z| = 88
# the sigmoid has left the normal numbers. 88 (5 2^-24 + 1.17 2^-23) is below
# 2^-14. The normal distribution function at |g| <= 12: its
# exponential of -g^2 / 2 >= -72 by the same count is off by less than
# 72 (2 2^-24 + 1.17 2^-23) < 2^-15.7, and 2^-18 is left for what multiplies it.
REL = 2.0 ** -14
GONE = 1e-35       # what is left of a product of g beyond 88 / |z / g|
HALF = ref.HALF[BF]

RANGE = [0.0, 0.5, 1.0, 1.28, 2.0, 5.0, 20.0, 80.0, 88.0, 100.0, 1e4, 1e13, 1.8e19, 1.9e19, 1e20, 1e30, 1e38]
EVERYWHERE = RANGE + [-v for v in RANGE[1:]]


def _table(dense, gates, T, fusion, kind, tanh, opts):  # noqa: F811
    """The block on these gates, and the reference's (h, dg, du) for them."""
    I = -(-len(gates) // 8) * 8
    n = torch.Generator(device="cuda")
    n.manual_seed(T + kind)
    g = torch.tensor(gates + [0.25] * (I - len(gates)), device="cuda").to(BF)
    u = (torch.rand(I, generator=n, device="cuda") + 0.5).to(BF)
    u[1::2] *= -1
    b1 = torch.stack((g, u), 1).flatten() if fusion == 1 else torch.cat((g, u))
    x = torch.zeros(T, I, dtype=BF, device="cuda")
    w1, w2 = torch.zeros(2 * I, I, dtype=BF, device="cuda"), torch.eye(I, dtype=BF, device="cuda")
    dy = torch.zeros(T, I, dtype=BF, device="cuda")
    dy[T - 1] = (torch.rand(I, generator=n, device="cuda") + 0.5).to(BF)
    layer = dense.GatedFFN(I, I, activation_type=kind, swiglu_fusion=fusion, gelu_mode=tanh, **opts)
    y, gu = layer.forward_train(x, w1, w2, b1)
    grads = layer.backward(dy, x, w1, w2, gu, bias=True)
    r = ref.Block(x, w1, w2, b1, kind=kind, fusion=fusion, tanh=bool(tanh), alpha=opts.get("activation_alpha", 0.0),
                  beta=opts.get("activation_beta", 0.0), limit=opts.get("swiglu_limit", 0.0))
    r.forward()
    return r, y, layer.forward(x, w1, w2, b1), gu, grads, dy[T - 1].double()


def _close(got, want, slack, what, gates):
    got = got.double()
    err = (got - want).abs() - slack - HALF * (want.abs() + slack)
    assert torch.isfinite(got).all() and float(err.max()) <= 0.0, (what, [
        (gates[i], float(got[i]), float(want[i])) for i in range(len(gates)) if not err[i] <= 0.0])


def _check_table(dense, gates, T, fusion, kind, tanh, opts):  # noqa: F811
    r, y, y2, gu, grads, d = _table(dense, gates, T, fusion, kind, tanh, opts)
    a, u, slope = r.a[0], r.u[0], r.slope[0]
    if tanh:  # (1 + tanh v) / 2 as the sigmoid of 2 v, which does not cancel
        g, c = r.g[0], math.sqrt(8 / math.pi)
        s = torch.sigmoid(c * (g + 0.044715 * g ** 3))
        a, slope = g * s, s + g * c * (1 + 3 * 0.044715 * g * g) * (s * (1 - s))
    s = torch.where(r.g[0] == 0.0, torch.full_like(a, 0.5), a / r.g[0])
    g0, u0 = (t[0] for t in r.split(r.gu))
    gin, uin = (g0 <= r.limit).double(), (u0.abs() <= r.limit).double()
    assert torch.equal(gu, r.gu.float())
    ea, es = REL * a.abs() + GONE, REL * (2 * s.abs() + slope.abs()) + GONE
    for t in range(y.shape[0]):
        assert torch.equal(y[t], y[0])
    assert torch.equal(y2, y)
    _close(y[0], a * u, ea * u.abs(), "h", gates)
    dg, du = r.split(grads.db1.unsqueeze(0))
    _close(dg[0], gin * d * slope * u, gin * d.abs() * es * u.abs(), "slope by g", gates)
    _close(du[0], uin * d * a, uin * d.abs() * ea, "slope by u", gates)


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("fusion", [1, 2])
@pytest.mark.parametrize("kind,tanh,opts", [(*k, {}) for k in KINDS] + [
    (3, 0, SWIGLU_OPTS), (3, 0, dict(activation_alpha=1.702, activation_beta=1.0, swiglu_limit=7.0)),
    (3, 0, dict(activation_alpha=1.702, activation_beta=1.0)), (3, 0, dict(activation_alpha=-0.75))],
    ids=lambda v: "-".join(f"{k.split('_')[1]}{x}" for k, x in v.items()) or "plain" if isinstance(v, dict) else str(v))
def test_gate_over_its_whole_range(dense, kind, tanh, opts, fusion, T):  # noqa: F811
    """Gates up to 1e38, whose squares leave fp32, of both signs: finite, with
    the formula's values and slopes, on both kernels."""
    _check_table(dense, EVERYWHERE, T, fusion, kind, tanh, opts)


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("kind,tanh,opts", [(*k, {}) for k in KINDS] + [(3, 0, SWIGLU_OPTS)],
                         ids=lambda v: ("clamped" if v else "plain") if isinstance(v, dict) else str(v))
def test_gate_of_infinity(dense, kind, tanh, opts, T):  # noqa: F811
    """act(inf) is inf, or the clamp's value; it is not NaN."""
    I, H = 16, 8
    b1 = torch.ones(2 * I, dtype=BF, device="cuda")
    b1[0] = math.inf
    x, w1 = torch.zeros(T, H, dtype=BF, device="cuda"), torch.zeros(2 * I, H, dtype=BF, device="cuda")
    y = dense.GatedFFN(H, I, activation_type=kind, gelu_mode=tanh, **opts)(
        x, w1, torch.ones(H, I, dtype=BF, device="cuda"), b1)
    assert (torch.isfinite(y) if opts else torch.isposinf(y)).all()


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("fusion", [1, 2])
@pytest.mark.parametrize("tanh", [0, 1], ids=["erf", "tanh"])
def test_gelu_keeps_its_tail(dense, tanh, fusion, T):  # noqa: F811
    """Small values of large negative gates, relative to their own size."""
    _check_table(dense, [-0.1 * k for k in range(121)], T, fusion, ref.GELU, tanh, {})
