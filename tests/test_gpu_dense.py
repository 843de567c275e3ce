"""The dense operators on the GPU against their 64-bit references: MX4 rounding
code for code, the MX4 product, the gated feed-forward block and its gradients
within the bounds that dense_reference.py derives."""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import pytest
import torch

import dense_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dense(cuda_device):
    from weight_only_quantized_warp_b200 import dense
    return dense


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def within(got, want, bound, what=""):
    assert got.shape == want.shape, what
    got = got.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), what
    err = torch.where(nan, torch.zeros_like(want), (got - want).abs() - bound)
    worst = float(err.max()) if err.numel() else 0.0
    assert worst <= 0.0, f"{what}: {worst:.3e} outside the bound at {int(err.argmax())} of {tuple(err.shape)}"


# ------------------------------------------------------------ MX4 rounding

def _edge_rows(rows, K, dtype, seed):
    n = _gen(seed)
    x = n(rows, K) * torch.exp(3 * n(rows, 1))
    b = x.view(rows, K // 32, 32)
    if rows > 2:
        b[1] = 0.0
        b[1, -1, ::2] = -0.0
        # every grid value, every midpoint and their neighbours, with 6 in the block
        v = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 7.5, 0.2578125],
                         device="cuda")
        b[2, 0, :16], b[2, 0, 16:] = v, -v
    if rows > 8:
        b[3] *= 1e-37                       # subnormal scales
        b[4, 0, 0] = 2.0 ** -133            # a subnormal maximum
        b[4, 0, 1:] = 0.0
        b[5, -1, 5], b[6, 0, 31], b[7, 0, 0] = math.nan, math.inf, -math.inf
        b[8, 0, 0] = 3.3e38                 # the largest scale
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (9, 96), (37, 480), (130, 1056), (5, 4096), (1000, 2880)])
def test_mx4_rounding(dense, dtype, rows, K):
    x = _edge_rows(rows, K, dtype, rows + K)
    codes, scales = dense.mx4_quantize(x)
    rc, rs = ref.mx4_quantize(x)
    assert torch.equal(codes, rc) and torch.equal(scales, rs)
    v = dense.mx4_dequantize(codes, scales, dtype)
    want = ref.mx4_values(rc, rs)
    assert torch.equal(torch.isnan(v), torch.isnan(want))
    assert torch.equal(v.double().nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
def test_mx4_rounding_of_strided_and_stacked_rows(dense, dtype):
    base = _gen(5)(33, 256).to(dtype)
    for x in (base[:, 64:160], base[::2, :96], base[:, ::2][:, :96], base[1:, 1:97], base.t()[:, :32], base[:1, 32:64]):
        codes, scales = dense.mx4_quantize(x)
        rc, rs = ref.mx4_quantize(x)
        assert torch.equal(codes, rc) and torch.equal(scales, rs)
    x = base.view(3, 11, 256)
    codes, scales = dense.mx4_quantize(x)
    assert codes.shape == (3, 11, 128) and scales.shape == (3, 11, 8)
    assert torch.equal(codes.view(33, -1), ref.mx4_quantize(base)[0])
    assert dense.mx4_dequantize(codes, scales).shape == x.shape
    codes, scales = dense.mx4_quantize(base[:0])
    assert codes.shape == (0, 128) and dense.mx4_dequantize(codes, scales).shape == (0, 256)
    assert dense.mx4_quantize(base[3])[0].shape == (128,)


def test_mx4_rounding_leaves_the_rest_of_a_strided_output(dense):
    from weight_only_quantized_warp_b200 import qmoe
    codes, scales = dense.mx4_quantize(_gen(1)(6, 64))
    out = torch.full((6, 96), 5.0, device="cuda")
    qmoe.qmoe_mx4_dequantize(codes, scales, 6, 64, out, qmoe.DTYPE_F32, 96)
    assert torch.equal(out[:, 64:], torch.full((6, 32), 5.0, device="cuda"))
    assert torch.equal(out[:, :64].double(), ref.mx4_values(codes, scales))


def test_mx4_every_code_and_scale(dense):
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(-1, 16).repeat(16, 1).contiguous()   # 16 x 16 bytes
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").view(-1, 1)
    v = dense.mx4_dequantize(codes, scales, torch.float32).double()
    want = ref.mx4_values(codes, scales)
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, torch.copysign(torch.full_like(want, math.inf), want), want)
    assert torch.equal(v.nan_to_num(nan=7.0, posinf=8.0, neginf=9.0), want.nan_to_num(nan=7.0, posinf=8.0, neginf=9.0))


# ------------------------------------------------------------- MX4 product

LINEAR = [(1, 1, 32), (1, 128, 64), (1, 1000, 4096), (2, 7, 96), (3, 129, 160), (8, 256, 2880), (9, 130, 256),
          (16, 5760, 512), (17, 255, 288), (33, 96, 1408), (64, 257, 544), (65, 64, 1024), (100, 384, 992),
          (128, 128, 128), (129, 300, 224), (255, 511, 2880), (256, 256, 256), (257, 1411, 1408), (700, 130, 64),
          (1025, 640, 32), (600, 1030, 4096)]


def _linear_case(dense, T, N, K, dtype, bias, seed):
    n = _gen(seed)
    x = n(T, K) * torch.exp(n(T, 1))
    w = n(N, K) / math.sqrt(K)
    xq, wq = dense.mx4_quantize(x), dense.mx4_quantize(w)
    b = n(N).to(dtype) if bias else None
    return xq, wq, b


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", LINEAR)
def test_mx4_linear(dense, T, N, K, dtype):
    xq, wq, b = _linear_case(dense, T, N, K, dtype, (T + N) % 2 == 1, T * 31 + N)
    y = dense.mx4_linear(*xq, *wq, b, dtype)
    want, bound = ref.mx4_linear(ref.mx4_values(*xq), ref.mx4_values(*wq), b, dtype)
    within(y, want, bound, "y")
    assert torch.equal(y, dense.mx4_linear(*xq, *wq, b, dtype))      # the same on every call


def test_mx4_linear_uneven_scales_and_zero_rows(dense):
    """Scales far apart within a row, zero rows, and sums that cancel."""
    n = _gen(3)
    x, w = n(70, 512), n(140, 512)
    x *= torch.exp2(torch.randint(-20, 20, (70, 16), device="cuda").float()).repeat_interleave(32, 1)
    w *= torch.exp2(torch.randint(-20, 20, (140, 16), device="cuda").float()).repeat_interleave(32, 1)
    x[5], w[7] = 0.0, 0.0
    xq, wq = dense.mx4_quantize(x), dense.mx4_quantize(w)
    y = dense.mx4_linear(*xq, *wq, None, torch.float32)
    want, bound = ref.mx4_linear(ref.mx4_values(*xq), ref.mx4_values(*wq), None, torch.float32)
    within(y, want, bound)
    assert not y[5].any() and not y[:, 7].any()


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", [(1, 200, 4096), (33, 130, 96), (64, 300, 992), (65, 300, 992), (129, 640, 1408),
                                   (300, 1030, 2880), (700, 260, 32), (1025, 700, 544)])
def test_mx4_linear_on_dense_rows(dense, T, N, K, dtype):
    """The call that rounds its rows equals rounding first: contiguous, strided
    and misaligned rows, with an all-zero row and a NaN."""
    n = _gen(T + K)
    base = n(T, K + 64).to(dtype)
    base[T // 2] = 0.0
    if T > 2:
        base[2, 40] = math.nan
    lin = dense.MX4Linear.from_weights(n(N, K) / math.sqrt(K), n(N).to(dtype))
    for x in (base[:, :K].contiguous(), base[:, 32:32 + K], base[:, 1:1 + K]):
        y = lin(x)
        codes, scales = dense.mx4_quantize(x)
        assert torch.equal(codes, ref.mx4_quantize(x)[0])
        want = dense.mx4_linear(codes, scales, lin.w_codes, lin.w_scales, lin.bias, dtype)
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y.nan_to_num(), want.nan_to_num())
        ref_y, bound = ref.mx4_linear(ref.mx4_values(codes, scales), ref.mx4_values(lin.w_codes, lin.w_scales), lin.bias, dtype)
        within(y, ref_y, torch.nan_to_num(bound))


@pytest.mark.parametrize("T", [1, 20, 300])
def test_mx4_linear_nan_scales_stay_in_their_rows(dense, T):
    n = _gen(4)
    x, w = n(T, 96), n(150, 96)
    if T > 1:
        x[1, 40] = math.nan
    w[149, 0] = math.inf
    xq, wq = dense.mx4_quantize(x), dense.mx4_quantize(w)
    y = dense.mx4_linear(*xq, *wq, None)
    want, bound = ref.mx4_linear(ref.mx4_values(*xq), ref.mx4_values(*wq), None, BF)
    within(y, want, torch.nan_to_num(bound))


def test_mx4_linear_writes_only_its_rows(dense):
    """y is the middle of a larger buffer, at an address only its elements align."""
    from weight_only_quantized_warp_b200 import qmoe
    for T, N in ((3, 131), (70, 131), (300, 257)):
        xq, wq, b = _linear_case(dense, T, N, 160, BF, True, T)
        buf = torch.full((T * N + 20,), 3.0, dtype=BF, device="cuda")
        ws = torch.empty(qmoe.qmoe_mx4_linear_workspace_size(T, N, 160), dtype=torch.uint8, device="cuda")
        qmoe.qmoe_mx4_linear(T, N, 160, *xq, *wq, b, buf.data_ptr() + 2 * 7, qmoe.DTYPE_BF16, ws, ws.numel())
        want, bound = ref.mx4_linear(ref.mx4_values(*xq), ref.mx4_values(*wq), b, BF)
        within(buf[7:7 + T * N].view(T, N), want, bound)
        assert (buf[:7] == 3.0).all() and (buf[7 + T * N:] == 3.0).all()
        assert qmoe.qmoe_dense_read_device_status(ws) == qmoe.QMOE_OK


@pytest.mark.parametrize("T", [1, 2, 64, 65, 300])
def test_dense_calls_stay_inside_their_workspaces(dense, T):
    """Every call with a workspace of the stated size, between canaries."""
    from weight_only_quantized_warp_b200 import qmoe
    H, I = 264, 520
    p, dy = _block(T, H, I, T)
    layer = dense.GatedFFN(H, I, swiglu_fusion=1)
    y, gu = layer.forward_train(p["x"], p["w1"], p["w2"], p["b1"], p["b2"])
    full = layer.backward(dy, p["x"], p["w1"], p["w2"], gu, bias=True)
    xq, wq, b = _linear_case(dense, T, 1000, 4096, BF, True, T)

    def guarded(n, call):
        buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        call(buf[256:256 + n], n)
        torch.cuda.synchronize()
        assert (buf[:256] == 0xA5).all() and (buf[256 + n:] == 0xA5).all()

    # outputs between canaries too
    frames = []

    def framed(like):
        buf = torch.full((like.numel() + 64,), -7.0, dtype=like.dtype, device="cuda")
        frames.append((buf, like.numel()))
        return buf[32:32 + like.numel()].view(like.shape)

    out, y2, gu2 = framed(torch.empty(T, 1000, dtype=BF)), framed(y), framed(gu)
    guarded(qmoe.qmoe_mx4_linear_workspace_size(T, 1000, 4096), lambda ws, n: qmoe.qmoe_mx4_linear(
        T, 1000, 4096, *xq, *wq, b, out, qmoe.DTYPE_BF16, ws, n))
    assert torch.equal(out, dense.mx4_linear(*xq, *wq, b))
    guarded(qmoe.qmoe_gated_ffn_workspace_size(layer.cfg, T, False), lambda ws, n: qmoe.qmoe_gated_ffn_forward(
        layer.cfg, T, p["x"], p["w1"], p["b1"], p["w2"], p["b2"], gu2, y2, ws, n))
    assert torch.equal(y, y2) and torch.equal(gu, gu2)
    x32 = p["x"].float()[:, :256].contiguous()
    lin = dense.MX4Linear.from_weights(_gen(1)(1000, 256), None)
    out2 = framed(torch.empty(T, 1000))
    guarded(qmoe.qmoe_mx4_linear_rows_workspace_size(T, 1000, 256), lambda ws, n: qmoe.qmoe_mx4_linear_rows(
        T, 1000, 256, x32, 256, lin.w_codes, lin.w_scales, None, out2, qmoe.DTYPE_F32, ws, n))
    assert torch.equal(out2, lin(x32))
    g = [framed(t) for t in full]
    guarded(qmoe.qmoe_gated_ffn_workspace_size(layer.cfg, T, True), lambda ws, n: qmoe.qmoe_gated_ffn_backward(
        layer.cfg, T, dy, p["x"], p["w1"], p["w2"], gu, g[0], g[1], g[3], g[2], g[4], ws, n))
    for a, b in zip(g, full):
        assert torch.equal(a, b)
    for buf, n in frames:
        assert (buf[:32] == -7.0).all() and (buf[32 + n:] == -7.0).all()


def test_mx4_linear_layer(dense):
    n = _gen(11)
    w, b, x = n(200, 352) / 18, n(200).to(BF), n(2, 9, 352).to(BF)
    layer = dense.MX4Linear.from_weights(w, b)
    y = layer(x)
    xv = ref.mx4_values(*ref.mx4_quantize(x.view(18, 352)))
    want, bound = ref.mx4_linear(xv, ref.mx4_values(*ref.mx4_quantize(w)), b, BF)
    within(y.view(18, 200), want, bound)
    assert layer(x[:, :0]).shape == (2, 0, 200)


# ------------------------------------------------------------- gated block

def _block(T, H, I, seed, bias=True, scale=1.0):
    n = _gen(seed)
    p = dict(x=(n(T, H) * scale).to(BF), w1=(n(2 * I, H) / math.sqrt(H)).to(BF), w2=(n(H, I) / math.sqrt(I)).to(BF))
    p["b1"], p["b2"] = (n(2 * I).to(BF), n(H).to(BF)) if bias else (None, None)
    return p, n(T, H).to(BF)


KINDS = [(0, 0), (1, 0), (1, 1), (2, 0), (3, 0), (4, 0)]
SWIGLU_OPTS = dict(activation_alpha=1.702, activation_beta=1.0, swiglu_limit=1.5)


def _run(dense, p, dy, kind, fusion, tanh=0, opts=None, **kw):
    T, H = p["x"].shape
    I = p["w2"].shape[1]
    opts = opts or {}
    layer = dense.GatedFFN(H, I, activation_type=kind, swiglu_fusion=fusion, gelu_mode=tanh, **opts)
    y, gu = layer.forward_train(p["x"], p["w1"], p["w2"], p["b1"], p["b2"])
    g = layer.backward(dy, p["x"], p["w1"], p["w2"], gu, bias=True, **kw)
    r = ref.Block(**p, kind=kind, fusion=fusion, tanh=bool(tanh), alpha=opts.get("activation_alpha", 0.0),
                  beta=opts.get("activation_beta", 0.0), limit=opts.get("swiglu_limit", 0.0))
    return layer, y, gu, g, r


def _check(y, gu, g, r, dy):
    want, bound = r.forward()
    within(gu, r.gu, r.egu, "gu")
    within(y, want, bound, "y")
    for name, (v, e) in r.backward(dy).items():
        within(getattr(g, name), v, e, name)


SHAPES = [(1, 8, 8), (1, 2048, 1408), (2, 64, 72), (7, 136, 24), (16, 264, 520), (17, 72, 136), (33, 512, 264),
          (64, 256, 1408), (65, 120, 64), (127, 264, 128), (128, 128, 128), (129, 520, 136), (255, 64, 392),
          (257, 200, 264), (300, 1032, 520), (513, 256, 256), (1030, 136, 72)]


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_gated_block(dense, T, H, I):
    fusion = 1 + (T + I // 8) % 2
    opts = SWIGLU_OPTS if T % 2 else {}
    p, dy = _block(T, H, I, T + H + I, bias=T % 3 != 0)
    layer, y, gu, g, r = _run(dense, p, dy, ref.SWIGLU, fusion, opts=opts)
    _check(y, gu, g, r, dy)
    # serving form: the same y, and the same again
    assert torch.equal(layer.forward(p["x"], p["w1"], p["w2"], p["b1"], p["b2"]), y)
    again = layer.backward(dy, p["x"], p["w1"], p["w2"], gu, bias=True)
    for a, b in zip(g, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [65, 100, 128, 129])
def test_gated_block_large_weights(dense, T):
    """Token counts on both sides of the switch for weights of 32 MB and more."""
    p, dy = _block(T, 2056, 4104, T)
    layer, y, gu, g, r = _run(dense, p, dy, ref.SWIGLU, 1, opts=SWIGLU_OPTS)
    _check(y, gu, g, r, dy)
    xq, wq, b = _linear_case(dense, T, 8200, 8224, BF, True, T)
    y = dense.mx4_linear(*xq, *wq, b)
    want, bound = ref.mx4_linear(ref.mx4_values(*xq), ref.mx4_values(*wq), b, BF)
    within(y, want, bound)


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("fusion", [1, 2])
@pytest.mark.parametrize("kind,tanh", KINDS)
def test_gated_block_activations(dense, kind, tanh, fusion, T):
    p, dy = _block(T, 96, 200, 7 * kind + fusion + T, scale=2.0)
    opts = SWIGLU_OPTS if kind == ref.SWIGLU else {}
    _, y, gu, g, r = _run(dense, p, dy, kind, fusion, tanh, opts)
    _check(y, gu, g, r, dy)


@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("kind,tanh", KINDS)
def test_gated_block_saturated_activations(dense, kind, tanh, T):
    """Projections around 1e13: sigmoids at 0 or 1, whose slopes' factors leave
    fp32; every result stays finite and within its bound."""
    p, dy = _block(T, 64, 72, kind + T, bias=False, scale=1e13)
    _, y, gu, g, r = _run(dense, p, dy, kind, 2, tanh, SWIGLU_OPTS if kind == ref.SWIGLU else {})
    assert all(torch.isfinite(t).all() for t in (y, *g))
    _check(y, gu, g, r, dy)


def test_gated_block_skips_what_is_not_asked_for(dense):
    p, dy = _block(70, 128, 136, 1)
    layer, y, gu, full, r = _run(dense, p, dy, ref.SILU, 2)
    dx = layer.backward(dy, p["x"], p["w1"], p["w2"], gu, need_weights=False)
    assert dx.dw1 is None and dx.db1 is None and torch.equal(dx.dx, full.dx)
    dw = layer.backward(dy, p["x"], p["w1"], p["w2"], gu, need_dx=False)
    assert dw.dx is None and torch.equal(dw.dw1, full.dw1) and torch.equal(dw.dw2, full.dw2)
    db = layer.backward(dy, p["x"], p["w1"], p["w2"], gu, need_dx=False, need_weights=False, bias=True)
    assert torch.equal(db.db1, full.db1) and torch.equal(db.db2, full.db2)


def test_gated_block_without_tokens(dense):
    p, dy = _block(0, 64, 72, 1)
    layer, y, gu, g, _ = _run(dense, p, dy, ref.SILU, 1)
    assert y.shape == (0, 64) and g.dx.shape == (0, 64)
    assert g.dw1.shape == (144, 64)
    for t in g[1:]:
        assert not t.any()


def test_gated_block_extreme_rows(dense):
    """A NaN or an infinity stays in its token's row of y and dx; a zero row
    gives the bias path alone; large rows saturate without NaN."""
    p, dy = _block(40, 64, 136, 9)
    x = p["x"]
    x[3, 5], x[4, 6], x[7] = math.nan, math.inf, 0.0
    x[9] = (x[9].float() * 1e4).to(BF)
    _, y, gu, g, r = _run(dense, p, dy, ref.SWIGLU, 2)
    clean = [i for i in range(40) if i not in (3, 4)]
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[4]).all()
    p2 = dict(p, x=x[clean].contiguous())
    _, y2, gu2, g2, r2 = _run(dense, p2, dy[clean].contiguous(), ref.SWIGLU, 2)
    assert torch.equal(y[clean], y2) and torch.equal(g.dx[clean], g2.dx)
    assert torch.isfinite(y2).all()
    want, bound = r2.forward()
    within(y2, want, bound)


def test_gated_block_clamps_let_nan_through(dense):
    p, dy = _block(5, 64, 72, 2)
    p["x"][2, 1] = math.nan
    _, y, _, g, _ = _run(dense, p, dy, ref.SWIGLU, 1, opts=SWIGLU_OPTS)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3, 4]]).all() and torch.isnan(g.dx[2]).all()


def test_gated_gradients_against_differences(dense):
    """The kernel's gradients along random directions against central
    differences of the 64-bit loss."""
    p, dy = _block(48, 64, 136, 21)
    _, y, gu, g, r = _run(dense, p, dy, ref.SWIGLU, 1, opts=dict(activation_alpha=1.702, activation_beta=1.0))
    r.forward()
    bounds = r.backward(dy)
    n = _gen(22)
    for name in p:
        v = n(*p[name].shape).double()

        def loss(s):
            q = {k: t.double() for k, t in p.items()}
            q[name] = q[name] + s * v
            return float((ref.Block(**q, kind=ref.SWIGLU, fusion=1, alpha=1.702, beta=1.0).forward()[0] * dy.double()).sum())

        eps = 1e-5
        diff = (loss(eps) - loss(-eps)) / (2 * eps)
        got = float((getattr(g, "d" + name).double() * v).sum())
        slack = float((bounds["d" + name][1] * v.abs()).sum())
        assert abs(diff - got) <= slack + 1e-5 * abs(diff) + 1e-5, name


# ------------------------------------------------------- streams and graphs

def test_dense_calls_on_two_streams(dense):
    """Two blocks and two products at once, on two streams, keep apart."""
    cases = [(_block(130, 256, 520, s), _linear_case(dense, 130, 700, 1024, BF, False, s)) for s in (1, 2)]
    layer = dense.GatedFFN(256, 520, activation_type=ref.SILU)

    def once(c):
        (p, dy), (xq, wq, _) = c
        y, gu = layer.forward_train(p["x"], p["w1"], p["w2"], p["b1"], p["b2"])
        return (y, *layer.backward(dy, p["x"], p["w1"], p["w2"], gu, bias=True), dense.mx4_linear(*xq, *wq))

    want = [once(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(once(cases[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for g in runs:
            for a, b in zip(w, g):
                assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 5, 300])
def test_dense_calls_in_graphs(dense, T):
    """Captured once, replayed on new inputs; two graphs in one pool replayed
    alternately."""
    n = _gen(T)
    layers = [dense.GatedFFN(128, 264, activation_type=k) for k in (ref.SILU, ref.GELU)]
    ps = [_block(T, 128, 264, k)[0] for k in (1, 2)]
    x, dy = n(T, 128).to(BF), n(T, 128).to(BF)
    lin = [dense.MX4Linear.from_weights(n(300, 128)) for _ in range(2)]

    def once(i):
        p = ps[i]
        y, gu = layers[i].forward_train(x, p["w1"], p["w2"], p["b1"], p["b2"])
        return (y, *layers[i].backward(dy, x, p["w1"], p["w2"], gu, bias=True), lin[i](x))

    once(0)
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], torch.cuda.graph_pool_handle()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(once(i))
        graphs.append(g)
    for rep in range(3):
        x.copy_(n(T, 128).to(BF))
        dy.copy_(n(T, 128).to(BF))
        for i in (0, 1):
            graphs[i].replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in outs[i]]
            for a, b in zip(got, once(i)):
                assert torch.equal(a, b)


# ------------------------------------------------- together, as they are used

def test_quantised_experts_with_a_shared_expert(dense):
    """Dense expert weights quantised here, bound as MXFP4, run with a shared
    expert's output, against the oracle on the same codes; then the shared
    expert is tuned a step against the dense experts' output, and served in
    4 bits."""
    import oracle
    from weight_only_quantized_warp_b200 import inputs as gen
    from weight_only_quantized_warp_b200 import qmoe

    cfg = gen.MoEConfig(T=24, H=256, I=192, E=4, k=2, bits=4, block_size=32, fusion=2, scale_dtype=gen.DT_E8M0,
                        weight_format=gen.WEIGHTS_MXFP4)
    inp = gen.make_inputs(cfg, 51)
    n = _gen(51)
    w1, w2 = n(cfg.E, 2 * cfg.I, cfg.H) / 16, n(cfg.E, cfg.H, cfg.I) / 14
    (c1, s1), (c2, s2) = dense.mx4_quantize(w1), dense.mx4_quantize(w2)
    m = qmoe.QMoE(cfg, "cuda:0")
    m.set_weights(c1, s1, c2, s2)
    x, lg = qmoe.to_device(inp.x, "cuda:0"), qmoe.to_device(inp.logits, "cuda:0")
    p, _ = _block(1, cfg.H, 136, 52)
    block = dense.GatedFFN(cfg.H, 136, swiglu_fusion=2)
    shared, gu = block.forward_train(x, p["w1"], p["w2"], p["b1"], p["b2"])
    y = m.forward(x, lg, shared)
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    ref_inp = dataclasses.replace(inp, fc1_w=c1.cpu().numpy(), fc1_s=s1.cpu().numpy(), fc2_w=c2.cpu().numpy(),
                                  fc2_s=s2.cpu().numpy(), shared=bits(shared))
    want = oracle.forward(ref_inp)["y"]
    err = np.abs(y.float().cpu().numpy() - want).max() / np.abs(want).max()
    assert err <= 1e-2
    # the residual of the routed experts as the block's target: gradients as the formula's
    target = n(cfg.T, cfg.H).to(BF)
    dy = ((y.float() - target.float()) / cfg.T).to(BF)
    g = block.backward(dy, x, p["w1"], p["w2"], gu, need_dx=False, bias=True)
    r = ref.Block(x, p["w1"], p["w2"], p["b1"], p["b2"], kind=ref.SWIGLU, fusion=2)
    r.forward()
    for name, (v, e) in r.backward(dy).items():
        if name != "dx":
            within(getattr(g, name), v, e, name)
    # the block's down projection served in 4 bits
    h = n(24, 160).to(BF)
    lin = dense.MX4Linear.from_weights(n(cfg.H, 160) / 12)
    served = m.forward(x, lg, lin(h))
    assert torch.isfinite(served).all()
