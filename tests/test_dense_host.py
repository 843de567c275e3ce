"""Refusals of the dense operators, before any device is touched, and the
64-bit references that the GPU tests hold the kernels to (their gradients
against differences, their rounding against a table)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import dense_reference as ref
from weight_only_quantized_warp_b200 import build as libbuild


@pytest.fixture(scope="module")
def q():
    libbuild.build()
    from weight_only_quantized_warp_b200 import qmoe
    return qmoe


A = 1 << 20      # an aligned address that is never read
OK, INVALID, UNSUPPORTED = 0, 1, 3

QUANT = [  # dtype, rows, K, ldx, x, codes, scales
    ((2, 4, 64, 64, A, A, A), INVALID), ((-1, 4, 64, 64, A, A, A), INVALID), ((1, -1, 64, 64, A, A, A), INVALID),
    ((1, 4, 0, 64, A, A, A), INVALID), ((1, 4, 48, 48, A, A, A), INVALID), ((1, 4, -32, 64, A, A, A), INVALID),
    ((1, 4, 64, 63, A, A, A), INVALID), ((1, 4, 64, 68, A, A, A), INVALID), ((0, 4, 64, 66, A, A, A), INVALID),
    ((1, 4, 64, 64, None, A, A), INVALID), ((1, 4, 64, 64, A, None, A), INVALID), ((1, 4, 64, 64, A, A, None), INVALID),
    ((1, 4, 64, 64, A + 8, A, A), INVALID), ((1, 4, 64, 64, A, A + 2, A), INVALID),
    ((1, 1 << 40, 64, 64, A, A, A), UNSUPPORTED), ((1, 0, 64, 64, None, None, None), OK),
    ((1, 4, 64, 1 << 60, A, A, A), INVALID),
]


@pytest.mark.parametrize("args,status", QUANT, ids=[str(i) for i in range(len(QUANT))])
def test_mx4_rounding_refuses(q, args, status):
    dtype, rows, K, ldx, x, codes, scales = args
    assert q.lib.qmoe_mx4_quantize(x, dtype, rows, K, ldx, codes, scales, None) == status
    assert q.lib.qmoe_mx4_dequantize(codes, scales, rows, K, x, dtype, ldx, None) == status
    if status:
        assert q.lib.qmoe_dense_last_error()


LINEAR = [
    (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(K=16), INVALID), (dict(K=40), INVALID), (dict(dtype=2), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED), (dict(T=0, y=None), OK),
    (dict(xc=None), INVALID), (dict(xs=None), INVALID), (dict(wc=None), INVALID), (dict(ws=None), INVALID),
    (dict(y=None), INVALID), (dict(xc=A + 8), INVALID), (dict(wc=A + 4), INVALID), (dict(xs=A + 2), INVALID),
    (dict(ws=A + 1), INVALID), (dict(y=A + 1), INVALID), (dict(bias=A + 1), INVALID), (dict(dtype=0, y=A + 2), INVALID),
    (dict(work=None), INVALID), (dict(work=A + 128), INVALID), (dict(size=0), INVALID),
]


@pytest.mark.parametrize("kw,status", LINEAR, ids=[str(i) for i in range(len(LINEAR))])
def test_mx4_linear_refuses(q, kw, status):
    a = dict(T=4, N=8, K=64, xc=A, xs=A, wc=A, ws=A, bias=None, y=A, dtype=1, work=A, size=1 << 40)
    a.update(kw)
    assert q.lib.qmoe_mx4_linear(a["T"], a["N"], a["K"], a["xc"], a["xs"], a["wc"], a["ws"], a["bias"], a["y"],
                                 a["dtype"], a["work"], a["size"], None) == status
    if status == INVALID and not {"work", "size"} & set(kw):
        assert q.lib.qmoe_dense_last_error()


ROWS = [
    (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(K=40), INVALID), (dict(dtype=2), INVALID),
    (dict(T=1 << 31), UNSUPPORTED), (dict(T=0, x=None, y=None, work=None), OK), (dict(ldx=63), INVALID),
    (dict(ldx=68), INVALID), (dict(x=None), INVALID), (dict(x=A + 8), INVALID), (dict(wc=None), INVALID),
    (dict(ws=None), INVALID), (dict(wc=A + 4), INVALID), (dict(ws=A + 1), INVALID), (dict(y=None), INVALID),
    (dict(y=A + 1), INVALID), (dict(bias=A + 1), INVALID), (dict(work=None), INVALID), (dict(work=A + 64), INVALID),
    (dict(size=256), INVALID),
]


@pytest.mark.parametrize("kw,status", ROWS, ids=[str(i) for i in range(len(ROWS))])
def test_mx4_linear_rows_refuses(q, kw, status):
    a = dict(T=4, N=8, K=64, x=A, ldx=64, wc=A, ws=A, bias=None, y=A, dtype=1, work=A, size=1 << 40)
    a.update(kw)
    assert q.lib.qmoe_mx4_linear_rows(a["T"], a["N"], a["K"], a["x"], a["ldx"], a["wc"], a["ws"], a["bias"], a["y"],
                                      a["dtype"], a["work"], a["size"], None) == status


def _ffn(q, **kw):
    base = dict(hidden_size=64, inter_size=128, activation_type=3, swiglu_fusion=2, act_dtype=1)
    base.update(kw)
    return q.qmoe_gated_ffn_config(**base)


FFN = [
    (dict(hidden_size=0), INVALID), (dict(inter_size=-8), INVALID), (dict(hidden_size=60), UNSUPPORTED),
    (dict(inter_size=12), UNSUPPORTED), (dict(activation_type=5), INVALID), (dict(activation_type=-1), INVALID),
    (dict(swiglu_fusion=0), INVALID), (dict(swiglu_fusion=3), INVALID), (dict(gelu_mode=2), INVALID),
    (dict(act_dtype=0), UNSUPPORTED), (dict(act_dtype=2), INVALID), (dict(reserved=1), INVALID),
    (dict(activation_alpha=float("nan")), INVALID), (dict(activation_beta=float("inf")), INVALID),
    (dict(hidden_size=1 << 31), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", FFN, ids=[str(i) for i in range(len(FFN))])
def test_gated_ffn_refuses_a_config(q, kw, status):
    c = ctypes.byref(_ffn(q, **kw))
    assert q.lib.qmoe_gated_ffn_workspace_size(c, 4, 0) == 0
    assert q.lib.qmoe_gated_ffn_forward(c, 4, A, A, None, A, None, None, A, A, 1 << 40, None) == status
    assert q.lib.qmoe_gated_ffn_backward(c, 4, A, A, A, A, A, A, A, None, A, None, A, 1 << 40, None) == status


FORWARD = [(1, None), (2, None), (4, None), (7, None), (8, None), (1, A + 8), (2, A + 2), (3, A + 1), (4, A + 4),
           (5, A + 1), (6, A + 4), (7, A + 8), (8, A + 128), (9, 64)]


@pytest.mark.parametrize("i,value", FORWARD, ids=[str(i) for i in range(len(FORWARD))])
def test_gated_ffn_forward_refuses(q, i, value):
    args = [4, A, A, None, A, None, None, A, A, 1 << 40, None]   # T, x, w1, b1, w2, b2, gu, y, workspace, bytes
    args[i] = value
    assert q.lib.qmoe_gated_ffn_forward(ctypes.byref(_ffn(q)), *args) == INVALID
    assert q.lib.qmoe_gated_ffn_forward(None, *args) == INVALID


BACKWARD = [(1, None), (2, None), (3, None), (4, None), (5, None), (11, None), (1, A + 8), (2, A + 8), (3, A + 8),
            (4, A + 8), (5, A + 8), (6, A + 8), (7, A + 8), (8, A + 1), (9, A + 8), (10, A + 1), (11, A + 64), (12, 256)]


@pytest.mark.parametrize("i,value", BACKWARD, ids=[str(i) for i in range(len(BACKWARD))])
def test_gated_ffn_backward_refuses(q, i, value):
    # T, dy, x, w1, w2, gu, dx, dw1, db1, dw2, db2, workspace, bytes
    args = [4, A, A, A, A, A, A, A, A, A, A, A, 1 << 40, None]
    args[i] = value
    assert q.lib.qmoe_gated_ffn_backward(ctypes.byref(_ffn(q)), *args) == INVALID


def test_empty_calls_are_no_ops(q):
    c = ctypes.byref(_ffn(q))
    assert q.lib.qmoe_gated_ffn_forward(c, 0, None, None, None, None, None, None, None, None, 0, None) == OK
    assert q.lib.qmoe_gated_ffn_backward(c, 4, *[None] * 11, 0, None) == OK       # no gradient asked for
    assert q.lib.qmoe_gated_ffn_backward(c, 0, *[None] * 5, A, *[None] * 5, 0, None) == OK
    assert q.lib.qmoe_gated_ffn_forward(c, -1, A, A, None, A, None, None, A, A, 1 << 40, None) == INVALID
    assert q.lib.qmoe_dense_read_device_status(None, None) == INVALID


def test_config_layout_and_sizes(q):
    assert ctypes.sizeof(q.qmoe_gated_ffn_config) == 48
    c = ctypes.byref(_ffn(q))
    size = q.lib.qmoe_gated_ffn_workspace_size
    assert 0 < size(c, 1, 0) <= size(c, 300, 0) < size(c, 300, 1)
    assert size(c, -1, 0) == 0
    assert q.lib.qmoe_mx4_linear_workspace_size(4, 8, 64) >= 256
    assert q.lib.qmoe_mx4_linear_workspace_size(4, 8, 65) == 0
    assert q.lib.qmoe_mx4_linear_rows_workspace_size(300, 8, 64) > q.lib.qmoe_mx4_linear_workspace_size(300, 8, 64) > 256
    assert q.lib.qmoe_mx4_linear_rows_workspace_size(4, 0, 64) == 0


def test_tensor_checks():
    libbuild.build()
    from weight_only_quantized_warp_b200 import dense, qmoe
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        dense.mx4_quantize(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        dense.mx4_quantize(torch.zeros(4, 48))
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        dense.mx4_dequantize(c, s[:, :1])
    with pytest.raises(ValueError):
        dense.mx4_dequantize(c, s, torch.float16)
    with pytest.raises(ValueError):
        dense.mx4_linear(c, s, c[:, :16].contiguous(), s[:, :1].contiguous())
    with pytest.raises(ValueError):
        dense.mx4_linear(c, s, c, s, bias=torch.zeros(3, dtype=bf))
    with pytest.raises(ValueError):
        dense.mx4_linear(c, s, c, s, bias=torch.zeros(4))
    with pytest.raises(ValueError):                      # on the CPU
        dense.mx4_quantize(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        dense.mx4_linear(c, s, c, s)
    lin = dense.MX4Linear(c, s, torch.zeros(4, dtype=bf))
    for x in (torch.zeros(2, 64, dtype=bf), torch.zeros(2, 32, dtype=bf), torch.zeros(2, 64, dtype=torch.float16)):
        with pytest.raises(ValueError):
            lin(x)
    with pytest.raises(ValueError):
        dense.MX4Linear(c, s, torch.zeros(5, dtype=bf))
    with pytest.raises(qmoe.QMoEError):
        dense.GatedFFN(60, 64)
    layer = dense.GatedFFN(64, 128)
    x, w1, w2 = torch.zeros(4, 64, dtype=bf), torch.zeros(256, 64, dtype=bf), torch.zeros(64, 128, dtype=bf)
    for args in ((x.float(), w1, w2), (x[:, :32], w1, w2), (x, w1[:128], w2), (x, w1, w2.t()), (x, w1, w2.float()),
                 (x.t().contiguous().t(), w1, w2), (x, w1, w2, torch.zeros(64, dtype=bf))):
        with pytest.raises(ValueError):
            layer.forward(*args)
    with pytest.raises(ValueError):
        layer.backward(x, x, w1, w2, torch.zeros(4, 256, dtype=bf))
    with pytest.raises(ValueError):
        layer.backward(x[:2], x, w1, w2, torch.zeros(4, 256))


# ---------------------------------------------------------------- references

def test_reference_rounding_against_a_table():
    v = torch.tensor([0.0, 0.2, 0.25, 0.26, 0.75, 1.0, 1.25, 1.3, 1.75, 2.4, 2.5, 2.6, 3.5, 4.9, 5.0, 5.1, 6.0, 7.9, -0.75,
                      -5.0] + [0.0] * 12)
    want = [0, 0, 0, 1, 2, 2, 2, 3, 4, 4, 4, 5, 6, 6, 6, 7, 7, 7, 10, 14] + [0] * 12
    for e in (-100, 0, 60):
        codes, scales = ref.mx4_quantize((v * 2.0 ** e).reshape(1, 32))
        got = torch.stack((codes % 16, codes // 16), -1).flatten().tolist()
        assert got == want and scales.tolist() == [[127 + e]]


@pytest.mark.parametrize("kind,tanh", [(0, False), (1, False), (1, True), (2, False), (3, False), (4, False)])
@pytest.mark.parametrize("fusion", [1, 2])
def test_reference_gradients_against_differences(kind, tanh, fusion):
    torch.manual_seed(kind + 10 * fusion)
    T, H, I = 5, 8, 16
    r = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    p = {"x": r(T, H), "w1": r(2 * I, H), "w2": r(H, I), "b1": r(2 * I), "b2": r(H)}
    dy = r(T, H)
    opts = dict(kind=kind, fusion=fusion, alpha=1.702, beta=1.0, limit=2.0, tanh=tanh)

    def loss(**kw):
        return float((ref.Block(**{**p, **kw}, **opts).forward()[0] * dy).sum())

    b = ref.Block(**p, **opts)
    b.forward()
    grads = b.backward(dy)
    eps = 1e-6
    for name in p:
        v = r(*p[name].shape)
        diff = (loss(**{name: p[name] + eps * v}) - loss(**{name: p[name] - eps * v})) / (2 * eps)
        got = float((grads["d" + name][0] * v).sum())
        assert abs(diff - got) <= 1e-6 * (1 + abs(diff)) + 1e-7 * float(grads["d" + name][0].abs().sum()), name
