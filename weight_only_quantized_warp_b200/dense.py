"""Dense operators beside the routed experts, on torch tensors.

* ``mx4_quantize`` / ``mx4_dequantize``: rows to 4-bit microscaling blocks
  (e2m1 codes and E8M0 scales, the layout ``QMoE.set_weights`` takes for
  MXFP4 experts) and back.
* ``MX4Linear``: y = x W^T + b with both operands in 4 bits.
* ``GatedFFN``: the gated feed-forward block of a shared expert, whose output
  is ``QMoE.forward``'s ``shared_output``, and its backward pass.

Marshalling only: shapes are checked and memory is allocated here, the work
runs in the library (``include/qmoe.h`` has the formulas) on the current
stream of the tensors' device. Every call allocates its own workspace from
torch's allocator, so calls on several streams and captured graphs share none.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import qmoe

_DTYPES = {torch.float32: qmoe.DTYPE_F32, torch.bfloat16: qmoe.DTYPE_BF16}
MX4_BLOCK = 32


def _dtype_code(dtype) -> int:
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float32 or bfloat16, not {dtype}")
    return _DTYPES[dtype]


def _need(cond, text):
    if not cond:
        raise ValueError(text)


def _tensor(t, name, shape, dtype, device):
    """Check an operand: a contiguous tensor of this shape, type and device."""
    _need(t.shape == shape, f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    _need(t.dtype == dtype, f"{name} must be {dtype}, not {t.dtype}")
    _need(t.device == device, f"{name} is on {t.device}, not on {device}")
    _need(t.is_contiguous(), f"{name} must be contiguous")


def _workspace(n, device):
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _rows(x):
    """x as (tensor, rows, K, row stride): a 2-D tensor with unit stride along
    K is taken as it lies, any other one through a contiguous copy."""
    if x.dim() != 2:
        x = x.reshape(-1, x.shape[-1])
    rows, K = x.shape
    es = x.element_size()
    if K and not (x.stride(1) == 1 and x.data_ptr() % 16 == 0
                  and (rows <= 1 or (x.stride(0) >= K and x.stride(0) * es % 16 == 0))):
        x = x.clone(memory_format=torch.contiguous_format)
    return x, rows, K, (x.stride(0) if rows > 1 else K)


def mx4_quantize(x):
    """x [..., K] (float32 or bfloat16, K a multiple of 32) to ``(codes, scales)``:
    uint8 [..., K/2] and [..., K/32]."""
    code = _dtype_code(x.dtype)
    _need(x.dim() >= 1 and x.shape[-1] > 0 and x.shape[-1] % MX4_BLOCK == 0,
          f"the last dimension must be a positive multiple of {MX4_BLOCK}")
    lead = x.shape[:-1]
    with torch.cuda.device(x.device):
        x, rows, K, ldx = _rows(x)
        codes = torch.empty(*lead, K // 2, dtype=torch.uint8, device=x.device)
        scales = torch.empty(*lead, K // MX4_BLOCK, dtype=torch.uint8, device=x.device)
        if rows:
            qmoe.qmoe_mx4_quantize(x.data_ptr(), code, rows, K, ldx, codes, scales)
    return codes, scales


def _check_mx4(codes, scales, name):
    _need(codes.dtype == torch.uint8 and scales.dtype == torch.uint8, f"{name}codes and {name}scales must be uint8")
    _need(codes.dim() >= 1 and codes.shape[-1] > 0 and codes.shape[-1] % (MX4_BLOCK // 2) == 0,
          f"{name}codes must hold a positive multiple of {MX4_BLOCK} per row")
    _tensor(scales, f"{name}scales", (*codes.shape[:-1], codes.shape[-1] * 2 // MX4_BLOCK), torch.uint8, codes.device)
    _need(codes.is_contiguous(), f"{name}codes must be contiguous")


def mx4_dequantize(codes, scales, dtype=torch.bfloat16):
    """The values of MX4 rows, [..., K] of ``dtype``."""
    code = _dtype_code(dtype)
    _check_mx4(codes, scales, "")
    K = codes.shape[-1] * 2
    with torch.cuda.device(codes.device):
        x = torch.empty(*codes.shape[:-1], K, dtype=dtype, device=codes.device)
        if x.numel():
            qmoe.qmoe_mx4_dequantize(codes, scales, x.numel() // K, K, x, code, K)
    return x


def mx4_linear(x_codes, x_scales, w_codes, w_scales, bias=None, dtype=torch.bfloat16):
    """y [..., N] = deq(x) deq(w)^T + bias for MX4 rows x [..., K] and w [N, K];
    bias and y are ``dtype``."""
    code = _dtype_code(dtype)
    _check_mx4(x_codes, x_scales, "x_")
    _check_mx4(w_codes, w_scales, "w_")
    dev = x_codes.device
    _need(w_codes.dim() == 2 and w_codes.shape[0] > 0, "w_codes must be [N, K/2]")
    _need(w_codes.shape[1] == x_codes.shape[-1], "x and w rows differ in length")
    _need(w_codes.device == dev, "x and w are on different devices")
    N, K = w_codes.shape[0], w_codes.shape[1] * 2
    if bias is not None:
        _tensor(bias, "bias", (N,), dtype, dev)
    with torch.cuda.device(dev):
        y = torch.empty(*x_codes.shape[:-1], N, dtype=dtype, device=dev)
        T = y.numel() // N
        if T:
            n = qmoe.qmoe_mx4_linear_workspace_size(T, N, K)
            ws = _workspace(n, dev)
            qmoe.qmoe_mx4_linear(T, N, K, x_codes, x_scales, w_codes, w_scales, bias, y, code, ws, n)
    return y


class MX4Linear:
    """A linear layer kept in 4 bits: ``layer(x)`` quantises x's rows and
    multiplies. Weights come as MX4 rows [N, K/2], [N, K/32], or dense through
    ``from_weights``."""

    def __init__(self, w_codes, w_scales, bias=None):
        _check_mx4(w_codes, w_scales, "w_")
        _need(w_codes.dim() == 2, "w_codes must be [N, K/2]")
        self.w_codes, self.w_scales, self.bias = w_codes, w_scales, bias

    @classmethod
    def from_weights(cls, w, bias=None):
        return cls(*mx4_quantize(w), bias)

    def forward(self, x):
        codes, scales = mx4_quantize(x)
        return mx4_linear(codes, scales, self.w_codes, self.w_scales, self.bias, x.dtype)

    __call__ = forward


class GatedFFNGrads(NamedTuple):
    dx: Optional[torch.Tensor]
    dw1: Optional[torch.Tensor]
    dw2: Optional[torch.Tensor]
    db1: Optional[torch.Tensor]
    db2: Optional[torch.Tensor]


class GatedFFN:
    """The gated feed-forward block y = act(x Wg^T + bg) * (x Wu^T + bu) W2^T + b2
    in bfloat16. ``w1`` [2I, H] holds gate and up rows interleaved
    (``swiglu_fusion`` 1) or one after the other (2); ``w2`` is [H, I]."""

    def __init__(self, hidden_size: int, inter_size: int, activation_type: int = qmoe.ACT_SWIGLU,
                 swiglu_fusion: int = 2, activation_alpha: float = 0.0, activation_beta: float = 0.0,
                 swiglu_limit: float = 0.0, gelu_mode: int = qmoe.GELU_ERF):
        self.hidden_size, self.inter_size = hidden_size, inter_size
        self.cfg = qmoe.qmoe_gated_ffn_config(
            hidden_size=hidden_size, inter_size=inter_size, activation_type=activation_type,
            swiglu_fusion=swiglu_fusion, activation_alpha=activation_alpha, activation_beta=activation_beta,
            swiglu_limit=swiglu_limit, gelu_mode=gelu_mode, act_dtype=qmoe.DTYPE_BF16, reserved=0)
        if not qmoe.qmoe_gated_ffn_workspace_size(self.cfg, 1, False):
            raise qmoe.QMoEError(qmoe.QMOE_INVALID_ARGUMENT, qmoe.lib.qmoe_dense_last_error().decode())

    def _check_x(self, x, name):
        _need(x.dim() >= 1 and x.shape[-1] == self.hidden_size, f"{name} must be [..., {self.hidden_size}]")
        _need(x.dtype == torch.bfloat16, f"{name} must be bfloat16, not {x.dtype}")
        _need(x.is_contiguous(), f"{name} must be contiguous")

    def _check_weights(self, w1, w2, b1, b2, dev):
        H, I, bf = self.hidden_size, self.inter_size, torch.bfloat16
        _tensor(w1, "w1", (2 * I, H), bf, dev)
        _tensor(w2, "w2", (H, I), bf, dev)
        if b1 is not None:
            _tensor(b1, "b1", (2 * I,), bf, dev)
        if b2 is not None:
            _tensor(b2, "b2", (H,), bf, dev)

    def _forward(self, x, w1, w2, b1, b2, keep):
        self._check_x(x, "x")
        dev = x.device
        self._check_weights(w1, w2, b1, b2, dev)
        T = x.numel() // self.hidden_size
        with torch.cuda.device(dev):
            y = torch.empty_like(x)
            gu = torch.empty(T, 2 * self.inter_size, dtype=torch.float32, device=dev) if keep else None
            if T:
                n = qmoe.qmoe_gated_ffn_workspace_size(self.cfg, T, False)
                qmoe.qmoe_gated_ffn_forward(self.cfg, T, x, w1, b1, w2, b2, gu, y, _workspace(n, dev), n)
        return y, gu

    def forward(self, x, w1, w2, b1=None, b2=None):
        """y, shaped like x [..., H]."""
        return self._forward(x, w1, w2, b1, b2, False)[0]

    __call__ = forward

    def forward_train(self, x, w1, w2, b1=None, b2=None):
        """``(y, gu)``: the projections gu [T, 2I] fp32 are what ``backward`` needs."""
        return self._forward(x, w1, w2, b1, b2, True)

    def backward(self, dy, x, w1, w2, gu, need_dx=True, need_weights=True, bias=False):
        """The gradients of the block for the output's gradient ``dy``; those
        not asked for are None."""
        self._check_x(dy, "dy")
        self._check_x(x, "x")
        _need(dy.shape == x.shape and dy.device == x.device, "dy and x differ in shape or device")
        dev = x.device
        self._check_weights(w1, w2, None, None, dev)
        T, I, H = x.numel() // self.hidden_size, self.inter_size, self.hidden_size
        _tensor(gu, "gu", (T, 2 * I), torch.float32, dev)
        with torch.cuda.device(dev):
            new = lambda want, *s: torch.empty(*s, dtype=torch.bfloat16, device=dev) if want else None  # noqa: E731
            g = GatedFFNGrads(torch.empty_like(x) if need_dx else None, new(need_weights, 2 * I, H),
                              new(need_weights, H, I), new(bias, 2 * I), new(bias, H))
            n = qmoe.qmoe_gated_ffn_workspace_size(self.cfg, T, True)
            qmoe.qmoe_gated_ffn_backward(self.cfg, T, dy, x, w1, w2, gu, g.dx, g.dw1, g.db1, g.dw2, g.db2,
                                         _workspace(n, dev), n)
        return g
