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

No call records an autograd graph. The block's gradients come from
``forward_train`` and ``backward``; a call that only serves refuses tensors that
require grad where autograd is on, instead of dropping their gradients.

Device waits in the products are bounded (two seconds); results are valid when
``check_device_status``, called after them, returns.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import qmoe

_DTYPES = {torch.float32: qmoe.DTYPE_F32, torch.bfloat16: qmoe.DTYPE_BF16}
MX4_BLOCK = 32


def _dtype_code(dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"dtype must be float32 or bfloat16, not {dtype}")
    return code


def _tensor(t, name, shape, dtype, index):
    """Check an operand: a contiguous tensor of this shape and type on GPU ``index``."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on GPU {index}, "
                         f"not {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _gpu(t, name) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on a GPU, not on {t.device}")
    return index


def _serves(*tensors):
    """Refuse tensors whose gradients a call without a backward pass would drop."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("an operand requires grad, and this call records no graph: run it under torch.no_grad() or "
                             "on detached tensors (a GatedFFN's gradients come from forward_train and backward)")


def _enqueue(index, call, *args):
    """``call(*args, stream)`` on GPU ``index``, on torch's current stream of it."""
    if torch.cuda.current_device() == index:
        status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        raise qmoe.QMoEError(status, qmoe.lib.qmoe_dense_last_error().decode())


def check_device_status(device=None):
    """Wait for torch's current stream of ``device`` (default: the current one)
    and raise ``QMoEError`` (QMOE_TIMEOUT) if a device wait of any dense call or
    replay on that GPU gave up since the last check: results since then are
    undefined. Work on other streams counts once it has finished. Synchronises,
    so it belongs after a step, not after every call, and not into a capture."""
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError(f"the status is a GPU's, not {device}'s")
    _enqueue(torch.cuda.current_device() if device.index is None else device.index, qmoe.lib.qmoe_dense_take_device_status)


def _address(t):
    return None if t is None else t.data_ptr()


def _rows(x):
    """``(x, ldx)``: a 2-D x with unit stride along K and 16-byte aligned rows as
    it lies, any other layout through a contiguous copy."""
    ldx = x.shape[-1]
    if not x.is_contiguous():
        if x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= ldx and x.stride(0) * x.element_size() % 16 == 0:
            ldx = x.stride(0)
        else:
            x = x.contiguous()
    if x.data_ptr() % 16:
        x, ldx = x.clone(memory_format=torch.contiguous_format), x.shape[-1]
    return x, ldx


def _aligned(codes, scales):
    """MX4 rows at the addresses the products take (a slice's need not be):
    copies of what is off them."""
    return (codes.clone() if codes.data_ptr() % 16 else codes), (scales.clone() if scales.data_ptr() % 4 else scales)


def mx4_quantize(x):
    """x [..., K] (float32 or bfloat16, K a multiple of 32) to ``(codes, scales)``:
    uint8 [..., K/2] and [..., K/32]. A 2-D x with unit stride along K and
    16-byte aligned rows is read where it lies, any other layout through a
    contiguous copy."""
    code = _dtype_code(x.dtype)
    shape = x.shape
    if not shape or shape[-1] < MX4_BLOCK or shape[-1] % MX4_BLOCK:
        raise ValueError(f"the last dimension must be a positive multiple of {MX4_BLOCK}")
    index, K = _gpu(x, "x"), shape[-1]
    x, ldx = _rows(x)
    lead = shape[:-1]
    codes = x.new_empty((*lead, K // 2), dtype=torch.uint8)
    scales = x.new_empty((*lead, K // MX4_BLOCK), dtype=torch.uint8)
    rows = x.numel() // K
    if rows:
        _enqueue(index, qmoe.lib.qmoe_mx4_quantize, x.data_ptr(), code, rows, K, ldx, codes.data_ptr(),
                 scales.data_ptr())
    return codes, scales


def _check_mx4(codes, scales, name) -> int:
    """Check MX4 rows; their length K."""
    c = codes.shape
    if not c or c[-1] < MX4_BLOCK // 2 or c[-1] % (MX4_BLOCK // 2):
        raise ValueError(f"{name}codes must hold a positive multiple of {MX4_BLOCK} per row")
    index = codes.get_device()
    _tensor(codes, name + "codes", c, torch.uint8, index)
    _tensor(scales, name + "scales", (*c[:-1], c[-1] // (MX4_BLOCK // 2)), torch.uint8, index)
    return c[-1] * 2


def mx4_dequantize(codes, scales, dtype=torch.bfloat16):
    """The values of MX4 rows, [..., K] of ``dtype``."""
    code = _dtype_code(dtype)
    K = _check_mx4(codes, scales, "")
    index = _gpu(codes, "codes")
    codes, scales = _aligned(codes, scales)
    x = codes.new_empty((*codes.shape[:-1], K), dtype=dtype)
    rows = x.numel() // K
    if rows:
        _enqueue(index, qmoe.lib.qmoe_mx4_dequantize, codes.data_ptr(), scales.data_ptr(), rows, K, x.data_ptr(), code, K)
    return x


def mx4_linear(x_codes, x_scales, w_codes, w_scales, bias=None, dtype=torch.bfloat16):
    """y [..., N] = deq(x) deq(w)^T + bias for MX4 rows x [..., K] and w [N, K];
    bias and y are ``dtype``."""
    _serves(bias)
    code = _dtype_code(dtype)
    K = _check_mx4(x_codes, x_scales, "x_")
    if _check_mx4(w_codes, w_scales, "w_") != K or w_codes.dim() != 2 or not w_codes.shape[0]:
        raise ValueError(f"w_codes must be [N, K/2] with x's row length {K}, not {tuple(w_codes.shape)}")
    index, N = x_codes.get_device(), w_codes.shape[0]
    if w_codes.get_device() != index:
        raise ValueError(f"x is on {x_codes.device}, w on {w_codes.device}")
    if bias is not None:
        _tensor(bias, "bias", (N,), dtype, index)
    _gpu(x_codes, "x_codes")
    (x_codes, x_scales), (w_codes, w_scales) = _aligned(x_codes, x_scales), _aligned(w_codes, w_scales)
    y = x_codes.new_empty((*x_codes.shape[:-1], N), dtype=dtype)
    T = y.numel() // N
    if T:
        n = qmoe.lib.qmoe_mx4_linear_workspace_size(T, N, K)
        ws = x_codes.new_empty(n)
        _enqueue(index, qmoe.lib.qmoe_mx4_linear, T, N, K, x_codes.data_ptr(), x_scales.data_ptr(), w_codes.data_ptr(),
                 w_scales.data_ptr(), _address(bias), y.data_ptr(), code, ws.data_ptr(), n)
    return y


class MX4Linear:
    """A linear layer kept in 4 bits: ``layer(x)`` rounds x's rows to MX4 and
    multiplies; the output has x's dtype, which the bias must have too. Weights
    come as MX4 rows [N, K/2], [N, K/32], or dense through ``from_weights``."""

    def __init__(self, w_codes, w_scales, bias=None):
        self.in_features = _check_mx4(w_codes, w_scales, "w_")
        if w_codes.dim() != 2 or not w_codes.shape[0]:
            raise ValueError(f"w_codes must be [N, K/2], not {tuple(w_codes.shape)}")
        self.out_features = w_codes.shape[0]
        if bias is not None:
            _tensor(bias, "bias", (self.out_features,), bias.dtype, w_codes.get_device())
            bias = bias.detach()
        self.w_codes, self.w_scales = _aligned(w_codes, w_scales)
        self.bias = bias

    @classmethod
    def from_weights(cls, w, bias=None):
        return cls(*mx4_quantize(w), bias)

    def forward(self, x):
        _serves(x)
        code, shape, K, N, bias = _dtype_code(x.dtype), x.shape, self.in_features, self.out_features, self.bias
        index = _gpu(x, "x")
        if not shape or shape[-1] != K or self.w_codes.get_device() != index:
            raise ValueError(f"x must be [..., {K}] on {self.w_codes.device}, not {tuple(shape)} on {x.device}")
        if bias is not None and bias.dtype != x.dtype:
            raise ValueError(f"the bias is {bias.dtype}, x is {x.dtype}")
        x, ldx = _rows(x)
        y = x.new_empty((*shape[:-1], N))
        T = x.numel() // K
        if T:
            n = qmoe.lib.qmoe_mx4_linear_rows_workspace_size(T, N, K)
            ws = x.new_empty(n, dtype=torch.uint8)
            _enqueue(index, qmoe.lib.qmoe_mx4_linear_rows, T, N, K, x.data_ptr(), ldx, self.w_codes.data_ptr(),
                     self.w_scales.data_ptr(), _address(bias), y.data_ptr(), code, ws.data_ptr(), n)
        return y

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
        self._cfg = ctypes.byref(self.cfg)
        # the forward's refusal of the configuration comes before its other checks
        status = qmoe.lib.qmoe_gated_ffn_forward(self._cfg, 0, *[None] * 8, 0, None)
        if status:
            raise qmoe.QMoEError(status, qmoe.lib.qmoe_dense_last_error().decode())

    def _rows(self, x, name) -> int:
        if not x.shape or x.shape[-1] != self.hidden_size or x.dtype != torch.bfloat16 or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bfloat16 tensor [..., {self.hidden_size}], not {x.dtype} "
                             f"{tuple(x.shape)} with strides {x.stride()}")
        return x.numel() // self.hidden_size

    def _weights(self, w1, w2, b1, b2, index):
        H, I, bf = self.hidden_size, self.inter_size, torch.bfloat16
        _tensor(w1, "w1", (2 * I, H), bf, index)
        _tensor(w2, "w2", (H, I), bf, index)
        if b1 is not None:
            _tensor(b1, "b1", (2 * I,), bf, index)
        if b2 is not None:
            _tensor(b2, "b2", (H,), bf, index)

    def _forward(self, x, w1, w2, b1, b2, keep):
        T, index = self._rows(x, "x"), x.get_device()
        self._weights(w1, w2, b1, b2, index)
        _gpu(x, "x")
        y = torch.empty_like(x)
        gu = x.new_empty((T, 2 * self.inter_size), dtype=torch.float32) if keep else None
        if T:
            n = qmoe.lib.qmoe_gated_ffn_workspace_size(self._cfg, T, 0)
            ws = x.new_empty(n, dtype=torch.uint8)
            _enqueue(index, qmoe.lib.qmoe_gated_ffn_forward, self._cfg, T, x.data_ptr(), w1.data_ptr(), _address(b1),
                     w2.data_ptr(), _address(b2), _address(gu), y.data_ptr(), ws.data_ptr(), n)
        return y, gu

    def forward(self, x, w1, w2, b1=None, b2=None):
        """y, shaped like x [..., H]."""
        _serves(x, w1, w2, b1, b2)
        return self._forward(x, w1, w2, b1, b2, False)[0]

    __call__ = forward

    def forward_train(self, x, w1, w2, b1=None, b2=None):
        """``(y, gu)``: the projections gu [T, 2I] fp32 are what ``backward`` needs."""
        return self._forward(x, w1, w2, b1, b2, True)

    def backward(self, dy, x, w1, w2, gu, need_dx=True, need_weights=True, bias=False):
        """The gradients of the block for the output's gradient ``dy``; those
        not asked for are None."""
        T, index, I, H = self._rows(x, "x"), x.get_device(), self.inter_size, self.hidden_size
        if self._rows(dy, "dy") != T or dy.shape != x.shape or dy.get_device() != index:
            raise ValueError("dy and x differ in shape or device")
        self._weights(w1, w2, None, None, index)
        _tensor(gu, "gu", (T, 2 * I), torch.float32, index)
        _gpu(x, "x")
        g = GatedFFNGrads(torch.empty_like(x) if need_dx else None, torch.empty_like(w1) if need_weights else None,
                          torch.empty_like(w2) if need_weights else None, x.new_empty(2 * I) if bias else None,
                          x.new_empty(H) if bias else None)
        n = qmoe.lib.qmoe_gated_ffn_workspace_size(self._cfg, T, 1)
        ws = x.new_empty(n, dtype=torch.uint8)
        _enqueue(index, qmoe.lib.qmoe_gated_ffn_backward, self._cfg, T, dy.data_ptr(), x.data_ptr(), w1.data_ptr(),
                 w2.data_ptr(), gu.data_ptr(), _address(g.dx), _address(g.dw1), _address(g.db1), _address(g.dw2),
                 _address(g.db2), ws.data_ptr(), n)
        return g
