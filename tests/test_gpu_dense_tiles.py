"""The gated block at sizes whose tiles come out uneven: more dx tiles than the
GPU runs at once with a remainder, short and long beside the weight gradients',
and few tiles with a long reduction."""
from __future__ import annotations

import pytest
import torch

import dense_reference as ref
from test_gpu_dense import SWIGLU_OPTS, _block, _check, _gen, _run, dense  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,I", [
    (2500, 2056, 2600),    # 90 dx tiles; two short tiles in the time of a dx tile
    (1300, 4104, 1400),    # 102 dx tiles
    (2500, 2056, 264),     # dx tiles shorter than the weight gradients'
    (300, 4104, 136),      # fewer tiles than pairs in all
    (300, 64, 14336),      # two dx tiles of 448 stages
    (512, 256, 14336),
    (4096, 64, 64),        # weight gradients of one tile over all tokens
])
def test_gated_block_of_uneven_tiles(dense, T, H, I):  # noqa: F811
    p, dy = _block(T, H, I, T + H + I)
    layer, y, gu, g, r = _run(dense, p, dy, ref.SWIGLU, 1 + T % 2, opts=SWIGLU_OPTS)
    _check(y, gu, g, r, dy)
    # one product at a time: other launches, the same bits
    one = layer.backward(dy, p["x"], p["w1"], p["w2"], gu, need_weights=False)
    assert torch.equal(one.dx, g.dx)
    two = layer.backward(dy, p["x"], p["w1"], p["w2"], gu, need_dx=False)
    assert torch.equal(two.dw1, g.dw1) and torch.equal(two.dw2, g.dw2)


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_mx4_rounding_by_the_c_call(dense, bf16):  # noqa: F811
    """Rows in the middle of wider ones, into the middle of larger buffers."""
    from weight_only_quantized_warp_b200 import qmoe
    x = _gen(3)(7, 160).to(torch.bfloat16 if bf16 else torch.float32)
    codes = torch.full((7 * 48 + 32,), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((7 * 3 + 32,), 9, dtype=torch.uint8, device="cuda")
    qmoe.qmoe_mx4_quantize(x.data_ptr() + 32 * x.element_size(), qmoe.DTYPE_BF16 if bf16 else qmoe.DTYPE_F32, 7, 96, 160,
                           codes.data_ptr() + 16, scales.data_ptr() + 5)
    rc, rs = ref.mx4_quantize(x[:, 32:128].contiguous())
    assert torch.equal(codes[16:16 + 7 * 48].view(7, 48), rc) and torch.equal(scales[5:26].view(7, 3), rs)
    assert (codes[:16] == 9).all() and (codes[16 + 7 * 48:] == 9).all()
    assert (scales[:5] == 9).all() and (scales[26:] == 9).all()


@pytest.mark.parametrize("T", [1, 40, 200])
def test_mx4_slices_at_any_address(dense, T):  # noqa: F811
    """Rows of stacked codes and scales whose addresses the products do not take
    as they are: 3 scales a row, and views off the 16 bytes."""
    n = _gen(T)
    xc, xs = dense.mx4_quantize(n(T + 1, 96))
    wc, ws = dense.mx4_quantize(n(2, 51, 96))
    bias = n(51).to(torch.bfloat16)
    copies = [t.clone() for t in (xc[1:], xs[1:], wc[1], ws[1])]
    want = dense.mx4_linear(*copies, bias)
    assert ws[1].data_ptr() % 4 and torch.equal(dense.mx4_linear(xc[1:], xs[1:], wc[1], ws[1], bias), want)
    assert torch.equal(dense.MX4Linear(wc[1], ws[1], bias)(dense.mx4_dequantize(xc[1:], xs[1:])),
                       dense.MX4Linear(*copies[2:], bias)(dense.mx4_dequantize(*copies[:2])))
    odd = torch.empty(xc[1:].numel() + 1, dtype=torch.uint8, device="cuda")[1:].view(T, 48).copy_(xc[1:])
    assert torch.equal(dense.mx4_linear(odd, xs[1:], *copies[2:], bias), want)
    assert torch.equal(dense.mx4_dequantize(odd, xs[1:]), dense.mx4_dequantize(*copies[:2]))
