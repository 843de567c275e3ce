"""Dense calls that record no graph refuse tensors that require grad, before
any device is touched."""
from __future__ import annotations

import pytest
import torch

from weight_only_quantized_warp_b200 import build as libbuild

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dense():
    libbuild.build()
    from weight_only_quantized_warp_b200 import dense
    return dense


def _block():
    return [torch.zeros(s, dtype=BF) for s in ((4, 64), (256, 64), (64, 128), (256,), (64,))]


@pytest.mark.parametrize("i", range(5))
def test_gated_forward_refuses_to_drop_a_gradient(dense, i):
    layer, args = dense.GatedFFN(64, 128), _block()
    args[i].requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        layer(*args)
    for call in (torch.no_grad, torch.inference_mode):
        with call(), pytest.raises(ValueError, match="on a GPU"):     # past that check
            layer(*args)
    with pytest.raises(ValueError, match="on a GPU"):                 # its gradients come from backward
        layer.forward_train(*args)


def test_mx4_linear_refuses_to_drop_a_gradient(dense):
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    bias, x = torch.nn.Parameter(torch.zeros(4, dtype=BF)), torch.zeros(2, 64, dtype=BF, requires_grad=True)
    with pytest.raises(ValueError, match="requires grad"):
        dense.mx4_linear(c, s, c, s, bias)
    layer = dense.MX4Linear(c, s, bias)
    assert not layer.bias.requires_grad and layer.bias.data_ptr() == bias.data_ptr()
    with pytest.raises(ValueError, match="requires grad"):
        layer(x)
    with pytest.raises(ValueError, match="on a GPU"):
        layer(x.detach())
