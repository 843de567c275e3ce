"""The gated block's bias gradients: the same bits whichever of them are asked
for."""
from __future__ import annotations

import pytest
import torch

from test_gpu_dense import BF, _block, _gen, dense  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,I", [(1023, 2880, 2880), (300, 264, 520), (64, 2048, 1408), (2500, 64, 2056), (2500, 2056, 64)])
def test_bias_gradients_do_not_depend_on_what_is_asked_for(dense, T, H, I):  # noqa: F811
    """Terms of many sizes that cancel in pairs of tokens: any other order of
    the sum gives other bits in most columns."""
    from weight_only_quantized_warp_b200 import qmoe
    p, _ = _block(T, H, I, T)
    half = T // 2
    n = _gen(T + 1)
    dy = n(T, H) * torch.exp2(12 * n(T, 1))
    dy[half:2 * half] = -dy[:half]
    dy, x = dy.to(BF), p["x"]
    x[half:2 * half] = x[:half]
    layer = dense.GatedFFN(H, I, swiglu_fusion=1)
    gu = layer.forward_train(x, p["w1"], p["w2"])[1]
    both = layer.backward(dy, x, p["w1"], p["w2"], gu, need_dx=False, need_weights=False, bias=True)
    ws = torch.empty(qmoe.qmoe_gated_ffn_workspace_size(layer.cfg, T, True), dtype=torch.uint8, device="cuda")
    for want1, want2 in ((True, False), (False, True)):
        db1, db2 = torch.zeros_like(both.db1), torch.zeros_like(both.db2)
        qmoe.qmoe_gated_ffn_backward(layer.cfg, T, dy, x, p["w1"], p["w2"], gu, None, None, db1 if want1 else None,
                                     None, db2 if want2 else None, ws, ws.numel())
        if want1:
            assert torch.equal(db1, both.db1)
        if want2:
            assert torch.equal(db2, both.db2)
