"""The gated block's bias gradients: the same bits whichever of them are asked
for, and sums of unrounded terms."""
from __future__ import annotations

import pytest
import torch

import dense_reference as ref
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


@pytest.mark.parametrize("fusion", [1, 2])
@pytest.mark.parametrize("T", [1, 6, 30, 64, 66, 128, 513, 1030])
def test_bias_gradient_sums_unrounded_terms(dense, fusion, T):  # noqa: F811
    """db1 is the sum of fp32 terms, rounded once. With x = 0 and w2 = 1 the
    terms are dy times a slope that all tokens share; dy cancels between pairs
    of tokens to less than 2^-6 of its size, so that terms rounded to bf16
    would show. The bound: the slopes' 2^-14 (see test_gpu_dense_gate) of the
    sum, fp32 roundings of terms and sums, and the result's own rounding."""
    I = 136
    n = _gen(T)
    g, u = (n(I).to(BF) for _ in range(2))
    b1 = torch.stack((g, u), 1).flatten() if fusion == 1 else torch.cat((g, u))
    x, w1 = torch.zeros(T, I, dtype=BF, device="cuda"), torch.zeros(2 * I, I, dtype=BF, device="cuda")
    w2 = torch.eye(I, dtype=BF, device="cuda")
    half = T // 2
    dy = (n(T, I) * (1.0 if T == 1 else 2.0 ** -6)).to(BF)
    dy[:half] = n(half, I).to(BF)
    dy[half:2 * half] = (-dy[:half].float() * (1 + 2.0 ** -6 * torch.rand(half, I, device="cuda"))).to(BF)
    layer = dense.GatedFFN(I, I, activation_type=ref.SILU, swiglu_fusion=fusion)
    gu = layer.forward_train(x, w1, w2, b1)[1]
    db1 = layer.backward(dy, x, w1, w2, gu, need_dx=False, need_weights=False, bias=True).db1
    r = ref.Block(x, w1, w2, b1, kind=ref.SILU, fusion=fusion)
    r.forward()
    s, d, mag = (r.a / r.g)[0], dy.double().sum(0), dy.double().abs().sum(0)
    by_g, by_u = (r.slope * r.u)[0], r.a[0]
    eg, eu = 2.0 ** -14 * (2 * s + r.slope[0].abs()) * r.u[0].abs(), 2.0 ** -14 * by_u.abs()
    want = r.join((d * by_g).unsqueeze(0), (d * by_u).unsqueeze(0))[0]
    slack = r.join((d.abs() * eg).unsqueeze(0), (d.abs() * eu).unsqueeze(0))[0]
    size = r.join((mag * (by_g.abs() + eg)).unsqueeze(0), (mag * (by_u.abs() + eu)).unsqueeze(0))[0]
    slack = slack + (T + 2) * ref.ADD * size
    err = (db1.double() - want).abs() - slack - ref.HALF[BF] * (want.abs() + slack)
    assert float(err.max()) <= 0.0, f"{float(err.max()):.3e} outside the bound"
