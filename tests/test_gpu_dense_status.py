"""A bounded device wait of the dense products that runs out is reported, to a
caller who keeps the workspace and to one who does not; no fault is raised.

With QMOE_OPT_TEST_WITHHOLD the MMA warp keeps back its first accumulator's
signal, so the epilogue's wait (limited to 1 ms here) expires: every role
leaves its loop, the call returns, and the calls after it are normal ones.
"""
from __future__ import annotations

import contextlib

import pytest
import torch

from test_gpu_dense import _block, _gen, dense  # noqa: F401

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def _withheld(qmoe):
    qmoe.qmoe_dense_set_option(qmoe.QMOE_OPT_WAIT_LIMIT_NS, 10**6)
    qmoe.qmoe_dense_set_option(qmoe.QMOE_OPT_TEST_WITHHOLD, 1)
    try:
        yield
        torch.cuda.synchronize()
    finally:
        qmoe.qmoe_dense_set_option(qmoe.QMOE_OPT_TEST_WITHHOLD, 0)
        qmoe.qmoe_dense_set_option(qmoe.QMOE_OPT_WAIT_LIMIT_NS, 2 * 10**9)


def _expired(dense):  # noqa: F811
    """The next check raises QMOE_TIMEOUT, the one after it does not."""
    with pytest.raises(dense.qmoe.QMoEError) as e:
        dense.check_device_status()
    assert e.value.status == dense.qmoe.QMOE_TIMEOUT
    dense.check_device_status("cuda:0")


@pytest.mark.parametrize("T", [3, 150])
def test_expired_wait_is_reported_without_a_workspace(dense, T):  # noqa: F811
    p, dy = _block(T, 128, 264, T)
    layer = dense.GatedFFN(128, 264, activation_type=dense.qmoe.ACT_SILU)
    lin = dense.MX4Linear.from_weights(_gen(T)(300, 128))
    args = (p["x"], p["w1"], p["w2"], p["b1"], p["b2"])
    y, gu = layer.forward_train(*args)
    calls = {"forward": lambda: layer.forward(*args), "linear": lambda: lin(p["x"]),
             "backward": lambda: layer.backward(dy, p["x"], p["w1"], p["w2"], gu, bias=True).dx}
    want = {k: f() for k, f in calls.items()}
    dense.check_device_status()
    for name, f in calls.items():
        with _withheld(dense.qmoe):
            f()                                        # the call itself returns
        _expired(dense)
        assert torch.equal(f(), want[name])            # and the next one is a normal one
        dense.check_device_status()


@pytest.mark.parametrize("T", [3, 150])
def test_expired_wait_stands_in_the_workspace(dense, T):  # noqa: F811
    q = dense.qmoe
    p, _ = _block(T, 64, 72, T)
    cfg = dense.GatedFFN(64, 72).cfg
    y, ws = torch.empty_like(p["x"]), torch.empty(q.qmoe_gated_ffn_workspace_size(cfg, T, False), dtype=torch.uint8, device="cuda")

    def call():
        q.qmoe_gated_ffn_forward(cfg, T, p["x"], p["w1"], None, p["w2"], None, None, y, ws, ws.numel())
        return q.qmoe_dense_read_device_status(ws)

    assert call() == q.QMOE_OK
    with _withheld(q):
        assert call() == q.QMOE_TIMEOUT
    assert call() == q.QMOE_OK
    _expired(dense)


def test_check_refuses_a_capture_and_sees_replays(dense):  # noqa: F811
    lin, x = dense.MX4Linear.from_weights(_gen(1)(64, 64)), _gen(2)(4, 64)
    want = lin(x)
    torch.cuda.synchronize()
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lin(x)
        with pytest.raises(dense.qmoe.QMoEError) as e:
            dense.check_device_status()
        assert e.value.status == dense.qmoe.QMOE_INVALID_ARGUMENT
    with _withheld(dense.qmoe), torch.cuda.graph(h):
        lin(x)
    g.replay()
    dense.check_device_status()
    assert torch.equal(y, want)
    h.replay()                                         # keeps the options of its capture
    _expired(dense)
