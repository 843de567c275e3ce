"""Options of the dense products: refusals, without a device."""
from __future__ import annotations

import pytest

from weight_only_quantized_warp_b200 import build as libbuild


@pytest.mark.parametrize("option,value,status", [(2, 99999, 1), (2, 6 * 10**10 + 1, 1), (2, -1, 1), (3, 2, 1), (3, -1, 1),
                                                 (1, 0, 1), (4, 1, 1), (99, 1, 1), (2, 2 * 10**9, 0), (3, 0, 0)])
def test_dense_options(option, value, status):
    libbuild.build()
    from weight_only_quantized_warp_b200 import qmoe
    assert qmoe.lib.qmoe_dense_set_option(option, value) == status
    if status:
        with pytest.raises(qmoe.QMoEError):
            qmoe.qmoe_dense_set_option(option, value)


def test_device_status_is_a_gpus():
    libbuild.build()
    from weight_only_quantized_warp_b200 import dense
    with pytest.raises(ValueError):
        dense.check_device_status("cpu")
