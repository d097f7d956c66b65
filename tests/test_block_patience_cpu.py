"""The few tokens' wait is bounded whatever it is set to (no GPU needed)."""

import pytest

import bit_weight_gemm_amd as bw
from test_q4_cpu import L  # noqa: F401  (the fixture)


def test_patience_has_a_limit(L):  # noqa: F811
    was = bw.moe_layer_set_patience(7)
    try:
        assert was == 1 << 16
        for bad in (-1, (1 << 16) + 1, (1 << 31) - 1):
            with pytest.raises(bw.Tq2Error):
                bw.moe_layer_set_patience(bad)
        assert bw.moe_layer_set_patience(1 << 16) == 7, "a refused setting changes nothing"
    finally:
        bw.moe_layer_set_patience(was)
