"""The compiled calls given something that is no weight's handle, or no truth value: an exception, not a crash (no GPU needed)."""

import subprocess
import sys

import pytest

import bit_weight_gemm_amd as bw

CALL = """
import torch, bit_weight_gemm_amd as bw
c, x, i, w = bw._calls(), torch.zeros((2, 128)), torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1))
try:
    %s
except %s as e:
    print("refused", type(e).__name__)
"""


@pytest.mark.parametrize("call,error", [("c.gemm('w', 0, x, None, None)", "TypeError"), ("c.gemm(None, 0, x, None, None)", "TypeError"),
                                        ("c.gemm(0, 0, x, None, None)", "ValueError"),
                                        ("c.moe(x, i, w, 0, 0, 0, 0, None, None)", "ValueError"),
                                        ("c.moe(x, i, w, None, 1.5, 'd', 0, None, None)", "TypeError"),
                                        ("c.address(x, 'f32', ('a', 128), 'x', None)", "TypeError"),
                                        ("bw.moe_route(x, 2, renorm=torch.zeros(2))", "RuntimeError"),
                                        ("bw.moe_route_backward(x, i, w, renorm=torch.zeros(2))", "RuntimeError")])
def test_what_is_no_handle_or_truth_value_is_refused(call, error):
    bw.lib()
    out = subprocess.run([sys.executable, "-c", CALL % (call, error)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.startswith("refused"), (out.returncode, out.stderr[-400:])
