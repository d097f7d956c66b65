"""GPU: gates of numbers that do not divide into the chip's workgroups, with rows of one and of several pieces a thread.

Runs of rows with one gate are dealt to workgroups whole or in parts: 129 to 500 gates are neither one round of 256 nor two.
Tolerances as in test_gpu_block_norm.py.
"""

import pytest

from gpu_util import note
from test_gpu_block_norm import check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,dtype,kind", [(4096, "bf16", "rms"), (2050, "f32", "layer"), (4100, "f16", "layer"), (264, "bf16", "rms")])
@pytest.mark.parametrize("gates,run", [(130, 1), (130, 3), (257, 2), (300, 1), (511, 1), (513, 2), (1025, 1)])
def test_gates(gates, run, n, dtype, kind):
    m = gates * run
    a = inputs(m, n, dtype, kind, True, True, gates, wide=dtype == "bf16")
    note(f"[block_norm] gates={gates} of {run} rows N={n} {kind} {dtype}")
    y = check_forward(a, m, n, dtype, kind, 0.9)
    check_backward(a, y, m, n, dtype, kind, 0.9)
