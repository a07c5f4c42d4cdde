"""GPU parity of the feed-forward block's kernels of many positions, at sizes
that reach each of them (tests/test_ffn_plan_cpu.py holds the lists below to
that).  The cases are whole numbers, so results are exact
(test_gpu_ffn.py says why).
"""
import pytest

from test_gpu_ffn import _run_whole

pytestmark = pytest.mark.gpu

# positions, hidden units, share dropped
WHOLE = [(8193, 1000, 0.5), (4001, 1000, 0.0), (1100, 2848, 0.5), (617, 13080, 0.0), (1025, 2992, 0.5)]


@pytest.mark.parametrize("T,F,p", WHOLE)
def test_whole_numbers(T, F, p):
    _run_whole(T, F, p)
