"""The example runs: training in 8 bits follows float32, and the quantised
layers stay within what 3 fraction bits give.

A value keeps a relative error of at most 2^-4 (3 fraction bits), about 0.026 in
the root mean square over a binade; a product of two quantised operands has
about 0.037, a SwiGLU of three products (the gated product of two, then one
more) about 0.037 * sqrt(3) + 0.026 < 0.1.  Weights alone: about 0.026 * sqrt(3) < 0.06."""
import os
import sys

import pytest

from gpu_common import note, require_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def test_fp8_experts_example():
    require_gpu()
    note("example fp8_experts")
    import fp8_experts
    l8, lp, dense, experts = fp8_experts.main(["--steps", "40"])
    assert l8[-1] < 0.5 * l8[0] and lp[-1] < 0.5 * lp[0]
    assert abs(l8[-1] - lp[-1]) < 0.25 * lp[0]
    assert dense < 0.1
    assert all(e < 0.06 for e in experts.values())
