"""The vocabulary head's rows far from zero through the bounds-checked library,
as test_gpu_operators_bounds.py does for the rest: their sums are taken again by
code of its own."""

import os
import subprocess
import sys

import pytest

from conftest import HERE

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

CHILD = r"""
import sys
sys.path.insert(0, sys.argv[1])
import conftest
from ring_allreduce_gb300 import binding, operators as ops
import test_gpu_operators_masks as t
for s in t.CASES:
    if s[2] in (0.7, 1e-3):
        t.test_logprobs_of_far_rows(ops, s)
        t.test_distill_of_far_rows(ops, s)
        t.test_logprob_gradient_of_far_rows(ops, s)
        t.test_distill_gradient_of_far_rows(ops, s)
for d in ("bf16", "f32"):
    t.test_a_far_row_alone(ops, d)
print("stray accesses:", *binding.ra_debug_bounds_report())
"""


def test_no_stray_access():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_gb300 import build
    build.build(debug=True)
    res = subprocess.run([sys.executable, "-c", CHILD, HERE], env=dict(os.environ, RA_GB300_DEBUG_BOUNDS="1"),
                         capture_output=True, text=True, timeout=900)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert "stray accesses: 0 0" in res.stdout, res.stdout
