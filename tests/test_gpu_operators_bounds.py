"""The model operators through the bounds-checked library
(libra_gb300_debug.so): every global access of their kernels is checked
against the byte ranges of the call's buffers, and one outside them is counted
and skipped.  A child process runs the operators' own tests through it."""

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
import test_gpu_operators as t
for s in t.NORMS:
    t.test_norm_forward_and_backward(ops, s)
for s in t.HEADS:
    t.test_logprobs_and_gradient(ops, s)
    t.test_distill_and_gradient(ops, s, "f32")
    t.test_distill_and_gradient(ops, s, "own")
t.test_shards_are_column_slices_of_one_matrix(ops)
t.test_offsets_beyond_32_bits(ops)
for d in ("bf16", "f32"):
    t.test_top_alternatives_with_many_ties(ops, d)
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
