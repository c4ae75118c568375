"""FeedForward and Checkpoint through the bounds-checked library, as
test_gpu_operators_bounds.py does for the operators before them: every access
that is not a copy by tensor map (those end at their matrix's own bounds)."""

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
import test_gpu_feed_forward as f
import test_gpu_checkpoint as c
for shape in f.SHAPES[:-1]:
    for off in (0, 1):
        f.test_forward_and_backward(ops, shape, off)
for shape in f.SHAPES[2:-1:3]:
    f.test_types_activations_and_kept_forms(ops, shape, "f16", "gelu", 16, 1, "f32")
for T in (1, 17, 48, 130):
    f.test_forward_of_few_tokens(ops, T, 3, 1000, 700, "f16", "gelu")
f.test_no_rows(ops)
for T, D in c.SHAPES[:-1]:
    for pad in (0, 3, 16):
        c.test_store_and_load(ops, "bf16", T, D, pad)
        c.test_normalised_rows(ops, "f32", "bf16", "f32", T, D, pad)
c.test_offsets_beyond_32_bits(ops)
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
