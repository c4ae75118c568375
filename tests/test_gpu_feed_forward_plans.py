"""FeedForward on every kernel, token tile and split that the host may choose,
whatever it would choose for these sizes: in the bounds-checked library the
choice can be set."""

import os
import subprocess
import sys

import pytest

from conftest import HERE

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

PLANS = [(0, 0, 1)] + [(1, nt, split) for nt in range(16, 129, 16) for split in (1, 2, 4, 8) if split == 1 or nt <= 96]

CHILD = r"""
import sys
sys.path.insert(0, sys.argv[1])
import conftest
from ring_allreduce_gb300 import binding, operators as ops
import test_gpu_feed_forward as f
import test_gpu_feed_forward_padding as p
from test_gpu_feed_forward_plans import PLANS
lib = binding._lib
for bad in ((1, 0, 1), (1, 8, 1), (1, 144, 1), (1, 16, 3), (1, 16, 16), (1, 112, 2), (0, 0, 2)):
    assert lib.ra_debug_ffn_plan(*bad) == 1, bad


def both_ways(b, in_place=False):
    op = ops.FeedForward(b.R, b.D, b.F, b.dtype, b.act, b.grad_dtype)
    b.forward(op)
    b.check_forward()
    b.backward(op, in_place=in_place)
    b.check_backward()
    assert op.device_status()[0] == binding.Status.OK


for n, (few, nt, split) in enumerate(PLANS):
    assert lib.ra_debug_ffn_plan(few, nt, split) == 0
    few_tokens = nt - 5 if few else 40       # no multiple of any split
    for T in (few_tokens, 2 * (nt or 128) + 3):
        try:
            # two steps of terms (fewer than splits); the second segment of the tokens' gradients begins inside a part
            both_ways(f.Block(70 + n, 2, T, 72, 300))
            both_ways(f.Block(71 + n, 2, T, 200, 770, "f16", "gelu", keep=16, grad_dtype="f32"), in_place=True)
            both_ways(p.Hostile(16, 72 + n, 3, T, 131, 515, "f16", "gelu", 8, 2))
            both_ways(p.Hostile(16, 73 + n, 1, T, 13, 129, "bf16", "silu", 16))
            both_ways(f.Block(74 + n, 17, T, 136, 40))   # more ranks than a launch's short arguments hold; some without columns
        except AssertionError as e:
            raise AssertionError(f"plan {(few, nt, split)}, {T} tokens: {e}")
    # an infinity stays in its row
    clean, dirty = f.Block(75, 2, 37, 264, 520), f.Block(75, 2, 37, 264, 520)
    dirty.x[0][20, 5] = float("inf")
    op = ops.FeedForward(2, 264, 520)
    for b in (clean, dirty):
        b.forward(op)
    rows = [t for t in range(37) if t != 20]
    for r in range(2):
        for name in ("hidden", "parts", "gate", "up"):
            assert (getattr(clean, name)[r][rows] == getattr(dirty, name)[r][rows]).all(), (name, few, nt, split)
        assert dirty.scales[0][r][20].isnan().all() and dirty.scales[1][r][20].isnan().all()
print("plans:", len(PLANS), "stray accesses:", *binding.ra_debug_bounds_report())
"""


def test_every_plan():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_gb300 import build
    build.build(debug=True)
    res = subprocess.run([sys.executable, "-c", CHILD, HERE], env=dict(os.environ, RA_GB300_DEBUG_BOUNDS="1"),
                         capture_output=True, text=True, timeout=900)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert "plans: 27 stray accesses: 0 0" in res.stdout, res.stdout
