"""What FeedForward.device_status says of a wait that gave up.  No wait is made
to run out: the bounds-checked library has a kernel that writes down what one would."""

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
import torch
from ring_allreduce_gb300 import binding, operators as ops
from ring_allreduce_gb300.binding import Status
lib = binding._lib


def give_up(op):
    assert lib.ra_debug_ffn_give_up(binding._P(op._config[0]), None) == 0


a, b = ops.FeedForward(2, 64, 128), ops.FeedForward(1, 72, 300)
assert a.device_status()[0] == Status.OK and b.device_status()[0] == Status.OK
give_up(a)
status, err = b.device_status()           # whoever asks first ...
assert status == Status.ERR_TIMEOUT and err.code == 2, (status, err.code)
status, err = a.device_status()           # ... does not take it from the one it concerns
assert status == Status.ERR_TIMEOUT and err.code == 2, (status, err.code)
late = ops.FeedForward(1, 8, 8)
side = torch.cuda.Stream()
for op in (a, b, late):                   # told once
    status, err = op.device_status(side)
    assert status == Status.OK and err.code == 0, (status, err.code)
give_up(a)
give_up(a)
torch.cuda.synchronize()
for op in (late, a, b):
    assert op.device_status(side)[0] == Status.ERR_TIMEOUT
    assert op.device_status()[0] == Status.OK
give_up(b)
a.close()
assert b.device_status()[0] == Status.ERR_TIMEOUT and late.device_status()[0] == Status.ERR_TIMEOUT
print("stray accesses:", *binding.ra_debug_bounds_report())
"""


def test_every_handle_is_told():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_gb300 import build
    build.build(debug=True)
    res = subprocess.run([sys.executable, "-c", CHILD, HERE], env=dict(os.environ, RA_GB300_DEBUG_BOUNDS="1"),
                         capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    assert "stray accesses: 0 0" in res.stdout, res.stdout


def test_status_does_not_end_a_capture():
    """Asked of a stream that is being captured it is refused, and the capture goes on."""
    from ring_allreduce_gb300 import build
    build.build()
    from ring_allreduce_gb300 import operators as ops
    from ring_allreduce_gb300.binding import Status
    import test_gpu_feed_forward as f
    b = f.Block(80, 2, 30, 136, 300)
    op = ops.FeedForward(2, 136, 300)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(op)
        with pytest.raises(ops.RAError) as err:
            op.device_status()
        b.backward(op)
    assert err.value.status == Status.ERR_UNSUPPORTED
    graph.replay()
    assert op.device_status()[0] == Status.OK
    b.before = [b.kept(r) for r in range(2)]
    b.check_forward()
    b.check_backward()
