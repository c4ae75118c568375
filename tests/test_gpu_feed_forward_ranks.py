"""FeedForward with ranks that hold no columns: where their copies of x and of
the gradient lie does not matter."""

import pytest

import test_gpu_feed_forward as f

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ops = f.ops


def copy_of(t, off):
    """A copy of t, its rows as far apart, that begins `off` elements after a 16-byte boundary."""
    T, D = t.shape
    big = torch.zeros(T * t.stride(0) + 16, dtype=t.dtype, device="cuda")
    v = big[off:].as_strided((T, D), (t.stride(0), 1))
    v.copy_(t)
    return v


@pytest.mark.parametrize("R,T,F", [(3, 1, 4), (3, 40, 4), (3, 600, 4), (7, 300, 9), (21, 50, 40), (21, 700, 40)])
@pytest.mark.parametrize("keep", [8, 16])
def test_copies_of_ranks_without_columns_off_the_grid(ops, R, T, F, keep):
    D = 136
    b = f.Block(60, R, T, D, F, keep=keep, copies=2)
    assert b.widths[-1] == 0
    b.dy = [copy_of(b.dy[0], 0) for _ in range(R)]
    for r, n in enumerate(b.widths):
        if n == 0:
            b.x[r], b.dy[r] = copy_of(b.x[r], 1), copy_of(b.dy[r], 1)
    with ops.FeedForward(R, D, F) as op:
        b.forward(op)
        b.check_forward()
        b.backward(op)
        b.check_backward()
