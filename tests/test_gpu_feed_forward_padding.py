"""FeedForward where `dim` or a shard's width is no multiple of what a copy
fetches: odd dims in padded rows (on the tensor cores) and without padding (on
the CUDA cores), with NaN in everything that lies beside the rows.  Nothing there may be
read into a result, and nothing there may be written."""

import pytest

import test_gpu_feed_forward as f

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ops = f.ops


class Surrounded:
    """A [rows, width] view in a larger matrix that holds NaN (whole numbers: -128) all around it."""

    def __init__(self, rows, width, dtype, stride, lead):
        self.hostile = float("nan") if dtype.is_floating_point else -128
        self.big = torch.full((rows + 2, stride), self.hostile, device="cuda", dtype=dtype)
        self.at = (lead, lead + width)
        self.view = self.big[1:-1, lead:lead + width]
        self.view.zero_()

    def intact(self):
        whole = self.big.isnan() if self.big.dtype.is_floating_point else self.big == self.hostile
        whole[1:-1, self.at[0]:self.at[1]] = True
        return bool(whole.all())


class Hostile(f.Block):
    """`to`: rows start on multiples of as many bytes; 0: they lie end to end."""

    def __init__(self, to, *args, **kw):
        self.to = to
        super().__init__(*args, **kw)

    def place(self, rows, width, dtype):
        unit = max(self.to // dtype.itemsize, 1)
        t = Surrounded(rows, width, dtype, -(-width // unit) * unit, 0)
        self.guards.append(t)
        return t.view


SHAPES = [   # R, T, D, F
    (1, 1, 13, 5), (2, 1, 1029, 770), (2, 20, 131, 300), (3, 40, 1029, 515), (1, 130, 13, 129), (2, 257, 131, 513),
    (2, 300, 1029, 1100), (3, 700, 517, 2050), (1, 1500, 259, 1003), (2, 1100, 1033, 1535)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,act,keep,copies,grad_dtype", [("bf16", "silu", 8, 1, "bf16"), ("f16", "gelu", 16, 2, "f32")])
@pytest.mark.parametrize("to", [16, 64, 0])
def test_odd_rows(ops, shape, dtype, act, keep, copies, grad_dtype, to):
    R, T, D, F = shape
    b = Hostile(to, 50, *shape, dtype, act, keep, copies, grad_dtype=grad_dtype)
    with ops.FeedForward(R, D, F, dtype, act, grad_dtype) as op:
        b.forward(op)
        b.check_forward()
        b.backward(op)
        b.check_backward()


@pytest.mark.parametrize("T", [1, 7, 29, 100, 500])
def test_padding_of_new_rows(ops, T):
    """What ``rows`` gives has padding that nobody has written."""
    R, D, F = 2, 136, 1001
    b = f.Block(51, R, T, D, F, keep=16)
    with ops.FeedForward(R, D, F) as op:

        def rows():
            made = op.rows(T)
            for t in made:
                t.as_strided((T, t.stride(0)), (t.stride(0), 1)).fill_(float("nan"))
            return made

        b.hidden, b.gate, b.up, b.hidden2, b.dg, b.du = (rows() for _ in range(6))
        b.parts = [torch.empty_like(b.x[0]) for _ in range(R)]
        op.forward(b.x, b.wg, b.wu, b.wd, b.hidden, b.parts, b.gate, b.up)
        b.check_forward()
        b.before = [b.kept(r) for r in range(R)]
        b.dx = [torch.empty_like(b.x[0]) for _ in range(R)]
        b.gw = [[torch.empty_like(w) for w in ws] for ws in (b.wg, b.wu, b.wd)]
        op.backward(b.dy, b.x, b.wg, b.wu, b.wd, b.gate, b.up, b.hidden2, b.dg, b.du, b.dx, *b.gw)
        b.check_backward()
