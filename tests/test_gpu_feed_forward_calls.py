"""How FeedForward may be called: buffers that lie in other ways, several host threads, far rows."""

import ctypes
import threading

import pytest

import test_gpu_feed_forward as f

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ops = f.ops


def both_ways(op, b):
    b.forward(op)
    b.check_forward()
    b.backward(op)
    b.check_backward()


class Mixed(f.Block):
    """Every n-th buffer begins off the 16-byte grid, the others on it."""

    def __init__(self, n, which, *args, **kw):
        self.n, self.which, self.count = n, which, 0
        super().__init__(*args, **kw)

    def place(self, rows, width, dtype):
        off = int(self.count % self.n == self.which)
        self.count += 1
        t = f.Guarded(rows, width, dtype, -width % 16 + 16 - off, off)
        self.guards.append(t)
        return t.view


@pytest.mark.parametrize("n,which", [(2, 0), (2, 1), (3, 0), (3, 1), (3, 2), (7, 3), (50, 1), (50, 8), (50, 12)])
@pytest.mark.parametrize("keep", [8, 16])
def test_some_buffers_off_the_grid(ops, n, which, keep):
    """Products with an operand off the grid run on the CUDA cores, the others on the tensor cores."""
    both_ways(ops.FeedForward(2, 136, 700), Mixed(n, which, 30, 2, 150, 136, 700, keep=keep))


class Offset(f.Block):
    """Rows that begin `start` bytes after a 32-byte boundary."""

    def __init__(self, start, *args, **kw):
        self.start = start
        super().__init__(*args, **kw)

    def place(self, rows, width, dtype):
        t = f.Guarded(rows, width, dtype, -width % 32 + 32, 0)
        lead = self.start // t.big.element_size()
        t.big = torch.full((rows + 2, lead + t.big.shape[1] + 32 - lead), f.SENTINEL, device="cuda").to(dtype)
        t.at = (lead, width)
        t.view = t.big[1:-1, lead:lead + width]
        self.guards.append(t)
        return t.view


@pytest.mark.parametrize("start", [8, 16, 24])
@pytest.mark.parametrize("T", [20, 300])
def test_rows_on_smaller_boundaries(ops, start, T):
    both_ways(ops.FeedForward(2, 144, 640), Offset(start, 31, 2, T, 144, 640))


@pytest.mark.parametrize("T", [5, 200])
def test_shards_are_slices_of_one_matrix(ops, T):
    """Weights as rows of one matrix, hidden and kept values as columns of one, outputs of one allocation."""
    R, D, F = 3, 128, 1000
    b = f.Block(32, R, T, D, F, keep=16)
    op = ops.FeedForward(R, D, F)
    big = [torch.cat(w) for w in (b.wg, b.wu, b.wd)]
    b.wg, b.wu, b.wd = (list(w.split(op.widths)) for w in big)
    cols = lambda: list(torch.full((T, F), 7.0, dtype=b.dt, device="cuda").split(op.widths, 1))   # noqa: E731
    b.hidden, b.gate, b.up = cols(), cols(), cols()
    parts = torch.empty((R, T, D), dtype=b.dt, device="cuda")
    op.forward(b.x, b.wg, b.wu, b.wd, b.hidden, parts, b.gate, b.up)
    b.parts = list(parts)
    b.check_forward()
    b.before = [b.kept(r) for r in range(R)]
    b.hidden2, b.dg, b.du = cols(), cols(), cols()
    dx = torch.empty((R, T, D), dtype=b.dt, device="cuda")
    grads = [torch.empty_like(w) for w in big]
    b.gw = [list(g.split(op.widths)) for g in grads]
    op.backward(torch.stack(b.dy), torch.stack(b.x), b.wg, b.wu, b.wd, b.gate, b.up, b.hidden2, b.dg, b.du, dx, *b.gw)
    b.dx = list(dx)
    b.check_backward()


@pytest.mark.parametrize("T", [3, 140])
def test_many_ranks(ops, T):
    """More ranks than one launch takes, some without columns."""
    both_ways(ops.FeedForward(19, 72, 560, "f16", "gelu", "f32"), f.Block(33, 19, T, 72, 560, "f16", "gelu", grad_dtype="f32"))


def test_offsets_beyond_32_bits(ops):
    """Rows of the tokens and of the outputs 2^30 elements apart: the fourth begins beyond 2^32 bytes."""
    T, D, F, stride = 4, 64, 256, 2 ** 30 + 64
    b = f.Block(34, 1, T, D, F, keep=0)
    op = ops.FeedForward(1, D, F)
    far = lambda width: torch.empty(3 * stride + width, dtype=b.dt, device="cuda").as_strided((T, width), (stride, 1))   # noqa: E731
    x, hidden, out = far(D), far(F), far(D)
    x.copy_(b.x[0])
    op.forward([x], b.wg, b.wu, b.wd, [hidden], [out])
    b.hidden, b.parts = [hidden], [out]
    b.check_forward()


def test_two_host_threads(ops):
    """A handle and a stream for each of two host threads."""
    blocks = [f.Block(35, 2, 300, 136, 900), f.Block(36, 3, 40, 264, 500)]
    handles = [ops.FeedForward(b.R, b.D, b.F) for b in blocks]
    torch.cuda.synchronize()
    failures = []

    def work(op, b):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                b.forward(op)
                for _ in range(200):
                    op.forward(b.x, b.wg, b.wu, b.wd, b.hidden, b.parts, b.gate, b.up, b.scales[0], b.scales[1])
                b.backward(op)
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(handles, blocks)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
    for b in blocks:
        b.check_forward()
        b.check_backward()


def test_the_same_tensor_twice(ops):
    """One tensor as two ranks' weights and as every rank's tokens."""
    R, T, D, F = 2, 60, 72, 256
    b = f.Block(37, R, T, D, F)
    for ws in (b.wg, b.wu, b.wd):
        ws[1] = ws[0]
    b.x = [b.x[0]] * R
    b.dy = [b.dy[0]] * R
    op = ops.FeedForward(R, D, F)
    both_ways(op, b)
    assert torch.equal(b.parts[0], b.parts[1]) and torch.equal(b.gw[0][0], b.gw[0][1])


def test_long_sums(ops):
    """Ten thousand columns against a rank's hundred, and the other way about."""
    both_ways(ops.FeedForward(2, 10000, 200, grad_dtype="f32"), f.Block(38, 2, 37, 10000, 200, grad_dtype="f32"))
    both_ways(ops.FeedForward(1, 72, 20011), f.Block(39, 1, 130, 72, 20011))


def test_refusals_at_the_c_boundary(ops):
    """What only a C caller can ask for."""
    lib = ops._lib

    class ForwardArgs(ctypes.Structure):   # ra_ffn_forward_args
        _fields_ = [(n, ctypes.c_int if n in ("xs", "keep_bits") else
                     ctypes.c_size_t if n in ("rows", "x_stride", "out_stride") else ctypes.c_void_p) for n in
                    ("rows x x_stride xs w_gate w_gate_strides w_up w_up_strides w_down w_down_strides hidden "
                     "hidden_strides out out_stride keep_bits gate gate_strides up up_strides gate_scales up_scales").split()]

    h = ctypes.c_void_p()
    assert lib.ra_ffn_create(2, 64, 256, 1, 0, 1, ctypes.byref(h)) == 0

    def call(**kw):
        args = ForwardArgs(**{**dict(rows=4, xs=1), **kw})
        return lib.ra_ffn_forward(h, ctypes.addressof(args), None)

    assert call(rows=0) == 0
    for bad in (dict(rows=2 ** 27 + 1), dict(xs=3), dict(xs=0), dict(keep_bits=4), dict(), dict(rows=2 ** 63)):
        assert call(**bad) == 1
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    host = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((128, 64), dtype=torch.bfloat16, device="cuda")
    hid, out = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda"), torch.full((2, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    held = []

    def array(kind, values):
        held.append((kind * len(values))(*values))
        return ctypes.addressof(held[-1])

    arr, sizes = (lambda *v: array(ctypes.c_void_p, v)), (lambda *v: array(ctypes.c_size_t, v))
    ok = dict(x=arr(x.data_ptr()), x_stride=64, w_gate=arr(w.data_ptr(), w.data_ptr()), w_gate_strides=sizes(64, 64),
              out=arr(out[0].data_ptr(), out[1].data_ptr()), out_stride=64, hidden=arr(hid[0].data_ptr(), hid[1].data_ptr()),
              hidden_strides=sizes(128, 128))
    ok.update(w_up=ok["w_gate"], w_up_strides=ok["w_gate_strides"], w_down=ok["w_gate"], w_down_strides=ok["w_gate_strides"])
    for bad in (dict(x=arr(host.data_ptr())), dict(x_stride=63), dict(hidden=arr(hid[0].data_ptr(), 0)),
                dict(hidden=arr(hid[0].data_ptr(), hid[0].data_ptr())), dict(w_up=None), dict(out=arr(x.data_ptr(), out[1].data_ptr())),
                dict(x=arr(x.data_ptr() + 1)), dict(keep_bits=8), dict(hidden_strides=sizes(128, 2 ** 50))):
        assert call(**{**ok, **bad}) == 1
        assert lib.ra_last_error()
    torch.cuda.synchronize()
    assert (out == 9).all()
    assert call(**ok) == 0
    torch.cuda.synchronize()
    assert (out == 0).all()
    assert lib.ra_ffn_set_option(h, 4, 2) == 1 and lib.ra_ffn_set_option(h, 1, 1) == 1 and lib.ra_ffn_set_option(h, 4, 0) == 0
    assert lib.ra_ffn_destroy(h) == 0
