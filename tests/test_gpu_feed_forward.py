"""FeedForward against its definitions in 64 bits, product by product: each is
checked from what the call itself wrote for the one before it.

Tolerances are derived, not fitted.  U is the unit roundoff of an output's type,
E that of binary32.  A sum of n products in binary32 loses at most n E of the
sum of their magnitudes where every addition is rounded, and 2 n E where the
tensor cores cut instead; an activation's slope is below 1.13, and it, its
derivative and the products after it lose 16 E of the magnitudes, times what the
rounding of the exponent adds: e^-a, of an exponent of |a| rounded by E twice, loses 2 E |a|
(and no more than its value where it underflows), e^(-a^2/2) so E a^2.  Every
output is rounded once, by U."""

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E = 2.0 ** -24
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -25}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SENTINEL = 7.0


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_gb300 import build
    build.build()
    from ring_allreduce_gb300 import operators
    return operators


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def close(got, want, loss, dtype, what):
    """|got - want| within one rounding of the type and `loss`."""
    want = want.double()
    err = (got.double() - want).abs()
    tol = U[dtype] * (want.abs() + loss) * 1.0001 + loss + TINY[dtype]
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {(err / tol).max().item():.2f} x"


def act64(a, kind):
    return a * torch.sigmoid(a) if kind == "silu" else a * torch.special.ndtr(a)


def slope64(a, kind):
    if kind == "silu":
        p = torch.sigmoid(a)
        return p * (1 + a * (1 - p))
    return torch.special.ndtr(a) + a * torch.exp(-a * a / 2) * 0.3989422804014327


def grow(a, kind):
    """What the exponent's size makes of a rounding; an exponential below binary32's range loses what it has."""
    return 1 + (a.abs().clamp(max=90) if kind == "silu" else (a * a).clamp(max=180))


class Guarded:
    """A [rows, width] view whose surroundings hold a sentinel: `pad` more columns, a row before and after."""

    def __init__(self, rows, width, dtype, pad, lead):
        self.big = torch.full((rows + 2, lead + width + pad), SENTINEL, device="cuda").to(dtype)
        self.at = (lead, width)
        self.view = self.big[1:-1, lead:lead + width]

    def intact(self):
        whole = self.big.float() == SENTINEL
        whole[1:-1, self.at[0]:sum(self.at)] = True
        return bool(whole.all())


class Block:
    """One block's tensors.  `off` elements before every row: 0 and padded rows keep the 16-byte grid, 1 leaves it."""

    def __init__(self, seed, R, T, D, F, dtype="bf16", act="silu", keep=8, copies=1, off=0, grad_dtype=None, sigma=1.0):
        self.g = gen(seed)
        self.R, self.T, self.D, self.F, self.dtype, self.act, self.keep = R, T, D, F, dtype, act, keep
        self.grad_dtype = grad_dtype or dtype
        self.dt, self.off, self.guards = TORCH[dtype], off, []
        C = -(-F // R)
        self.widths = [max(0, min((r + 1) * C, F) - r * C) for r in range(R)]
        self.x = [self.fill(T, D, sigma)] * copies if copies == 1 else []
        if copies > 1:
            first = self.fill(T, D, sigma)
            for _ in range(R):
                t = self.place(T, D, self.dt)
                t.copy_(first)
                self.x.append(t)
        self.wg, self.wu = ([self.fill(n, D, D ** -0.5) for n in self.widths] for _ in range(2))
        self.wd = [self.fill(n, D, F ** -0.5) for n in self.widths]
        self.dy = [self.fill(T, D, 1.0)]

    def place(self, rows, width, dtype):
        pad = 0 if self.off else -width % 16 + 16
        t = Guarded(rows, width, dtype, pad + self.off, self.off)
        self.guards.append(t)
        return t.view

    def fill(self, rows, width, sigma):
        t = self.place(rows, width, self.dt)
        t.copy_(torch.randn((rows, width), generator=self.g, device="cuda") * sigma)
        return t

    def forward(self, op):
        T, D = self.T, self.D
        self.hidden = [self.place(T, n, self.dt) for n in self.widths]
        # out rows have one stride
        self.parts = [self.place(T, D, self.dt) for _ in range(self.R)]
        kw = {}
        if self.keep:
            kdt = torch.int8 if self.keep == 8 else self.dt
            self.gate, self.up = ([self.place(T, n, kdt) for n in self.widths] for _ in range(2))
            kw = dict(gate=self.gate, up=self.up)
            if self.keep == 8:
                self.scales = [[torch.full((T, -(-n // 128)), SENTINEL, device="cuda") for n in self.widths]
                               for _ in range(2)]
                kw.update(gate_scales=self.scales[0], up_scales=self.scales[1])
        op.forward(self.x, self.wg, self.wu, self.wd, self.hidden, self.parts, **kw)

    def kept(self, r):
        """What backward reads of a and b, in 64 bits."""
        got = []
        for k, t in enumerate((self.gate[r], self.up[r])):
            v = t.double()
            if self.keep == 8:
                v = v * self.scales[k][r].double().repeat_interleave(128, 1)[:, :t.shape[1]]
            got.append(v)
        return got

    def check_forward(self):
        for r, n in enumerate(self.widths):
            x = self.x[r % len(self.x)].double()
            wg, wu, wd = self.wg[r].double(), self.wu[r].double(), self.wd[r].double()
            a, b = x @ wg.T, x @ wu.T
            loss = 2 * (self.D + 16) * E
            da, db = loss * (x.abs() @ wg.abs().T), loss * (x.abs() @ wu.abs().T)
            h = act64(a, self.act) * b
            mag = (act64(a, self.act).abs() + 1.13 * da) * (b.abs() + db)
            close(self.hidden[r], h, 1.13 * da * (b.abs() + db) + act64(a, self.act).abs() * db +
                  16 * E * grow(a, self.act) * mag, self.dtype, f"hidden[{r}]")
            h = self.hidden[r].double()
            close(self.parts[r], h @ wd, 2 * (n + 16) * E * (h.abs() @ wd.abs()), self.dtype, f"parts[{r}]")
            if self.keep == 16:
                close(self.gate[r], a, da, self.dtype, f"gate[{r}]")
                close(self.up[r], b, db, self.dtype, f"up[{r}]")
            elif self.keep == 8 and n:
                for k, (v, d) in enumerate(((a, da), (b, db))):
                    pad = torch.nn.functional.pad
                    groups = -(-n // 128)
                    most = pad(v, (0, groups * 128 - n)).view(self.T, groups, 128).abs().amax(2)
                    worst = pad(d, (0, groups * 128 - n)).view(self.T, groups, 128).amax(2)
                    s = self.scales[k][r].double()
                    assert ((s - most / 127).abs() <= worst / 127 + 2 * E * most / 127).all()
                    got = self.kept(r)[k]
                    # half a step of the scale, and what the sum and the product with 127 / most lose
                    tol = (0.5 * s + 4 * E * most).repeat_interleave(128, 1)[:, :n] + 2 * d
                    assert ((got - v).abs() <= tol).all(), f"kept {k}, rank {r}"
                    assert (self.gate[r] if k == 0 else self.up[r]).abs().max() <= 127
        assert all(t.intact() for t in self.guards)

    def backward(self, op, in_place=False, skip=()):
        T, D = self.T, self.D
        self.hidden2 = [self.place(T, n, self.dt) for n in self.widths]
        self.before = [self.kept(r) for r in range(self.R)]
        if in_place:
            self.dg, self.du = self.gate, self.up
        else:
            self.dg, self.du = ([self.place(T, n, self.dt) for n in self.widths] for _ in range(2))
        self.dx = [self.place(T, D, self.dt) for _ in range(self.R)]
        gdt = TORCH[self.grad_dtype]
        self.gw = [[self.place(n, D, gdt) for n in self.widths] for _ in range(3)]
        scales = dict(gate_scales=self.scales[0], up_scales=self.scales[1]) if self.keep == 8 else {}
        wanted = dict(grad_xs=self.dx, grad_w_gate=self.gw[0], grad_w_up=self.gw[1], grad_w_down=self.gw[2])
        op.backward(self.dy, self.x, self.wg, self.wu, self.wd, self.gate, self.up, self.hidden2, self.dg, self.du,
                    **{k: v for k, v in wanted.items() if k not in skip}, **scales)

    def check_backward(self, skip=()):
        dy = self.dy[0].double()
        for r, n in enumerate(self.widths):
            x = self.x[r % len(self.x)].double()
            wg, wu, wd = self.wg[r].double(), self.wu[r].double(), self.wd[r].double()
            a, b = self.before[r]
            dh, loss = dy @ wd.T, 2 * (self.D + 16) * E * (dy.abs() @ wd.abs().T)
            act, slope = act64(a, self.act), slope64(a, self.act)
            # 1 - p and the sums in the slope are of numbers up to 1 + |a|
            lost = 16 * E * (1 + a.abs()) * grow(a, self.act)
            close(self.hidden2[r], act * b, 16 * E * grow(a, self.act) * (act * b).abs(), self.dtype, f"hidden[{r}]")
            close(self.dg[r], dh * b * slope, (loss * slope.abs() + (dh.abs() + loss) * lost) * b.abs(), self.dtype,
                  f"grad_gate[{r}]")
            close(self.du[r], dh * act, (loss + 16 * E * grow(a, self.act) * (dh.abs() + loss)) * act.abs(),
                  self.dtype, f"grad_up[{r}]")
            dg, du, h = self.dg[r].double(), self.du[r].double(), self.hidden2[r].double()
            if "grad_xs" not in skip:
                close(self.dx[r], dg @ wg + du @ wu,
                      2 * (2 * n + 16) * E * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()), self.dtype, f"grad_xs[{r}]")
            for k, (left, right) in enumerate(((dg, x), (du, x), (h, dy))):
                if ("grad_w_gate", "grad_w_up", "grad_w_down")[k] not in skip:
                    close(self.gw[k][r], left.T @ right, 2 * (self.T + 16) * E * (left.abs().T @ right.abs()),
                          self.grad_dtype, f"grad_w[{k}][{r}]")
        assert all(t.intact() for t in self.guards)


SHAPES = [   # R, T, D, F: one row to many, widths that end inside a tile, ranks without columns
    (1, 1, 8, 1), (1, 1, 64, 128), (2, 3, 72, 130), (4, 5, 16, 9), (3, 16, 200, 385), (2, 17, 136, 1000),
    (1, 64, 520, 300), (2, 65, 256, 513), (1, 128, 512, 256), (3, 129, 328, 777), (2, 257, 1032, 640),
    (5, 300, 136, 1031), (1, 700, 264, 2050), (32, 33, 128, 1500)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("off", [0, 1])
def test_forward_and_backward(ops, shape, off):
    """Kept in 8 bits, bf16, on the 16-byte grid and off it."""
    b = Block(1, *shape, off=off)
    op = ops.FeedForward(*[shape[i] for i in (0, 2, 3)])
    assert op.widths == b.widths
    b.forward(op)
    b.check_forward()
    b.backward(op)
    b.check_backward()


@pytest.mark.parametrize("shape", SHAPES[2::3], ids=str)
@pytest.mark.parametrize("dtype,act,keep,copies,grad_dtype", [
    ("f16", "gelu", 8, 2, "f32"), ("bf16", "gelu", 16, 2, "f32"), ("f16", "silu", 16, 1, "f16"), ("bf16", "gelu", 8, 1, "bf16")])
def test_types_activations_and_kept_forms(ops, shape, dtype, act, keep, copies, grad_dtype):
    b = Block(2, *shape, dtype, act, keep, copies, grad_dtype=grad_dtype)
    op = ops.FeedForward(*[shape[i] for i in (0, 2, 3)], dtype, activation=act, grad_dtype=grad_dtype)
    b.forward(op)
    b.check_forward()
    b.backward(op)
    b.check_backward()


@pytest.mark.parametrize("T", [1, 2, 15, 16, 31, 32, 33, 48, 63, 64, 90, 127, 128, 200, 256, 300])
@pytest.mark.parametrize("R,D,F,dtype,act", [(2, 256, 1024, "bf16", "silu"), (3, 1000, 700, "f16", "gelu"),
                                             (1, 2048, 4096, "bf16", "gelu")])
def test_forward_of_few_tokens(ops, T, R, D, F, dtype, act):
    """Nothing kept, as in serving."""
    b = Block(3, R, T, D, F, dtype, act, keep=0, copies=2)
    op = ops.FeedForward(R, D, F, dtype, activation=act)
    b.forward(op)
    b.check_forward()


def test_large(ops):
    """Many tiles, every CTA with several of them."""
    b = Block(4, 3, 2311, 1544, 6001)
    op = ops.FeedForward(3, 1544, 6001)
    b.forward(op)
    b.check_forward()
    b.backward(op)
    b.check_backward()
    from ring_allreduce_gb300.binding import Status
    assert op.device_status()[0] == Status.OK


@pytest.mark.parametrize("skip", [("grad_xs",), ("grad_w_gate",), ("grad_w_up", "grad_w_down"),
                                  ("grad_w_gate", "grad_w_up", "grad_w_down")])
def test_gradients_that_are_not_wanted(ops, skip):
    b = Block(5, 2, 70, 136, 300)
    op = ops.FeedForward(2, 136, 300)
    b.forward(op)
    b.backward(op, skip=skip)
    b.check_backward(skip)
    for k, name in enumerate(("grad_w_gate", "grad_w_up", "grad_w_down")):
        if name in skip:
            assert all((t == SENTINEL).all() for t in b.gw[k])


def test_gradients_in_place_of_what_was_kept(ops):
    b = Block(6, 2, 150, 72, 270, keep=16)
    op = ops.FeedForward(2, 72, 270)
    b.forward(op)
    b.check_forward()
    b.backward(op, in_place=True)
    b.check_backward()


def test_gradients_against_differences(ops):
    """The gradients of sum(parts . dy) along random directions, from the
    definition's differences in 64 bits.  What the call works with is rounded to
    f16 (kept a, b, hidden, the gradients of a and b: U each), so each
    directional derivative is off by at most 6 U of the sum of its terms' magnitudes."""
    R, T, D, F, dtype = 2, 40, 64, 200, "f16"
    b = Block(7, R, T, D, F, dtype, "gelu", keep=16, grad_dtype="f32")
    op = ops.FeedForward(R, D, F, dtype, activation="gelu", grad_dtype="f32")
    b.forward(op)
    b.backward(op)
    x, dy = b.x[0].double(), b.dy[0].double()

    def value(x, w):
        return sum(((act64(x @ w[0][r].T, "gelu") * (x @ w[1][r].T)) @ w[2][r] * dy).sum() for r in range(R))

    w = [[t.double() for t in ws] for ws in (b.wg, b.wu, b.wd)]
    step = 1e-5
    for k in range(3):
        v = [torch.randn(t.shape, generator=b.g, device="cuda", dtype=torch.float64) for t in w[k]]
        moved = [[[t + s * step * d if i == k else t for t, d in zip(w[i], v)] for i in range(3)] for s in (1, -1)]
        want = (value(x, moved[0]) - value(x, moved[1])) / (2 * step)
        got = sum((g.double() * d).sum() for g, d in zip(b.gw[k], v))
        left = (b.dg, b.du, b.hidden2)[k]
        right = dy if k == 2 else x
        mag = sum((p.double().abs().T @ right.abs() * d.abs()).sum() for p, d in zip(left, v))
        assert (got - want).abs() <= 6 * U[dtype] * mag
    v = torch.randn(x.shape, generator=b.g, device="cuda", dtype=torch.float64)
    want = (value(x + step * v, w) - value(x - step * v, w)) / (2 * step)
    got = sum((g.double() * v).sum() for g in b.dx)
    mag = sum(((p.double().abs() @ m.abs() + q.double().abs() @ n.abs()) * v.abs()).sum()
              for p, q, m, n in zip(b.dg, b.du, *w[:2]))
    assert (got - want).abs() <= 6 * U[dtype] * mag


def test_rows_do_not_meet(ops):
    """An infinity in one token's row leaves every other row's outputs and kept codes as they were."""
    R, T, D, F = 2, 131, 264, 520
    op = ops.FeedForward(R, D, F)
    clean, dirty = Block(8, R, T, D, F), Block(8, R, T, D, F)
    dirty.x[0][77, 5] = float("inf")
    for b in (clean, dirty):
        b.forward(op)
    rows = torch.arange(T, device="cuda") != 77
    for r in range(R):
        for name in ("hidden", "parts", "gate", "up"):
            assert torch.equal(getattr(clean, name)[r][rows], getattr(dirty, name)[r][rows]), name
        for k in range(2):
            assert torch.equal(clean.scales[k][r][rows], dirty.scales[k][r][rows])
            assert dirty.scales[k][r][77].isnan().all()
    assert not any(torch.isfinite(dirty.parts[r][77]).any() for r in range(R))
    # and in the gradients of the rows
    for b in (clean, dirty):
        b.backward(op, skip=("grad_w_gate", "grad_w_up", "grad_w_down"))
    for r in range(R):
        assert torch.equal(clean.dx[r][rows], dirty.dx[r][rows]) and torch.equal(clean.dg[r][rows], dirty.dg[r][rows])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_activations(ops, act):
    """Gates far from zero: no NaN where the limit is a number."""
    R, T, D, F = 1, 4, 8, 160
    b = Block(9, R, T, D, F, act=act, keep=16)
    b.x[0].copy_(torch.tensor([[-3e4], [3e4], [-60.0], [0.0]], device="cuda").expand(T, D))
    b.wg[0].fill_(0.5)
    op = ops.FeedForward(R, D, F, activation=act)
    b.forward(op)
    b.check_forward()
    b.backward(op)
    b.check_backward()
    assert all(torch.isfinite(t).all() for t in b.hidden + b.parts + b.dx + b.gw[0])


def test_no_rows(ops):
    R, D, F = 2, 72, 300
    b = Block(10, R, 0, D, F)
    op = ops.FeedForward(R, D, F)
    b.forward(op)
    b.backward(op)
    assert all((t == 0).all() for k in range(3) for t in b.gw[k])
    assert all(t.intact() for t in b.guards)


def test_results_are_the_same_every_time(ops):
    got = []
    for _ in range(2):
        b = Block(11, 3, 333, 520, 1111)
        op = ops.FeedForward(3, 520, 1111)
        for _ in range(2):
            b.forward(op)
            b.backward(op)
            got.append([t.clone() for t in b.parts + b.dx + b.gw[0] + b.gw[1] + b.gw[2]])
    for other in got[1:]:
        assert all(torch.equal(p, q) for p, q in zip(got[0], other))


@pytest.mark.parametrize("T", [1, 40, 400])
def test_captured_and_replayed(ops, T):
    """A training step in a CUDA graph, replayed on new inputs, on another stream, after the handle is closed."""
    R, D, F = 2, 136, 600
    b, want = Block(12, R, T, D, F), Block(13, R, T, D, F)
    op = ops.FeedForward(R, D, F)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(op)
        b.backward(op)
    for mine, theirs in ((b.x, want.x), (b.wg, want.wg), (b.wu, want.wu), (b.wd, want.wd), (b.dy, want.dy)):
        for t, s in zip(mine, theirs):
            t.copy_(s)
    want.forward(op)
    want.backward(op)
    op.close()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            graph.replay()
    side.synchronize()
    for name in ("parts", "dx"):
        assert all(torch.equal(p, q) for p, q in zip(getattr(b, name), getattr(want, name)))
    assert all(torch.equal(p, q) for k in range(3) for p, q in zip(b.gw[k], want.gw[k]))
    with pytest.raises(ValueError):
        op.forward(b.x, b.wg, b.wu, b.wd, b.hidden, b.parts)


def test_calls_on_two_streams_at_once(ops):
    """Calls of one handle may overlap: there is no workspace."""
    R, D, F = 2, 264, 1030
    op = ops.FeedForward(R, D, F)
    blocks = [Block(20 + i, R, 500, D, F) for i in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        for s, b in zip(streams, blocks):
            with torch.cuda.stream(s):
                b.forward(op)
                b.backward(op)
    torch.cuda.synchronize()
    for b in blocks:
        b.check_forward()
        b.check_backward()


def test_stream_of_the_caller(ops):
    R, D, F, T = 2, 72, 200, 20
    b = Block(14, R, T, D, F, keep=0)
    op = ops.FeedForward(R, D, F)
    b.forward(op)
    want = [t.clone() for t in b.parts]
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for t in b.parts:
            t.zero_()
        torch.cuda.synchronize()
        op.forward((t for t in b.x), (t for t in b.wg), b.wu, b.wd, b.hidden, b.parts, stream=stream)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, b.parts))


def test_refusals(ops):
    from ring_allreduce_gb300 import RAError, Status
    R, D, F, T = 2, 72, 200, 20
    b = Block(15, R, T, D, F)
    op = ops.FeedForward(R, D, F)
    b.forward(op)
    ok = (b.x, b.wg, b.wu, b.wd, b.hidden, b.parts)
    for k, bad in ((0, b.parts[:0]), (0, [b.x[0].float()]), (0, [b.x[0].cpu()]), (1, b.wg[:1]), (1, [b.wg[0], None]),
                   (2, [b.wu[0].T, b.wu[1]]), (4, b.parts), (4, None), (5, b.parts[:1]), (5, 3)):
        with pytest.raises(ValueError):
            op.forward(*ok[:k], bad, *ok[k + 1:])
    for kw in (dict(gate=b.gate), dict(gate=b.gate, up=b.up), dict(gate_scales=b.scales[0]),
               dict(gate=b.gate, up=b.up, gate_scales=b.scales[1]),
               dict(gate=b.hidden, up=b.hidden, gate_scales=b.scales[0], up_scales=b.scales[1]),
               dict(gate=b.gate, up=b.hidden, gate_scales=b.scales[0], up_scales=b.scales[1])):
        with pytest.raises(ValueError):
            op.forward(*ok, **kw)
    for kw, args in ((dict(gate=b.hidden, up=b.hidden), ok), (dict(), ok[:5] + ([b.parts[0], b.parts[0]],)),
                     (dict(), ok[:4] + (b.hidden, [b.x[0], b.parts[1]]))):
        with pytest.raises(RAError) as err:
            op.forward(*args, **kw)
        assert err.value.status == Status.ERR_INVALID
    with pytest.raises(RAError) as err:   # hidden is where grad_w_down comes from
        op.backward(b.dy, b.x, b.wg, b.wu, b.wd, b.gate, b.up, None, *[op.rows(T) for _ in range(2)],
                    grad_w_down=[torch.empty_like(w) for w in b.wd], gate_scales=b.scales[0], up_scales=b.scales[1])
    assert err.value.status == Status.ERR_INVALID
    with pytest.raises(ValueError):
        op.backward(b.dy, b.x, b.wg, b.wu, b.wd, None, None, None, op.rows(T), op.rows(T))
    # without hidden, x and the projections' weights where they are not needed
    op.backward(b.dy, None, None, None, b.wd, b.gate, b.up, None, op.rows(T), op.rows(T), gate_scales=b.scales[0],
                up_scales=b.scales[1])
    b.check_forward()
