"""The model operators (BlockNorm, VocabHead) against their definitions in 64
bits.

Tolerances are derived, not fitted.  U is the unit roundoff of an output's type
(half a unit in the last place, relative), E that of binary32.  An output is
rounded once, so its error is at most U |value| plus what binary32 loses on the
way: every quantity is a sum or product of terms whose magnitudes are summed
alongside (each subtraction as an addition of magnitudes); n additions in a row
lose at most n E of that sum.  A row's sum runs over at most 16 columns a
thread, ten halvings across a block and R ranks; norm factors, products and
square roots add a few E each, which 64 covers throughout."""

import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E = 2.0 ** -24
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # 2^-p for p significand bits
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -25}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS, SCALE = 1e-5, 0.75
NOTHING_LEFT = -1e30   # rows with a smaller lse are masked everywhere: no gradient


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


def randn(g, *shape, dtype="f32", sigma=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma + mean).to(TORCH[dtype])


def close(got, want, loss, dtype, what):
    """|got - want| within one rounding of the type and `loss` (a tensor)."""
    want = want.double()
    err = (got.double() - want).abs()
    tol = U[dtype] * want.abs() * 1.0001 + loss + TINY[dtype]
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {(err / tol).max().item():.2f} x"


# ---------------------------------------------------------------- block end

def padded(t, pad):
    """The same rows in a wider buffer (a stride that is not the width)."""
    if not pad:
        return t
    big = torch.full((*t.shape[:-1], t.shape[-1] + pad), 7.0, dtype=t.dtype, device=t.device)
    big[..., :t.shape[-1]] = t
    return big[..., :t.shape[-1]]


class Norm:
    """One block end: inputs, 64-bit forward and backward with magnitudes."""

    def __init__(self, seed, R, T, D, dtype, rdtype, pdtype, post, G, pad=0):
        g = gen(seed)
        self.R, self.T, self.D, self.dtype, self.rdtype, self.G = R, T, D, dtype, rdtype, G
        self.parts = [padded(randn(g, T, D, dtype=dtype), pad) for _ in range(R)]
        self.residual = padded(randn(g, T, D, dtype=rdtype, sigma=2.0), pad)
        self.weight = randn(g, D, dtype=pdtype, sigma=0.2, mean=1.0)
        self.post = randn(g, D, dtype=pdtype, sigma=0.2, mean=1.0) if post else None
        self.gate = randn(g, G, D, dtype=pdtype, sigma=0.5) if G else None
        self.grad_z = [padded(randn(g, T, D, dtype=dtype), pad) for _ in range(R)]
        self.grad_h = padded(randn(g, T, D, dtype=rdtype), pad)

    def gate64(self):
        if self.gate is None:
            return torch.ones((), dtype=torch.float64, device="cuda")
        return self.gate.double().repeat_interleave(self.T // self.G, 0)

    def forward64(self, parts=None, residual=None, weight=None, post=None, gate=None):
        S = (sum(p.double() for p in self.parts) if parts is None else parts)
        h = self.residual.double() if residual is None else residual
        w = self.weight.double() if weight is None else weight
        r1 = torch.zeros(self.T, dtype=torch.float64, device="cuda")
        y = S
        if self.post is not None:
            r1 = (S.square().mean(1) + EPS).rsqrt()
            y = S * r1[:, None] * (self.post.double() if post is None else post)
        g = self.gate64() if gate is None else gate
        h2 = h + SCALE * g * y
        r2 = (h2.square().mean(1) + EPS).rsqrt()
        return S, r1, h2, r2, h2 * r2[:, None] * w

    def check_forward(self, z, h2, total, rstd):
        S, r1, want_h, r2, want_z = self.forward64()
        mag = sum(p.double().abs() for p in self.parts)
        # the norm factor moves with the sum's own loss, relative to its norm
        grow = max(1.0, (mag.norm() / S.norm()).item())
        n = (self.R + 64) * E * grow
        close(total, S, self.R * E * mag, self.dtype, "total")
        y = mag
        if self.post is not None:
            y = mag * r1[:, None] * self.post.double().abs()
            close(rstd[0], r1, n * r1, "f32", "rstd[0]")
        else:
            assert (rstd[0] == 0).all()
        hmag = self.residual.double().abs() + SCALE * self.gate64().abs() * y
        grow2 = max(1.0, (hmag.norm(dim=1) / want_h.norm(dim=1)).max().item())
        close(h2, want_h, n * hmag, self.rdtype, "residual_out")
        close(rstd[1], r2, 2 * n * grow2 * r2, "f32", "rstd[1]")
        for k, q in enumerate(z):
            close(q, want_z, 3 * n * grow2 * hmag * r2[:, None] * self.weight.double().abs(), self.dtype, f"out[{k}]")

    def backward64(self, total, h2, rstd, grads):
        """From what the kernel is given; (values, magnitudes) of every output."""
        r1, r2 = rstd[0].double()[:, None], rstd[1].double()[:, None]
        dz = sum(p.double() for p in grads)
        mz = sum(p.double().abs() for p in grads)
        x2, w = h2.double() * r2, self.weight.double()
        c2 = (w * dz * x2).mean(1, keepdim=True)
        m2 = (w.abs() * mz * x2.abs()).mean(1, keepdim=True)
        e = self.grad_h.double() + r2 * (w * dz - x2 * c2)
        me = self.grad_h.double().abs() + r2 * (w.abs() * mz + x2.abs() * m2)
        g = self.gate64()
        dy, my = SCALE * g * e, SCALE * g.abs() * me
        S = total.double()
        out = dict(grad_residual=(e, me), grad_weight=((dz * x2).sum(0), (mz * x2.abs()).sum(0)))
        y, ds, ms = S, dy, my
        if self.post is not None:
            p = self.post.double()
            x1 = S * r1
            y = x1 * p
            c1 = (p * dy * x1).mean(1, keepdim=True)
            m1 = (p.abs() * my * x1.abs()).mean(1, keepdim=True)
            ds, ms = r1 * (p * dy - x1 * c1), r1 * (p.abs() * my + x1.abs() * m1)
            out["grad_post_weight"] = ((dy * x1).sum(0), (my * x1.abs()).sum(0))
        out["grad_in"] = (ds, ms)
        if self.gate is not None:
            out["grad_gate"] = ((SCALE * y * e).view(self.G, -1, self.D).sum(1),
                                (SCALE * y.abs() * me).view(self.G, -1, self.D).sum(1))
        return out

    def run(self, ops, outs, stream=None, pad=0):
        z = [padded(torch.full((self.T, self.D), 9.0, dtype=TORCH[self.dtype], device="cuda"), pad)
             for _ in range(outs)]
        h2 = padded(torch.full((self.T, self.D), 9.0, dtype=TORCH[self.rdtype], device="cuda"), pad)
        total = padded(torch.full((self.T, self.D), 9.0, dtype=TORCH[self.dtype], device="cuda"), pad)
        rstd = torch.full((2, self.T), 9.0, device="cuda")
        pd = {v: k for k, v in TORCH.items()}[self.weight.dtype]
        op = ops.BlockNorm(self.R, self.D, self.dtype, self.rdtype, pd, eps=EPS, scale=SCALE)
        op.forward(self.parts, self.residual, self.weight, z, h2, post_weight=self.post, gate=self.gate, total=total,
                   rstd=rstd, stream=stream)
        return op, z, h2, total, rstd

    def run_backward(self, op, h2, total, rstd, grads, outs, pad=0):
        gin = [padded(torch.full((self.T, self.D), 9.0, dtype=TORCH[self.dtype], device="cuda"), pad)
               for _ in range(outs)]
        gh = padded(torch.full((self.T, self.D), 9.0, dtype=TORCH[self.rdtype], device="cuda"), pad)
        f32 = dict(dtype=torch.float32, device="cuda")
        gw = torch.full((self.D,), 9.0, **f32)
        gp = torch.full((self.D,), 9.0, **f32) if self.post is not None else None
        gg = torch.full((self.G, self.D), 9.0, **f32) if self.G else None
        op.backward(grads, self.grad_h, h2, rstd, self.weight, gin, gh, gw, post_weight=self.post, gate=self.gate,
                    total=total, grad_post_weight=gp, grad_gate=gg)
        return gin, gh, gw, gp, gg

    def check_backward(self, got, total, h2, rstd, grads):
        gin, gh, gw, gp, gg = got
        want = self.backward64(total, h2, rstd, grads)
        n = (self.R + 64) * E
        close(gh, want["grad_residual"][0], n * want["grad_residual"][1], self.rdtype, "grad_residual")
        for k, q in enumerate(gin):
            close(q, want["grad_in"][0], 2 * n * want["grad_in"][1], self.dtype, f"grad_in[{k}]")
        # columns: T additions
        m = (self.R + 64 + self.T) * E
        close(gw, want["grad_weight"][0], m * want["grad_weight"][1], "f32", "grad_weight")
        if gp is not None:
            close(gp, want["grad_post_weight"][0], m * want["grad_post_weight"][1], "f32", "grad_post_weight")
        if gg is not None:
            close(gg, want["grad_gate"][0], m * want["grad_gate"][1], "f32", "grad_gate")


# R, T, D, dtype, residual, params, post norm, gate rows, padding of the rows
NORMS = [
    (1, 1, 1, "f32", "f32", "f32", True, 0, 0),
    (2, 1, 64, "bf16", "bf16", "bf16", True, 1, 0),
    (3, 5, 7, "f16", "f32", "f32", True, 5, 0),
    (8, 33, 256, "bf16", "f32", "f32", False, 0, 0),
    (4, 17, 257, "bf16", "bf16", "f32", True, 17, 0),
    (2, 300, 128, "f32", "f32", "f32", True, 3, 4),
    (5, 12, 1000, "f16", "f16", "f16", False, 4, 8),
    (32, 9, 513, "bf16", "f32", "bf16", True, 3, 3),
    (8, 40, 4096, "bf16", "bf16", "bf16", True, 1, 0),
    (3, 21, 4104, "f16", "f16", "f32", True, 7, 0),
    (2, 700, 2048, "bf16", "f32", "f32", True, 2, 0),
    (7, 6, 8192, "bf16", "bf16", "bf16", True, 2, 0),
    (2, 5, 16384, "bf16", "f32", "f32", True, 5, 0),
    (2, 3, 16384, "f32", "f32", "f32", True, 1, 0),
    (1, 4, 16383, "f32", "f32", "f32", False, 2, 0),
    (2, 4, 12289, "f16", "f16", "f16", True, 0, 0),
    # rows that share a warp
    (3, 1003, 128, "bf16", "f32", "f32", True, 17, 0),
    (4, 77, 40, "f16", "f16", "f16", True, 7, 8),
    (2, 50, 16, "f32", "f32", "f32", False, 0, 0),
    (2, 9, 8, "bf16", "bf16", "f32", True, 3, 8),
    (6, 6000, 72, "bf16", "bf16", "bf16", True, 1, 0),
    (5, 33, 64, "f32", "f32", "f32", True, 33, 4),
]


@pytest.mark.parametrize("spec", NORMS, ids=lambda s: "-".join(map(str, s)))
def test_norm_forward_and_backward(ops, spec):
    c = Norm(11, *spec)
    pad = spec[-1]
    op, z, h2, total, rstd = c.run(ops, c.R if c.R <= 8 else 1, pad=pad)
    c.check_forward(z, h2, total, rstd)
    for grads, outs in ((c.grad_z, 1), (c.grad_z[:1], c.R)):
        c.check_backward(c.run_backward(op, h2, total, rstd, grads, outs, pad), total, h2, rstd, grads)


@pytest.mark.parametrize("T,D,dtype", [(5, 4096, "bf16"), (6, 999, "f32")])
def test_norm_in_place(ops, T, D, dtype):
    c = Norm(3, 2, T, D, dtype, dtype, "f32", True, 1)
    op, z, h2, total, rstd = c.run(ops, 2)
    parts, residual = [p.clone() for p in c.parts], c.residual.clone()
    op.forward(parts, residual, c.weight, parts, residual, post_weight=c.post, gate=c.gate)
    assert all(torch.equal(p, z[0]) for p in parts) and torch.equal(residual, h2)
    gin, gh, gw, gp, gg = c.run_backward(op, h2, total, rstd, c.grad_z, 2)
    g, d = [p.clone() for p in c.grad_z], c.grad_h.clone()
    op.backward(g, d, h2, rstd, c.weight, g, d, post_weight=c.post, gate=c.gate, total=total)
    assert all(torch.equal(p, gin[0]) for p in g) and torch.equal(d, gh)


def test_norm_stacked_and_optional_buffers(ops):
    c = Norm(4, 4, 37, 512, "bf16", "f32", "f32", False, 0)
    op, z, h2, total, rstd = c.run(ops, 1)
    out, res = torch.empty_like(torch.stack(z)), torch.empty_like(h2)
    op.forward(torch.stack(c.parts), c.residual, c.weight, out, res)
    assert torch.equal(out[0], z[0]) and torch.equal(res, h2)
    # no post norm, no gate gradient: total is not needed; no residual gradient: zero
    gin, gh = torch.empty_like(out), torch.empty_like(h2)
    op.backward(torch.stack(c.grad_z), None, h2, rstd, c.weight, gin, gh)
    c.grad_h = torch.zeros_like(c.grad_h)
    want = c.run_backward(op, h2, total, rstd, c.grad_z, 1)
    assert torch.equal(gin[0], want[0][0]) and torch.equal(gh, want[1])


def test_norm_zero_rows_of_values(ops):
    """A row of zeros (a padded token) has the norm of eps alone: all zeros, nothing infinite."""
    c = Norm(5, 2, 4, 640, "bf16", "bf16", "bf16", True, 1)
    for p in c.parts:
        p[2] = 0
    c.residual[2] = 0
    op, z, h2, total, rstd = c.run(ops, 1)
    c.check_forward(z, h2, total, rstd)
    assert (z[0][2] == 0).all()
    c.check_backward(c.run_backward(op, h2, total, rstd, c.grad_z, 1), total, h2, rstd, c.grad_z)


def test_norm_gradient_against_differences(ops):
    """The kernel's gradient along a random direction against central
    differences of the 64-bit forward (step 1e-5: truncation and rounding below
    1e-8 of the slope); binary32 inputs, so the kernel's loss is at most the
    derived one, here 1e-4 of the sum of magnitudes' scale."""
    c = Norm(6, 2, 8, 320, "f32", "f32", "f32", True, 4)
    op, z, h2, total, rstd = c.run(ops, 1)
    gin, gh, gw, gp, gg = c.run_backward(op, h2, total, rstd, c.grad_z, 1)
    g = gen(99)
    dz, dh = sum(p.double() for p in c.grad_z), c.grad_h.double()
    S, h = sum(p.double() for p in c.parts), c.residual.double()

    def value(t, v):
        _, _, h2, _, z = c.forward64(parts=S + t * v["S"], residual=h + t * v["h"], weight=c.weight.double() + t * v["w"],
                                     post=c.post.double() + t * v["p"],
                                     gate=c.gate64() + t * v["g"].repeat_interleave(c.T // c.G, 0))
        return ((z * dz).sum() + (h2 * dh).sum()).item()

    shapes = dict(S=(8, 320), h=(8, 320), w=(320,), p=(320,), g=(4, 320))
    grads = dict(S=gin[0], h=gh, w=gw, p=gp, g=gg)
    for name, shape in shapes.items():
        v = {k: torch.zeros(s, dtype=torch.float64, device="cuda") for k, s in shapes.items()}
        v[name] = torch.randn(shape, generator=g, device="cuda", dtype=torch.float64)
        slope = (value(1e-5, v) - value(-1e-5, v)) / 2e-5
        got = (grads[name].double() * v[name]).sum().item()
        scale = (grads[name].double().abs() * v[name].abs()).sum().item()
        assert abs(got - slope) <= 1e-4 * scale, (name, got, slope, scale)


# --------------------------------------------------------- vocabulary's head

def shards_of(full, R, pad=0, off=0):
    """The ranks' shards; pad: extra columns in each row's stride, off: first element's offset in its buffer."""
    V = full.shape[1]
    C = -(-V // R)
    out = []
    for r in range(R):
        part = full[:, min(r * C, V):min((r + 1) * C, V)]
        T, w = part.shape
        buf = torch.full((off + T * (w + pad) + 16,), 5.0, dtype=full.dtype, device="cuda")
        view = buf[off:off + T * (w + pad)].view(T, w + pad)[:, :w]
        view.copy_(part)
        out.append(view)
    return out


def logits(g, T, V, dtype):
    x = torch.randn((T, V), generator=g, device="cuda") * 2.0
    hot = torch.randint(V, (T, 8), generator=g, device="cuda")
    x.scatter_(1, hot, torch.randn((T, 8), generator=g, device="cuda") + 9.0)
    return x.to(TORCH[dtype]), hot


def mask_rows(x, g):
    """Rows as masks leave them: whole, nothing, one token, the type's lowest value in places or everywhere."""
    T, V = x.shape
    low = torch.finfo(x.dtype).min
    for t in range(T):
        kind = t % 7
        if kind == 1:
            x[t] = -math.inf
        elif kind == 2:
            keep = x[t, t * 31 % V].clone()
            x[t] = -math.inf
            x[t, t * 31 % V] = keep
        elif kind == 3:
            x[t, torch.rand(V, generator=g, device="cuda") < 0.9] = low
        elif kind == 4:
            x[t] = low
        elif kind == 5:
            x[t, torch.rand(V, generator=g, device="cuda") < 0.99] = -math.inf
            x[t, t * 17 % V] = 1.0
    return x


def stats64(x, tau):
    """log p, lse, entropy in 64 bits; rows of nothing but -inf: -inf, -inf, 0.
    (x - max) - log sum, since a row of lowest values, near -3e38, would take the
    logarithm of its sum in, even in 64 bits."""
    x = x.double() / tau
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    total = (x - m).exp().sum(1, keepdim=True).log()
    lse = (m + total)[:, 0]
    logp = torch.where((lse == -math.inf)[:, None], -math.inf, (x - m) - total)
    p = logp.exp()
    return logp, lse, -(torch.where(p > 0, p * logp, 0.0)).sum(1)


def stat_loss(x, tau, V):
    """What binary32 loses in a logarithm of a row's sum: every 2^t is good to
    2^-22 and its exponent's roundings (t 2^-t <= 1: 4 E), at least 128 threads add
    V / 128 and 16 more terms, ten joins; log and lse add their own roundings."""
    top = torch.where(torch.isfinite(x), x, 0).abs().amax(1).double() / tau
    return 2.0 ** -21 + (V / 128 + 64) * E + 0 * top


def same(got, want, tol, what):
    """Equal where infinite or NaN, within tol elsewhere."""
    got, want = got.double(), want.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = ~fin & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), what
    err = (got - want).abs()[fin]
    tol = (tol + 0 * want)[fin]
    assert (err <= tol).all(), f"{what}: worst {(err / tol).max().item():.2f} x"


def top_ids64(x, K):
    """Falling logits, equal ones by column, NaN first."""
    v = x.double() + 0.0
    v = torch.where(torch.isnan(v), math.inf, v)
    nan_first = torch.where(torch.isnan(x), 0, 1)
    order = torch.sort(v, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(nan_first.gather(1, order), dim=1, stable=True).indices)
    return order[:, :K]


# R, T, V, dtype, K, tau, masked, pad, off
HEADS = [
    (1, 1, 1, "f32", 1, 1.0, False, 0, 0),
    (2, 3, 2, "bf16", 2, 1.0, False, 0, 1),
    (32, 9, 66, "f16", 32, 0.5, True, 0, 0),       # shards without columns
    (3, 29, 1000, "bf16", 20, 1.0, True, 0, 0),
    (4, 15, 4096, "f32", 5, 2.0, True, 0, 0),
    (5, 22, 32003, "f16", 32, 0.7, True, 0, 3),
    (8, 4, 131072, "bf16", 20, 1.0, False, 0, 0),
    (8, 1, 131072, "bf16", 32, 1.0, False, 0, 0),
    (1, 8, 50021, "f32", 1, 1.0, True, 3, 1),
    (7, 400, 1537, "bf16", 3, 1.3, True, 5, 0),
    (2, 700, 8192, "bf16", 0, 1.0, False, 8, 0),
    (4, 650, 2050, "bf16", 20, 1.0, True, 0, 0),   # rows enough for a warp or two each
    (1, 615, 300, "f32", 32, 1.0, True, 0, 1),
    (2, 640, 20000, "f16", 5, 0.7, True, 0, 0),
    (3, 700, 9000, "bf16", 32, 1.0, False, 0, 0),
    # many short rows: CTAs of a warp or two
    (2, 700, 503, "f32", 32, 0.7, True, 0, 0),
    (3, 650, 1000, "f16", 20, 1.0, False, 1, 1),
    (4, 620, 4096, "bf16", 32, 1.3, True, 8, 3),
]


@pytest.mark.parametrize("spec", HEADS, ids=lambda s: "-".join(map(str, s)))
def test_logprobs_and_gradient(ops, spec):
    R, T, V, dtype, K, tau, masked, pad, off = spec
    g = gen(21)
    x, hot = logits(g, T, V, dtype)
    if masked:
        mask_rows(x, g)
    sh = shards_of(x, R, pad, off)
    targets = torch.where(torch.rand(T, generator=g, device="cuda") < 0.7, hot[:, 0],
                          torch.randint(V, (T,), generator=g, device="cuda"))
    targets[::5] = -1
    op = ops.VocabHead(R, V, dtype, temperature=tau)
    f32 = dict(dtype=torch.float32, device="cuda")
    lp, lse, H = (torch.full((T,), 9.0, **f32) for _ in range(3))
    ids = torch.full((T, K), -7, dtype=torch.int64, device="cuda") if K else None
    tlp = torch.full((T, K), 9.0, **f32) if K else None
    op.logprobs(sh, targets, lp, lse, H, ids, tlp)

    logp, lse64, H64 = stats64(x, tau)
    loss = stat_loss(x, tau, V)
    size = torch.where(torch.isfinite(lse64), lse64.abs(), 0.0)
    # values near the type's lowest, divided by tau < 1, leave binary32's range: rounded to it
    lse64 = lse64.float().double()
    same(lse, lse64, loss + 4 * E * size, "lse")
    want = torch.where(targets < 0, 0.0, logp.gather(1, targets.clamp(min=0)[:, None])[:, 0]).float().double()
    same(lp, want, loss + 4 * E * torch.where(torch.isfinite(want), want.abs(), 0.0), "logprob")
    same(H, H64, (loss + 4 * E) * (2 + math.log(V)), "entropy")
    if K:
        assert torch.equal(ids, top_ids64(x, K))
        want = logp.gather(1, ids).float().double()
        same(tlp, want, loss[:, None] + 4 * E * torch.where(torch.isfinite(want), want.abs(), 0.0), "top")

    # gradient, from what forward wrote
    glp, gH = randn(g, T), randn(g, T, sigma=0.3)
    grads = [torch.full_like(s, 9.0) for s in shards_of(x, R, pad, off)]
    for with_entropy in (True, False):
        op.logprobs_backward(sh, targets, lse, glp, grads, entropy=H if with_entropy else None,
                             grad_entropy=gH if with_entropy else None)
        check_logprob_gradient(x, tau, lse, H, targets, glp, gH if with_entropy else torch.zeros_like(gH),
                               torch.cat(grads, 1), dtype)
    # in place
    keep = torch.cat(grads, 1)
    op.logprobs_backward(sh, targets, lse, glp, sh)
    assert torch.equal(torch.cat(sh, 1), keep)


def check_logprob_gradient(x, tau, lse, H, targets, glp, gH, got, dtype):
    x = x.double() / tau
    empty = (lse < NOTHING_LEFT)[:, None]
    l = torch.where(empty, 0.0, lse.double()[:, None])
    logp = x - l
    p = torch.where(empty, 0.0, logp.exp())
    gl, gh = torch.where(targets < 0, 0.0, glp.double())[:, None], gH.double()[:, None]
    plogp = torch.where(p > 0, p * logp, 0.0)
    want = -(p * (gl + gh * H.double()[:, None]) + gh * plogp)
    mag = p * (gl.abs() + gh.abs() * H.double()[:, None].abs()) + gh.abs() * plogp.abs()
    hit = torch.zeros_like(want).scatter_(1, targets.clamp(min=0)[:, None], gl)
    want, mag = torch.where(empty, 0.0, want + hit) / tau, (mag + hit.abs()) / tau
    # log p loses 4 E of the size of x and lse, which moves p by as much, relative, and stands beside p log p
    # itself; 2^t is good to 2^-22
    far = torch.where(torch.isfinite(x), x.abs(), 0.0) + l.abs()
    moved = torch.clamp(2.0 ** -21 + 4 * E * far, max=1.0)
    close(got, want, mag * moved + torch.where(p > 0, gh.abs() * p * moved / tau, 0.0), dtype, "logits' gradient")


@pytest.mark.parametrize("spec", HEADS, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("teacher", ["f32", "own"])
def test_distill_and_gradient(ops, spec, teacher):
    R, T, V, dtype, _, tau, masked, pad, off = spec
    K = min(V, {66: 66, 1000: 256, 4096: 100}.get(V, 33))
    g = gen(31)
    x, _ = logits(g, T, V, dtype)
    tdt = "f32" if teacher == "f32" else dtype
    ids = (torch.randint(V, (T, 1), generator=g, device="cuda") + torch.randint(1, V // K + 1, (T, K), generator=g,
                                                                             device="cuda").cumsum(1)) % V
    t = randn(g, T, K, dtype=tdt, sigma=3.0)
    x.scatter_(1, ids, t.to(x.dtype))
    if masked:
        mask_rows(x, g)
    rows = torch.arange(T, device="cuda")
    ids[rows % 5 == 3] = -1                      # no teacher at all
    if K > 2:
        ids[rows % 5 == 2, 1] = V + 4            # no column
        t[rows % 4 == 1, 2] = -math.inf
        ids[rows % 3 == 1, K - 1] = ids[rows % 3 == 1, 0]   # a token twice
        t[rows % 13 == 12] = -math.inf
    sh = shards_of(x, R, pad, off)
    op = ops.VocabHead(R, V, dtype, temperature=tau)
    loss, lse = (torch.full((T,), 9.0, device="cuda") for _ in range(2))
    op.distill(sh, ids, t, loss, lse)

    logp, lse64, _ = stats64(x, tau)
    absent = (ids < 0) | (ids >= V) | (t == -math.inf)
    q = torch.softmax(torch.where(absent, -math.inf, t.double() / tau), 1)
    taught = ~absent.all(1)
    q = torch.where(taught[:, None], q, 0.0)
    at = logp.gather(1, ids.clamp(0, V - 1))
    logq = torch.where(q > 0, q, 1.0).log()
    terms = torch.where(q > 0, q * (logq - at), 0.0)
    want = (terms.sum(1) * tau ** 2).float().double()   # lowest-value logits: rounded to binary32's range
    slack = stat_loss(x, tau, V)
    size = torch.where(torch.isfinite(terms), (q * (logq.abs() + torch.where(q > 0, at, 0.0).abs())), 0.0).sum(1)
    tmag = torch.where(absent, 0.0, t.double().abs() / tau).amax(1)
    same(loss, want, tau ** 2 * (slack + (K + 64) * E * (1 + size) + 8 * E * tmag), "loss")
    lse64 = lse64.float().double()
    same(lse, lse64, slack + 4 * E * torch.where(torch.isfinite(lse64), lse64.abs(), 0.0), "lse")

    gl = randn(g, T, mean=1.0, sigma=0.2)
    grads = [torch.full_like(s, 9.0) for s in shards_of(x, R, pad, off)]
    op.distill_backward(sh, ids, t, lse, gl, grads)
    empty = (lse < NOTHING_LEFT)[:, None]
    l = torch.where(empty, 0.0, lse.double()[:, None])
    p = torch.where(empty | ~taught[:, None], 0.0, (x.double() / tau - l).exp())
    qs = torch.zeros_like(p).scatter_add_(1, ids.clamp(0, V - 1), torch.where(empty, 0.0, q))
    c = gl.double()[:, None] * tau
    far = torch.where(torch.isfinite(x), x.double().abs() / tau, 0.0) + l.abs()
    slackg = torch.clamp(2.0 ** -21 + 4 * E * far, max=1.0) * p + (K + 64 + 8 * tmag[:, None]) * E * qs
    close(torch.cat(grads, 1), c * (p - qs), c.abs() * (slackg + 4 * E * (p + qs)), dtype, "logits' gradient")
    keep = torch.cat(grads, 1)
    op.distill_backward(sh, ids, t, lse, gl, sh)
    assert torch.equal(torch.cat(sh, 1), keep)


@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_head_infinities_and_nan(ops, value):
    """+inf or NaN anywhere in a row makes that row's values NaN, and no other's; NaN is the largest alternative."""
    T, V, R = 6, 5000, 3
    g = gen(41)
    x, _ = logits(g, T, V, "f32")
    x[1, 4321] = value
    x[4, 77] = value
    x[4, 78:] = -math.inf
    op = ops.VocabHead(R, V, "f32")
    targets = torch.full((T,), 5, device="cuda")
    lp, lse, H = (torch.zeros(T, device="cuda") for _ in range(3))
    ids = torch.zeros((T, 4), dtype=torch.int64, device="cuda")
    tlp = torch.zeros((T, 4), device="cuda")
    op.logprobs(shards_of(x, R), targets, lp, lse, H, ids, tlp)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[1, 4]] = True
    for v in (lp, lse, H, tlp[:, 0], tlp[:, 3]):
        assert torch.equal(torch.isnan(v), bad)
    assert torch.equal(ids, top_ids64(x, 4))
    loss = torch.zeros(T, device="cuda")
    tid = torch.arange(8, device="cuda").expand(T, 8).contiguous()
    op.distill(shards_of(x, R), tid, randn(g, T, 8), loss, lse)
    assert torch.equal(torch.isnan(loss), bad)
    grads = [torch.zeros_like(s) for s in shards_of(x, R)]
    op.logprobs_backward(shards_of(x, R), targets, lse, torch.ones(T, device="cuda"), grads)
    assert torch.equal(torch.isnan(torch.cat(grads, 1)).all(1), bad)
    assert torch.equal(torch.isnan(torch.cat(grads, 1)).any(1), bad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_top_alternatives_with_many_ties(ops, dtype):
    """Equal logits everywhere, periodic ones that fall to few threads, rising and falling rows: ties to the lower column."""
    V, K, R = 40000, 32, 4
    j = torch.arange(V, device="cuda")
    x = torch.stack([torch.zeros(V, device="cuda"), (j % 2048 == 7).float(), (j % 512 == 3).float() + (j % 64 == 5),
                     j / 1000.0, -j / 1000.0, (j == V - 1).float(), -0.0 * (j % 3), (j * 7919 % V) / 100.0]).to(TORCH[dtype])
    T = x.shape[0]
    op = ops.VocabHead(R, V, dtype)
    lp, lse = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    ids = torch.zeros((T, K), dtype=torch.int64, device="cuda")
    tlp = torch.zeros((T, K), device="cuda")
    op.logprobs(shards_of(x, R), torch.zeros(T, dtype=torch.int64, device="cuda"), lp, lse, None, ids, tlp)
    assert torch.equal(ids, top_ids64(x, K))


def test_target_outside_the_vocabulary_is_nan(ops):
    x, _ = logits(gen(1), 3, 100, "f32")
    op = ops.VocabHead(2, 100, "f32")
    lp, lse = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
    targets = torch.tensor([99, 100, 1 << 40], device="cuda")
    op.logprobs(shards_of(x, 2), targets, lp, lse)
    assert torch.isnan(lp).tolist() == [False, True, True]
    grads = [torch.zeros_like(s) for s in shards_of(x, 2)]
    op.logprobs_backward(shards_of(x, 2), targets, lse, torch.ones(3, device="cuda"), grads)
    assert torch.isnan(torch.cat(grads, 1)).all(1).tolist() == [False, True, True]


def test_head_gradients_against_differences(ops):
    """Along a random direction, against central differences of the 64-bit
    definitions (step 1e-5); the kernel's own loss is below 1e-4 of the scale."""
    T, V, R, K, tau = 5, 301, 3, 7, 1.7
    g = gen(51)
    x = torch.randn((T, V), generator=g, device="cuda")
    v = torch.randn((T, V), generator=g, device="cuda", dtype=torch.float64)
    targets = torch.randint(V, (T,), generator=g, device="cuda")
    ids, t = torch.randint(V, (T, K), generator=g, device="cuda"), randn(g, T, K)
    a, b = randn(g, T), randn(g, T)
    op = ops.VocabHead(R, V, "f32", temperature=tau)
    lp, lse, H, loss = (torch.zeros(T, device="cuda") for _ in range(4))
    op.logprobs(shards_of(x, R), targets, lp, lse, H)
    grads = [torch.zeros_like(s) for s in shards_of(x, R)]

    def policy(s):
        logp, _, h = stats64(x.double() + s * v, tau)
        return (a.double() * logp.gather(1, targets[:, None])[:, 0] + b.double() * h).sum().item()

    def distill(s):
        logp, _, _ = stats64(x.double() + s * v, tau)
        q = torch.softmax(t.double() / tau, 1)
        return (a.double() * tau ** 2 * (q * (q.log() - logp.gather(1, ids))).sum(1)).sum().item()

    op.logprobs_backward(shards_of(x, R), targets, lse, a, grads, entropy=H, grad_entropy=b)
    got = torch.cat(grads, 1).double()
    slope = (policy(1e-5) - policy(-1e-5)) / 2e-5
    assert abs((got * v).sum().item() - slope) <= 1e-4 * (got * v).abs().sum().item()
    op.distill(shards_of(x, R), ids, t, loss, lse)
    op.distill_backward(shards_of(x, R), ids, t, lse, a, grads)
    got = torch.cat(grads, 1).double()
    slope = (distill(1e-5) - distill(-1e-5)) / 2e-5
    assert abs((got * v).sum().item() - slope) <= 1e-4 * (got * v).abs().sum().item()


def test_shards_are_column_slices_of_one_matrix(ops):
    """The shards (and their gradients) as slices of a full matrix: interleaved rows are no overlap."""
    T, V, R = 9, 1000, 4
    x, _ = logits(gen(61), T, V, "bf16")
    op = ops.VocabHead(R, V, "bf16")
    targets = torch.arange(T, device="cuda")
    lp, lse, one = (torch.ones(T, device="cuda") for _ in range(3))
    want_lp, want_lse = torch.zeros_like(lp), torch.zeros_like(lp)
    views = list(x.split(250, 1))
    op.logprobs(views, targets, lp, lse)
    op.logprobs(shards_of(x, R), targets, want_lp, want_lse)
    # the rows start elsewhere within their 16-byte vectors, so the sums are grouped differently
    slack = 2 * (stat_loss(x, 1.0, V) + 8 * E * (lp.abs() + lse.abs()))
    same(lp, want_lp, slack, "logprob")
    same(lse, want_lse, slack, "lse")
    grads = [torch.zeros_like(s) for s in shards_of(x, R)]
    op.logprobs_backward(shards_of(x, R), targets, lse, one, grads)
    op.logprobs_backward(views, targets, lse, one, views)
    assert torch.equal(x, torch.cat(grads, 1))


def test_offsets_beyond_32_bits(ops):
    """Rows 2^30 elements apart: the last one starts at element 2^31."""
    T, V, R, stride = 3, 1003, 2, 1 << 30
    x, hot = logits(gen(71), T, V, "bf16")
    buf = torch.zeros(2 * stride + 2048, dtype=torch.bfloat16, device="cuda")
    far = buf[:2 * stride + V].as_strided((T, V), (stride, 1))
    far.copy_(x)
    views = [far[:, :502], far[:, 502:]]
    op = ops.VocabHead(R, V, "bf16")
    lp, lse, one = (torch.ones(T, device="cuda") for _ in range(3))
    want_lp, want_lse = torch.zeros_like(lp), torch.zeros_like(lp)
    op.logprobs(views, hot[:, 0].contiguous(), lp, lse)
    op.logprobs(shards_of(x, R), hot[:, 0].contiguous(), want_lp, want_lse)
    slack = 2 * (stat_loss(x, 1.0, V) + 8 * E * (lp.abs() + lse.abs()))
    same(lp, want_lp, slack, "logprob")
    same(lse, want_lse, slack, "lse")
    grads = [torch.zeros_like(s) for s in shards_of(x, R)]
    op.logprobs_backward(shards_of(x, R), hot[:, 0].contiguous(), lse, one, grads)
    op.logprobs_backward(views, hot[:, 0].contiguous(), lse, one, views)
    assert torch.equal(far, torch.cat(grads, 1))
    # block end: parts of width 1000 in the same far rows
    far = buf[:2 * stride + 1000].as_strided((T, 1000), (stride, 1))
    c = Norm(72, 1, T, 1000, "bf16", "bf16", "bf16", True, 1)
    far.copy_(c.parts[0])
    c.parts = [far]
    op, z, h2, total, rstd = c.run(ops, 1)
    c.check_forward(z, h2, total, rstd)


def test_no_rows(ops):
    op = ops.BlockNorm(2, 64, "bf16")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    op.forward([e, e], e, w, [e], e)
    head = ops.VocabHead(2, 64, "bf16")
    s, i = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    f = torch.empty(0, device="cuda")
    head.logprobs([s, s], i, f, f)
    head.distill([s, s], torch.empty((0, 4), dtype=torch.int64, device="cuda"), torch.empty((0, 4), device="cuda"), f, f)


def test_other_stream_graph_and_repeats(ops):
    """On a stream of the caller's, in a CUDA graph, and again: the same bits."""
    c = Norm(81, 4, 130, 1024, "bf16", "f32", "f32", True, 2)
    op, z, h2, total, rstd = c.run(ops, 1)
    first = c.run_backward(op, h2, total, rstd, c.grad_z, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, z2, h3, _, _ = c.run(ops, 1, stream=side)
    side.synchronize()
    assert torch.equal(z[0], z2[0]) and torch.equal(h2, h3)
    gin, gh = [torch.zeros_like(first[0][0])], torch.zeros_like(first[1])
    gw, gp, gg = (torch.zeros_like(t) for t in first[2:])
    x, _ = logits(gen(82), 50, 30000, "bf16")
    head = ops.VocabHead(8, 30000, "bf16")
    sh = shards_of(x, 8)
    targets = torch.arange(50, device="cuda")
    lp, lse, H = (torch.zeros(50, device="cuda") for _ in range(3))
    ids, tlp = torch.zeros((50, 9), dtype=torch.int64, device="cuda"), torch.zeros((50, 9), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.backward(c.grad_z, c.grad_h, h2, rstd, c.weight, gin, gh, gw, post_weight=c.post, gate=c.gate, total=total,
                    grad_post_weight=gp, grad_gate=gg)
        head.logprobs(sh, targets, lp, lse, H, ids, tlp)
    for _ in range(2):
        for t in (gin[0], gh, gw, gp, gg, lp, lse, H, ids, tlp):
            t.zero_()
        graph.replay()
        for got, want in zip((gin[0], gh, gw, gp, gg), (first[0][0], *first[1:])):
            assert torch.equal(got, want)
        w = [torch.zeros_like(t) for t in (lp, lse, H, ids, tlp)]
        head.logprobs(sh, targets, *w)
        for got, want in zip((lp, lse, H, ids, tlp), w):
            assert torch.equal(got, want)


def test_calls_back_to_back_in_place(ops):
    """Dependent calls in a stream with nothing between them, each reading what
    the one before wrote in place: the same bits as with a wait after each."""
    c = Norm(91, 3, 40, 1024, "bf16", "f32", "f32", True, 2)
    head = ops.VocabHead(3, 1024, "bf16", temperature=1.5)
    op, z, h2, total, rstd = c.run(ops, 1)
    ids, t = torch.arange(40 * 6, device="cuda").view(40, 6) * 4 % 1024, randn(gen(92), 40, 6)

    def chain(wait):
        parts, residual = [p.clone() for p in c.parts], c.residual.clone()
        loss, lse, one = (torch.ones(40, device="cuda") for _ in range(3))
        gh, gw = torch.empty_like(residual), torch.empty(1024, device="cuda")
        for _ in range(5):
            op.forward(parts, residual, c.weight, parts, residual, post_weight=c.post, gate=c.gate, total=total,
                       rstd=rstd)
            wait()
            sh = list(parts[0].split(head.widths, 1))
            head.distill(sh, ids, t, loss, lse)
            wait()
            head.distill_backward(sh, ids, t, lse, one, sh)
            wait()
            op.backward(parts, residual, residual, rstd, c.weight, parts, gh, gw, post_weight=c.post, gate=c.gate,
                        total=total)
            wait()
        return parts + [residual, loss, lse, gh, gw]

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(chain(lambda: None), want):
            assert torch.equal(a, b)


def test_first_backward_in_a_capture_is_refused(ops):
    from ring_allreduce_gb300 import RAError, Status
    c = Norm(83, 2, 8, 64, "f32", "f32", "f32", True, 1)
    op, z, h2, total, rstd = c.run(ops, 1)
    out = torch.empty_like(h2)
    g = torch.empty_like(h2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RAError) as e:
            op.backward(c.grad_z, c.grad_h, h2, rstd, c.weight, [g], out, post_weight=c.post, total=total)
        out.zero_()
    assert e.value.status == Status.ERR_UNSUPPORTED


def test_refusals(ops):
    from ring_allreduce_gb300 import RAError, Status

    def refused(status, f, *a, **k):
        with pytest.raises(RAError) as e:
            f(*a, **k)
        assert e.value.status == status, e.value

    for args in ((0, 64), (33, 64), (2, 0)):
        refused(Status.ERR_INVALID, ops.BlockNorm, *args)
    refused(Status.ERR_UNSUPPORTED, ops.BlockNorm, 2, 16385)
    refused(Status.ERR_UNSUPPORTED, ops.BlockNorm, 2, 64, "bf16", "f16")
    refused(Status.ERR_UNSUPPORTED, ops.BlockNorm, 2, 64, "f32", "f32", "bf16")
    refused(Status.ERR_INVALID, ops.BlockNorm, 2, 64, eps=-1.0)
    refused(Status.ERR_INVALID, ops.BlockNorm, 2, 64, scale=math.inf)
    with pytest.raises(ValueError):
        ops.BlockNorm(2, 64, "i32")
    for args in ((0, 64), (33, 64), (2, 0), (2, (1 << 30) + 1)):
        refused(Status.ERR_INVALID, ops.VocabHead, *args)
    for tau in (0.0, -1.0, math.nan, math.inf):
        refused(Status.ERR_INVALID, ops.VocabHead, 2, 64, temperature=tau)

    op = ops.BlockNorm(2, 64, "f32")
    x, y, z, h = (torch.zeros((6, 64), device="cuda") for _ in range(4))
    w = torch.ones(64, device="cuda")
    gate = torch.ones((4, 64), device="cuda")
    op.forward([x, y], z, w, [h], z)
    refused(Status.ERR_INVALID, op.forward, [x, y], z, w, [h], h)              # two outputs in one place
    refused(Status.ERR_INVALID, op.forward, [x, y], z, w, [z], h)              # an output over an input
    refused(Status.ERR_INVALID, op.forward, [x, y], z, w, [y], h)              # in place on another rank's buffer
    refused(Status.ERR_INVALID, op.forward, [x, y], z, w, [h], torch.zeros((7, 64), device="cuda")[1:], gate=gate)
    refused(Status.ERR_INVALID, op.forward, [x, y], z, w, [h], torch.zeros((1, 64), device="cuda").expand(6, 64))
    for bad in ([x], [x, y, z], [x, y[:5]], [x, y.half()], [x, y.cpu()], [x, torch.zeros((64, 6), device="cuda").t()],
                [x, 7]):
        with pytest.raises(ValueError):
            op.forward(bad, z, w, [h], z)
    for kw in (dict(post_weight=w[:63]), dict(gate=w), dict(rstd=torch.zeros((6, 2), device="cuda")),
               dict(total=h.half())):
        with pytest.raises(ValueError):
            op.forward([x, y], z, w, [h], torch.empty_like(z), **kw)
    rstd = torch.zeros((2, 6), device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    refused(Status.ERR_INVALID, op.backward, [x, y], None, z, rstd, w, [a], b, post_weight=w)   # no total
    refused(Status.ERR_INVALID, op.backward, [x, y], None, z, rstd, w, [a], b, grad_post_weight=torch.zeros_like(w))
    with pytest.raises(ValueError):
        op.backward([x, y], None, z, rstd, w, [a], b, grad_gate=gate)
    op.close()
    with pytest.raises(ValueError):
        op.forward([x, y], z, w, [h], z)

    head = ops.VocabHead(2, 64, "f32")
    s = [torch.zeros((6, 32), device="cuda") for _ in range(2)]
    t = torch.zeros(6, dtype=torch.int64, device="cuda")
    lp, lse = torch.zeros(6, device="cuda"), torch.zeros(6, device="cuda")
    ids, tl = torch.zeros((6, 33), dtype=torch.int64, device="cuda"), torch.zeros((6, 33), device="cuda")
    refused(Status.ERR_INVALID, head.logprobs, s, t, lp, lse, None, ids, tl)
    refused(Status.ERR_INVALID, head.logprobs, s, t, lp, lp)
    refused(Status.ERR_INVALID, head.logprobs_backward, s, t, lse, lp, [s[1], torch.zeros_like(s[0])])
    refused(Status.ERR_INVALID, head.distill, s, torch.zeros((6, 257), dtype=torch.int64, device="cuda"),
            torch.zeros((6, 257), device="cuda"), lp, lse)
    refused(Status.ERR_INVALID, head.distill, s, torch.zeros((6, 0), dtype=torch.int64, device="cuda"),
            torch.zeros((6, 0), device="cuda"), lp, lse)
    for bad in ([s[0]], [s[0], s[1][:, :31]], [s[0], s[1].half()]):
        with pytest.raises(ValueError):
            head.logprobs(bad, t, lp, lse)
    with pytest.raises(ValueError):
        head.logprobs(s, t.int(), lp, lse)
    with pytest.raises(ValueError):
        head.logprobs(s, t, lp, lse, None, ids)
    small = ops.VocabHead(1, 8, "f32")
    refused(Status.ERR_INVALID, small.logprobs, [torch.zeros((6, 8), device="cuda")], t, lp, lse, None,
            ids[:, :9].contiguous(), tl[:, :9].contiguous())


def test_host_memory_is_refused_by_the_library(ops):
    """The C boundary itself: host addresses and NULL come back as RA_ERR_INVALID."""
    import ctypes
    from ring_allreduce_gb300 import binding

    class Args(ctypes.Structure):   # ra_norm_forward_args
        _fields_ = [(n, ctypes.c_int if n == "outs" else ctypes.c_size_t if n == "rows" or n.endswith("stride") or
                     n == "gate_rows" else ctypes.c_void_p) for n in
                    ("rows in in_stride residual residual_stride weight post_weight gate gate_rows out out_stride outs "
                     "residual_out residual_out_stride total total_stride rstd").split()]

    lib, h = binding._lib, ctypes.c_void_p()
    assert lib.ra_norm_create(1, 64, 0, 0, 0, 1e-6, 1.0, ctypes.byref(h)) == 0
    dev, host, w = torch.zeros((2, 64), device="cuda"), torch.zeros((2, 64)), torch.ones(64, device="cuda")
    out, res = torch.empty_like(dev), torch.empty_like(dev)
    for ptr, status in ((host.data_ptr(), 1), (None, 1), (dev.data_ptr(), 0)):
        ins, outs = (ctypes.c_void_p * 1)(ptr), (ctypes.c_void_p * 1)(out.data_ptr())
        a = Args(rows=2, residual=dev.data_ptr(), residual_stride=64, in_stride=64, weight=w.data_ptr(),
                 out=ctypes.addressof(outs), out_stride=64, outs=1, residual_out=res.data_ptr(), residual_out_stride=64)
        setattr(a, "in", ctypes.addressof(ins))
        assert lib.ra_norm_forward(h, ctypes.addressof(a), None) == status
    assert lib.ra_norm_set_option(h, binding.Option.VARIANT, 1) == 1
    assert lib.ra_norm_set_option(h, binding.Option.CHECK_POINTERS, 2) == 1
    assert lib.ra_norm_destroy(h) == 0
