"""The vocabulary head on rows whose logits are far from zero: masks of an
ordinary large value (-1e9, -1e10, -1e30, ...) over part or all of a row, rows
that lie far above zero, and temperatures that take logits there.  Against the
definitions in 64 bits, which take a row's largest logit off first.

What binary32 loses, beside the one rounding of an output (E its unit
roundoff): a row's sum of powers is good to 2^-21 (2^x: 2^-22, its exponent:
the weighted sum of |t| E over the terms, at most log2 V and a few) and loses at
most one E an addition, V / 32 of them a thread in the smallest CTAs and 64 in
the joins.  A value x / tau or x - max is good to a few roundings (the
reciprocal of tau, its product with log2 e, the product with x, the last sum and
product): 8 E of its size covers them."""

import math

import pytest

from test_gpu_operators import E, close, gen, logits, randn, same, shards_of, stats64, top_ids64

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

NO_GRADIENT = -1e30   # rows with a smaller lse have none
FILLS = {"f32": (-1e5, -1e7, -1e9, -1e10, -1e20, -1e30, -1e37, -3e38),
         "bf16": (-1e5, -1e7, -1e9, -1e10, -1e20, -1e30, -1e37, -3e38), "f16": (-1e3, -2e4, -6e4)}
KINDS = 7
# R, V, times the rows are there, pad, off: few rows, split over CTAs; many short ones
SHAPES = [(3, 50021, 1, 0, 1), (4, 1501, 24, 3, 0)]
CASES = [(s, d, tau) for s in SHAPES for d in FILLS for tau in (0.7, 1.0, 2.0, 1e-3)]


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_gb300 import build
    build.build()
    from ring_allreduce_gb300 import operators
    return operators


def far_rows(g, V, dtype, times):
    """Seven rows for each value: filled with it, all but one token, the first two thirds, nine tenths in places;
    spread around it; and filled with, or spread around, its negative."""
    x, _ = logits(g, KINDS * len(FILLS[dtype]) * times, V, dtype)
    most = torch.finfo(x.dtype).max
    for t in range(x.shape[0]):
        fill, kind = FILLS[dtype][t // KINDS % len(FILLS[dtype])], t % KINDS
        if kind == 1:
            keep = x[t, t * 31 % V].clone()
            x[t] = fill
            x[t, t * 31 % V] = keep
        elif kind == 2:
            x[t, :2 * V // 3] = fill
        elif kind == 3:
            x[t, torch.rand(V, generator=g, device="cuda") < 0.9] = fill
        else:
            spread = 2.0 ** -6 * torch.randn(V, generator=g, device="cuda") if kind in (4, 6) else torch.zeros_like(x[t])
            sign = -1.0 if kind > 4 else 1.0
            x[t] = (sign * fill * (1.0 + spread.float())).clamp(-most, most).to(x.dtype)
    return x


def sum_loss(V):
    return 2.0 ** -21 + (V / 32 + 64) * E


def size(v):
    return torch.where(torch.isfinite(v), v.abs(), 0.0)


def in_f32(v):
    """Values divided by tau may leave binary32's range: rounded to it."""
    return v.float().double()


def case(spec):
    (R, V, times, pad, off), dtype, tau = spec
    g = gen(101)
    x = far_rows(g, V, dtype, times)
    T = x.shape[0]
    targets = torch.where(torch.rand(T, generator=g, device="cuda") < 0.5, x.float().argmax(1),
                          torch.randint(V, (T,), generator=g, device="cuda"))
    return g, x, targets, shards_of(x, R, pad, off)


@pytest.mark.parametrize("spec", CASES, ids=lambda s: "-".join(map(str, (*s[0], *s[1:]))))
def test_logprobs_of_far_rows(ops, spec):
    (R, V, *_), dtype, tau = spec
    g, x, targets, sh = case(spec)
    T, K = x.shape[0], 20
    op = ops.VocabHead(R, V, dtype, temperature=tau)
    lp, lse, H = (torch.full((T,), 9.0, device="cuda") for _ in range(3))
    ids, tlp = torch.full((T, K), -7, device="cuda"), torch.full((T, K), 9.0, device="cuda")
    op.logprobs(sh, targets, lp, lse, H, ids, tlp)
    logp, lse64, H64 = stats64(x, tau)
    same(lse, in_f32(lse64), sum_loss(V) + 8 * E * size(lse64), "lse")
    want = logp.gather(1, targets[:, None])[:, 0]
    same(lp, in_f32(want), sum_loss(V) + 8 * E * size(want), "logprob")
    same(H, H64, (sum_loss(V) + 8 * E) * (2 + math.log(V)), "entropy")
    assert torch.equal(ids, top_ids64(x, K))
    want = logp.gather(1, ids)
    same(tlp, in_f32(want), sum_loss(V) + 8 * E * size(want), "top")


def teacher(g, T, V, K):
    ids = torch.randint(V, (T, K), generator=g, device="cuda")
    return ids, randn(g, T, K, sigma=3.0)


@pytest.mark.parametrize("spec", CASES, ids=lambda s: "-".join(map(str, (*s[0], *s[1:]))))
def test_distill_of_far_rows(ops, spec):
    (R, V, *_), dtype, tau = spec
    g, x, _, sh = case(spec)
    T, K = x.shape[0], 16
    ids, t = teacher(g, T, V, K)
    op = ops.VocabHead(R, V, dtype, temperature=tau)
    loss, lse = (torch.full((T,), 9.0, device="cuda") for _ in range(2))
    op.distill(sh, ids, t, loss, lse)
    logp, lse64, _ = stats64(x, tau)
    same(lse, in_f32(lse64), sum_loss(V) + 8 * E * size(lse64), "lse")
    logq = torch.log_softmax(t.double() / tau, 1)
    q, at = logq.exp(), logp.gather(1, ids)
    terms = torch.where(q > 0, q * (logq - at), 0.0)
    mags = torch.where(q > 0, q * (logq.abs() + at.abs()), 0.0)
    mag, tmag = mags.sum(1), t.double().abs().amax(1) / tau
    # shares: exp of (t - max) / tau, good to 8 E of that, and lost where they are below binary32's normal range;
    # terms: K additions and a few products
    lost = torch.where(q < 2.0 ** -126, 2 * mags, 0.0).sum(1)
    tol = tau ** 2 * (sum_loss(V) + (K + 64) * E * (1 + mag) + 8 * E * tmag * (1 + mag) + lost)
    same(loss, in_f32(terms.sum(1) * tau ** 2), tol, "loss")


def p_loss(x, tau, lse, logp, V):
    """What a probability loses, relative: the sum's loss and, where lse tells probabilities apart (|lse| up to 2^14),
    the roundings of x / tau and lse; else those of x - max alone."""
    sharp = (lse.abs() <= 2.0 ** 14)[:, None]
    far = torch.where(sharp, size(x.double() / tau) + size(lse.double())[:, None], 0.0)
    return torch.clamp(sum_loss(V) + 8 * E * (far + 1 + size(logp).clamp(max=150.0)), max=1.0)


@pytest.mark.parametrize("spec", CASES, ids=lambda s: "-".join(map(str, (*s[0], *s[1:]))))
def test_logprob_gradient_of_far_rows(ops, spec):
    """The gradient from the rows' own softmax in 64 bits, not from the lse that forward wrote."""
    (R, V, *_), dtype, tau = spec
    g, x, targets, sh = case(spec)
    T = x.shape[0]
    op = ops.VocabHead(R, V, dtype, temperature=tau)
    lp, lse, H = (torch.full((T,), 9.0, device="cuda") for _ in range(3))
    op.logprobs(sh, targets, lp, lse, H)
    glp, gH = randn(g, T), randn(g, T, sigma=0.3)
    grads = [torch.full_like(s, 9.0) for s in sh]
    op.logprobs_backward(sh, targets, lse, glp, grads, entropy=H, grad_entropy=gH)

    logp, _, _ = stats64(x, tau)
    none = (lse < NO_GRADIENT)[:, None]
    p = torch.where(none, 0.0, logp.exp())
    gl, gh, h = (v.double()[:, None] for v in (glp, gH, H))
    plogp = torch.where(p > 0, p * logp, 0.0)
    hit = torch.where(none, 0.0, torch.zeros_like(p).scatter_(1, targets[:, None], gl))
    want = (hit - p * (gl + gh * h) - gh * plogp) / tau
    mag = (hit.abs() + p * (gl.abs() + gh.abs() * h.abs()) + gh.abs() * plogp.abs() + gh.abs() * p) / tau
    close(torch.cat(grads, 1), want, mag * p_loss(x, tau, lse, logp, V), dtype, "logits' gradient")
    keep = torch.cat(grads, 1)
    op.logprobs_backward(sh, targets, lse, glp, sh, entropy=H, grad_entropy=gH)
    assert torch.equal(torch.cat(sh, 1), keep)


@pytest.mark.parametrize("spec", CASES, ids=lambda s: "-".join(map(str, (*s[0], *s[1:]))))
def test_distill_gradient_of_far_rows(ops, spec):
    (R, V, *_), dtype, tau = spec
    g, x, _, sh = case(spec)
    T, K = x.shape[0], 16
    ids, t = teacher(g, T, V, K)
    op = ops.VocabHead(R, V, dtype, temperature=tau)
    loss, lse = (torch.full((T,), 9.0, device="cuda") for _ in range(2))
    op.distill(sh, ids, t, loss, lse)
    gl = randn(g, T, mean=1.0, sigma=0.2)
    grads = [torch.full_like(s, 9.0) for s in sh]
    op.distill_backward(sh, ids, t, lse, gl, grads)

    logp, _, _ = stats64(x, tau)
    none = (lse < NO_GRADIENT)[:, None]
    p = torch.where(none, 0.0, logp.exp())
    q = torch.softmax(t.double() / tau, 1)
    qs = torch.where(none, 0.0, torch.zeros_like(p).scatter_add_(1, ids, q))
    c = gl.double()[:, None] * tau
    tmag = (t.double().abs().amax(1) / tau)[:, None]
    slack = p * p_loss(x, tau, lse, logp, V) + torch.clamp((K + 64 + 8 * tmag) * E, max=1.0) * qs + 4 * E * (p + qs)
    close(torch.cat(grads, 1), c * (p - qs), c.abs() * slack, dtype, "logits' gradient")
    keep = torch.cat(grads, 1)
    op.distill_backward(sh, ids, t, lse, gl, sh)
    assert torch.equal(torch.cat(sh, 1), keep)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_far_row_alone(ops, dtype):
    """One row over many CTAs, nothing left by a mask of -1e10: its gradient is that of equal probabilities, in place too."""
    V, R = 131072, 8
    x = torch.full((1, V), -1e10, device="cuda").to(logits(gen(1), 1, 8, dtype)[0].dtype)
    sh, targets = shards_of(x, R), torch.tensor([77777], device="cuda")
    op = ops.VocabHead(R, V, dtype)
    lp, lse, one = (torch.ones(1, device="cuda") for _ in range(3))
    op.logprobs(sh, targets, lp, lse)
    assert abs(lp.item() + math.log(V)) <= 1e-5
    op.logprobs_backward(sh, targets, lse, one, sh)
    want = torch.full((1, V), -1.0 / V, dtype=torch.float64, device="cuda")
    want[0, 77777] += 1.0
    close(torch.cat(sh, 1), want, sum_loss(V) * want.abs(), dtype, "logits' gradient")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [1e-3, 0.7])
def test_gradients_of_small_probabilities(ops, dtype, tau):
    """Probabilities below binary32's normal range, which over a small tau are numbers of the output's type again."""
    T, V = 9, 1000
    g = gen(103)
    x = (tau * (-86.0 - 12.0 * torch.rand((T, V), generator=g, device="cuda"))).to(logits(g, 1, 8, dtype)[0].dtype)
    x[:, 5] = 0.0
    sh, targets = shards_of(x, 3), torch.full((T,), 7, device="cuda")
    op = ops.VocabHead(3, V, dtype, temperature=tau)
    lp, lse, H = (torch.full((T,), 9.0, device="cuda") for _ in range(3))
    op.logprobs(sh, targets, lp, lse, H)
    glp, gH = randn(g, T), randn(g, T, sigma=0.3)
    grads = [torch.full_like(s, 9.0) for s in sh]
    op.logprobs_backward(sh, targets, lse, glp, grads, entropy=H, grad_entropy=gH)
    logp, _, _ = stats64(x, tau)
    p, gl, gh, h = logp.exp(), *(v.double()[:, None] for v in (glp, gH, H))
    hit = torch.zeros_like(p).scatter_(1, targets[:, None], gl)
    want = (hit - p * (gl + gh * h) - gh * p * logp) / tau
    mag = (hit.abs() + p * (gl.abs() + gh.abs() * (h.abs() + logp.abs() + 1))) / tau
    # x / tau is below 128 and lse below E: their roundings are 8 E of 128; log p stands as a factor too
    close(torch.cat(grads, 1), want, mag * (sum_loss(V) + 8 * E * 128), dtype, "logits' gradient")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tau", [0.7, 1.0, 1.3])
def test_no_entropy_below_zero_and_no_probability_above_one(ops, dtype, tau):
    """Rows with one allowed token (constrained decoding), and rows where one token leaves the others next to nothing."""
    T, V, R = 512, 4099, 4
    g = gen(111)
    x = randn(g, T, V, dtype=dtype)
    targets = torch.randint(V, (T,), generator=g, device="cuda")
    rows = torch.arange(T, device="cuda")
    own = x[rows, targets].clone()
    x[: T // 2] = -math.inf
    x[rows, targets] = torch.where(rows < T // 2, own, (own.float() + 30.0).to(x.dtype))
    op = ops.VocabHead(R, V, dtype, temperature=tau)
    lp, lse, H = (torch.full((T,), 9.0, device="cuda") for _ in range(3))
    ids, tlp = torch.zeros((T, 3), dtype=torch.int64, device="cuda"), torch.zeros((T, 3), device="cuda")
    op.logprobs(shards_of(x, R), targets, lp, lse, H, ids, tlp)
    assert (H >= 0).all() and (lp <= 0).all() and (tlp <= 0).all(), (H.min(), lp.max(), tlp.max())
    assert torch.equal(ids[:, 0], targets) and torch.equal(tlp[:, 0], lp)
    logp, _, H64 = stats64(x, tau)
    same(lp, logp[rows, targets], sum_loss(V), "logprob")
    same(H, H64, (sum_loss(V) + 8 * E) * (2 + math.log(V)), "entropy")


@pytest.mark.parametrize("tau", [0.7, 1.0, 2.0])
def test_loss_of_tokens_at_the_lowest_value(ops, tau):
    """Every token that the teacher knows at binary32's lowest value: the loss is that value's size times tau, a number
    up to tau = 1, whatever the rounded shares add up to."""
    T, V, K = 700, 300, 33
    g = gen(121)
    x, _ = logits(g, T, V, "f32")
    ids = torch.rand((T, V), generator=g, device="cuda").argsort(1)[:, :K].contiguous()
    t = randn(g, T, K, sigma=3.0)
    x.scatter_(1, ids, torch.finfo(torch.float32).min)
    op = ops.VocabHead(3, V, "f32", temperature=tau)
    loss, lse = (torch.full((T,), 9.0, device="cuda") for _ in range(2))
    op.distill(shards_of(x, 3), ids, t, loss, lse)
    logp, _, _ = stats64(x, tau)
    logq = torch.log_softmax(t.double() / tau, 1)
    want = in_f32(tau ** 2 * (logq.exp() * (logq - logp.gather(1, ids))).sum(1))
    assert torch.isfinite(want).all() == (tau <= 1)
    # shares are good to 8 E of (t - max) / tau and their sum, K of them to K E: all relative here
    tmag = (t.double().amax(1) - t.double().amin(1)) / tau
    same(loss, want, (K + 64 + 8 * tmag) * E * size(want), "loss")


@pytest.mark.parametrize("tau", [0.7, 1.0, 2.0])
@pytest.mark.parametrize("shift", [700.0, -700.0, 11.0])
def test_lse_is_rounded_once(ops, tau, shift):
    """lse within half a unit of its last place of the 64-bit one, and the loss of the row's sum: a gradient of binary32
    logits has lse's error in every probability."""
    T, V = 300, 1000
    x = randn(gen(131), T, V, sigma=2.0, mean=shift)
    op = ops.VocabHead(3, V, "f32", temperature=tau)
    lp, lse, loss, lse2 = (torch.full((T,), 9.0, device="cuda") for _ in range(4))
    op.logprobs(shards_of(x, 3), torch.zeros(T, dtype=torch.int64, device="cuda"), lp, lse)
    ids = torch.arange(4, device="cuda").expand(T, 4).contiguous()
    op.distill(shards_of(x, 3), ids, torch.zeros((T, 4), device="cuda"), loss, lse2)
    _, want, _ = stats64(x, torch.tensor(tau, dtype=torch.float32).item())   # the handle's temperature is a binary32 one
    half = 2.0 ** (torch.floor(torch.log2(want.abs())) - 24)
    for got in (lse, lse2):
        same(got, want, half + sum_loss(V), "lse")
