"""The operators of a tensor-parallel block in a row, as examples/feed_forward_step.py
has them: block end, feed-forward, block end, and back through codes."""

import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import feed_forward_step
    return feed_forward_step


def reference(example, block, parts, h0, grad_y, grad_h2):
    """Outputs and gradients of the same network in 64 bits, by autograd."""
    p = {k: [w.double().requires_grad_() for w in ws] for k, ws in block.weights.items()}
    n = {k: v.double().requires_grad_() for k, v in block.norms.items()}
    parts, h0 = parts.double().requires_grad_(), h0.double().requires_grad_()

    def end(parts, h, post, pre):
        S = parts.sum(0)
        h = h + S * (S.square().mean(1, keepdim=True) + example.EPS).rsqrt() * post
        return h * (h.square().mean(1, keepdim=True) + example.EPS).rsqrt() * pre, h

    z, h1 = end(parts, h0, n["post1"], n["pre1"])
    mid = torch.stack([(torch.nn.functional.silu(z @ g.T) * (z @ u.T)) @ d
                       for g, u, d in zip(p["gate"], p["up"], p["down"])])
    y, h2 = end(mid, h1, n["post2"], n["pre2"])
    ((y * grad_y.double()).sum() + (h2 * grad_h2.double()).sum()).backward()
    return y, h2, parts.grad[0], h0.grad, p, n


def test_gradients_match_autograd(example):
    """Outputs pass through at most eight roundings to bfloat16 (2^-8 each, of
    independent elements): 2^-5 of the norm.  The gradients, through as many
    again, and through six kept tensors: a code is off by at most half a
    scale, 1/254 of the largest of 128 values, of 1/sqrt(3) of that in the
    root mean square; the largest of 128 normal values is below five standard
    deviations in all but one group in 10^4, so each kept tensor is off by less than
    5 / (254 sqrt 3) = 1.2 % of its norm, and it enters a gradient at most twice
    (a product and a norm's correction): 2^-4 + 12 x 1.2 % = 21 %.  As the errors are independent their
    squares add: sqrt(12) x 1.2 % + 2^-5 < 2^-3."""
    block = example.Block(3)
    T = example.TOKENS
    s = block.buffers(T)
    parts, h0, _ = example.batch(5)
    g = torch.Generator(device="cuda").manual_seed(9)
    grad_y = torch.randn((T, example.DIM), generator=g, device="cuda").to(example.DT)
    grad_h2 = torch.randn((T, example.DIM), generator=g, device="cuda")
    y, h2 = (t.clone() for t in block.forward(s, parts, h0))
    for k in ("z", "y", "h1", "h2", "total", "parts"):   # nothing but codes and norm factors is needed for backward
        s[k].fill_(float("nan"))
    for t in s["hidden"]:
        t.fill_(float("nan"))
    grad_part, grad_h0 = block.backward(s, grad_y, grad_h2)
    wy, wh2, wpart, wh0, p, n = reference(example, block, parts, h0, grad_y, grad_h2)

    def near(got, want, most, what):
        err = ((got.double() - want).norm() / want.norm()).item()
        assert err <= most, (what, err)

    near(y, wy, 2.0 ** -5, "y")
    near(h2, wh2, 2.0 ** -5, "h2")
    near(grad_part, wpart, 2.0 ** -3, "grad_part")
    near(grad_h0, wh0, 2.0 ** -3, "grad_h0")
    for k, ws in p.items():
        for r, w in enumerate(ws):
            near(s["grads"][k][r], w.grad, 2.0 ** -3, (k, r))
    for k, v in n.items():
        near(s["grads"][k], v.grad, 2.0 ** -3, k)


def test_captured_step_replays(example):
    """The whole step in a CUDA graph gives what it gives outside, on inputs that came later."""
    block = example.Block(4)
    T = example.TOKENS
    s = block.buffers(T)
    parts, h0, _ = example.batch(6)
    grad_y = torch.zeros((T, example.DIM), dtype=example.DT, device="cuda")

    def step():
        y, h2 = block.forward(s, parts, h0)
        return [y, h2, *block.backward(s, grad_y, None)]

    step()   # the block ends' workspaces
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(2):
        parts.normal_()
        h0.normal_()
        grad_y.normal_()
        graph.replay()
        got = [t.clone() for t in outs + s["grads"]["gate"] + s["grads"]["down"]]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, outs + s["grads"]["gate"] + s["grads"]["down"]))


def test_example_runs(example):
    losses = example.train(3)
    assert len(losses) == 3 and all(v == v and v < 1e6 for v in losses)
