"""examples/distill_step.py: the operators and the AllReduce in one training
loop, its gradients against torch's own, and the loss falling."""

import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def example():
    from ring_allreduce_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import distill_step
    return distill_step


def test_gradients_match_autograd(example):
    """One step's loss and gradients against autograd on the same network in 64
    bits.  The step's activations, logits and their gradients are bfloat16
    (unit roundoff 2^-8): every gradient passes through at most eight such
    roundings, each of independent elements, so 2^-5 of the gradient's norm."""
    st = example.Student()
    act, residual, ids, teacher = example.teacher_batch(3)
    loss, grads = st.step(act, residual, ids, teacher)
    p = {k: v.double().requires_grad_() for k, v in st.params.items()}
    T = act.shape[0]
    a = act.view(T, example.RANKS, -1).transpose(0, 1).double()
    total = torch.bmm(a, p["proj"]).sum(0)
    y = total * (total.square().mean(1, keepdim=True) + 1e-6).rsqrt() * p["post"]
    h = residual.double() + p["gate"] * y
    z = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * p["pre"]
    logp = torch.log_softmax(z @ p["head"].T, 1)
    q = torch.softmax(teacher.double(), 1)
    want = (q * (q.log() - logp.gather(1, ids))).sum(1)
    (want.sum() / (T * example.REPLICAS)).backward()
    assert (loss.double() - want).norm() <= 2.0 ** -5 * want.norm()
    for k, v in p.items():
        err = (grads[k].double() - v.grad).norm() / v.grad.norm()
        assert err <= 2.0 ** -5, (k, err.item())


def test_training_lowers_the_loss(example):
    losses, scores = example.train(steps=12)
    assert losses[-1] < 0.8 * losses[0]
    assert all(b < a * 1.05 for a, b in zip(losses, losses[1:]))
    assert scores["entropy"] > 0 and scores["logprob"] < 0
