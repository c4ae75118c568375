"""Distillation of a small tensor-parallel block and head on one GPU: the
framework's operators and its AllReduce in one training loop.

Four tensor-parallel ranks hold slices of a projection and of the vocabulary;
two data-parallel replicas take a micro-batch each.  A step is

  parts[r]  = act[:, r] @ proj[r]             the ranks' partial products
  z         = BlockNorm: their sum, normed, gated, added to the residual, normed
  logits[r] = z @ head[r].T                   vocabulary shards
  loss      = VocabHead.distill against the teacher's top logits, and back,
              the logits' gradient in the logits' place
  dz[r]     = dlogits[r] @ head[r]            partial gradients, summed by BlockNorm.backward
  RingAllReduce over the replicas' gradients, a step of gradient descent

and after training VocabHead.logprobs scores the teacher's first choice.

    python examples/distill_step.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from ring_allreduce_gb300 import BlockNorm, RingAllReduce, VocabHead  # noqa: E402

RANKS, REPLICAS = 4, 2
TOKENS, DIM, INNER, VOCAB, TEACHER_K = 256, 512, 1024, 4000, 16
DT = torch.bfloat16


class Student:
    """Parameters in float32, and one replica's forward and backward."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, sigma):
            return torch.randn(shape, generator=g, device="cuda") * sigma

        self.params = dict(proj=normal(RANKS, INNER // RANKS, DIM, sigma=INNER ** -0.5),
                           head=normal(VOCAB, DIM, sigma=DIM ** -0.5), post=torch.ones(DIM, device="cuda"),
                           pre=torch.ones(DIM, device="cuda"), gate=torch.full((1, DIM), 0.5, device="cuda"))
        self.norm = BlockNorm(RANKS, DIM, "bf16", residual_dtype="f32", param_dtype="f32")
        self.vocab = VocabHead(RANKS, VOCAB, "bf16")

    def logits(self, act, residual):
        """The block's end and the head; what backward needs."""
        p, T = self.params, act.shape[0]
        s = dict(act=act.view(T, RANKS, -1).transpose(0, 1).to(DT), proj=p["proj"].to(DT), head=p["head"].to(DT))
        parts = torch.bmm(s["act"], s["proj"])
        s.update(z=torch.empty((1, T, DIM), dtype=DT, device="cuda"), residual=torch.empty_like(residual),
                 total=torch.empty((T, DIM), dtype=DT, device="cuda"), rstd=torch.empty((2, T), device="cuda"))
        self.norm.forward(parts, residual, p["pre"], s["z"], s["residual"], post_weight=p["post"], gate=p["gate"],
                          total=s["total"], rstd=s["rstd"])
        s["shards"] = [s["z"][0] @ w.T for w in s["head"].split(self.vocab.widths)]
        return s

    def step(self, act, residual, ids, teacher):
        """Loss per token and the parameters' gradients, float32."""
        p, T = self.params, act.shape[0]
        s = self.logits(act, residual)
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        self.vocab.distill(s["shards"], ids, teacher, loss, lse)
        scale = torch.full((T,), 1.0 / (T * REPLICAS), device="cuda")
        self.vocab.distill_backward(s["shards"], ids, teacher, lse, scale, s["shards"])   # in place
        dz = torch.stack([d @ w for d, w in zip(s["shards"], s["head"].split(self.vocab.widths))])
        grads = {k: torch.empty_like(v) for k, v in p.items()}
        torch.mm(torch.cat(s["shards"], 1).T.float(), s["z"][0].float(), out=grads["head"])
        dpart, dres = torch.empty_like(s["z"]), torch.empty_like(residual)
        self.norm.backward(dz, None, s["residual"], s["rstd"], p["pre"], dpart, dres, grads["pre"],
                           post_weight=p["post"], gate=p["gate"], total=s["total"], grad_post_weight=grads["post"],
                           grad_gate=grads["gate"])
        torch.bmm(s["act"].transpose(1, 2).float(), dpart.expand(RANKS, -1, -1).float(), out=grads["proj"])
        return loss, grads


def teacher_batch(seed):
    """Activations, and the top logits of a fixed random teacher for them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    act = torch.randn((TOKENS, INNER), generator=g, device="cuda")
    residual = torch.randn((TOKENS, DIM), generator=g, device="cuda")
    w = torch.randn((INNER, VOCAB), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    top = (act @ w * (2.0 * INNER ** -0.5)).topk(TEACHER_K, 1)
    return act, residual, top.indices, top.values


def train(steps=20, rate=4.0):
    """The mean loss before every step, and the final scores."""
    student = Student()
    batches = [teacher_batch(100 + r) for r in range(REPLICAS)]
    n = sum(v.numel() for v in student.params.values())
    buckets = [torch.empty(n, device="cuda") for _ in range(REPLICAS)]
    losses = []
    with RingAllReduce(REPLICAS, n, "f32", "sum") as ring:
        reduce = ring.prepare("allreduce", buckets, buckets)
        for _ in range(steps):
            mean = 0.0
            for bucket, batch in zip(buckets, batches):
                loss, grads = student.step(*batch)
                torch.cat([grads[k].reshape(-1) for k in student.params], out=bucket)
                mean = mean + loss.mean() / REPLICAS
            reduce()
            for v, d in zip(student.params.values(), buckets[0].split([v.numel() for v in student.params.values()])):
                v.sub_(d.view_as(v), alpha=rate)
            losses.append(mean.item())
    act, residual, ids, _ = batches[0]
    s = student.logits(act, residual)
    logprob, lse, entropy = (torch.empty(TOKENS, device="cuda") for _ in range(3))
    top = torch.empty((TOKENS, 3), dtype=torch.int64, device="cuda")
    top_logprobs = torch.empty((TOKENS, 3), device="cuda")
    student.vocab.logprobs(s["shards"], ids[:, 0].contiguous(), logprob, lse, entropy, top, top_logprobs)
    return losses, dict(logprob=logprob.mean().item(), entropy=entropy.mean().item(),
                        first=(top[:, 0] == ids[:, 0]).float().mean().item())


def main():
    losses, scores = train(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
    for i, v in enumerate(losses):
        print(f"step {i:3d}  distillation loss {v:.4f}")
    print("teacher's first choice: log probability %(logprob).3f, entropy %(entropy).3f, also the student's %(first).2f"
          % scores)


if __name__ == "__main__":
    main()
