"""One training step of a tensor-parallel block on one GPU, its activations kept
in 8 bits between the forward and the backward pass.

Four tensor-parallel ranks hold slices of a feed-forward block that stands
between two block ends.  Forward is

  z, h1 = BlockNorm: the ranks' partial products of the layer before summed,
          normed, added to the residual stream h0, normed
  parts = FeedForward: act(z gate^T) (z up^T) down, a partial product a rank
  y, h2 = BlockNorm: the same for these

and what backward reads is kept as codes: both sums and both residual streams
by Checkpoint, the two projections by FeedForward itself.  The normalised rows z
are not kept at all; they come back with the residual stream.  Backward runs
through the same operators in turn, each giving the partial gradients that the next one sums.

    python examples/feed_forward_step.py [steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from ring_allreduce_gb300 import BlockNorm, Checkpoint, FeedForward  # noqa: E402

RANKS, TOKENS, DIM, INNER = 4, 512, 512, 1500
DT, EPS = torch.bfloat16, 1e-6


class Block:
    """Parameters (weights in bfloat16, norms in float32), and a step's buffers."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.first = BlockNorm(RANKS, DIM, "bf16", residual_dtype="f32", param_dtype="f32", eps=EPS)
        self.last = BlockNorm(RANKS, DIM, "bf16", residual_dtype="f32", param_dtype="f32", eps=EPS)
        self.ffn = FeedForward(RANKS, DIM, INNER, "bf16", grad_dtype="f32")
        self.keep_sum = Checkpoint(DIM, "bf16")
        self.keep_stream = Checkpoint(DIM, "f32", normed_dtype="bf16", param_dtype="f32")

        def normal(*shape, sigma):
            return (torch.randn(shape, generator=g, device="cuda") * sigma).to(DT)

        widths = self.ffn.widths
        self.weights = {k: [normal(n, DIM, sigma=s) for n in widths]
                        for k, s in (("gate", DIM ** -0.5), ("up", DIM ** -0.5), ("down", INNER ** -0.5))}
        self.norms = {k: torch.ones(DIM, device="cuda") for k in ("post1", "pre1", "post2", "pre2")}

    def buffers(self, T):
        new = lambda *s, dtype=DT: torch.empty(s, dtype=dtype, device="cuda")   # noqa: E731
        f32 = torch.float32
        s = dict(z=new(1, T, DIM), y=new(1, T, DIM), h1=new(T, DIM, dtype=f32), h2=new(T, DIM, dtype=f32),
                 total=new(T, DIM), rstd1=new(2, T, dtype=f32), rstd2=new(2, T, dtype=f32), parts=new(RANKS, T, DIM),
                 hidden=self.ffn.rows(T), grad_gate=self.ffn.rows(T), grad_up=self.ffn.rows(T),
                 grad_part=new(1, T, DIM), grad_z=new(RANKS, T, DIM), grad_h=new(T, DIM, dtype=f32))
        # all that is left of the activations between the passes
        s["gate"], s["gate_scales"] = self.ffn.codes(T)
        s["up"], s["up_scales"] = self.ffn.codes(T)
        for k in ("total1", "total2", "stream1", "stream2"):
            s[k] = new(T, DIM, dtype=torch.int8), new(T, (DIM + 127) // 128, dtype=f32)
        s["grads"] = {k: [torch.empty(w.shape, device="cuda") for w in ws] for k, ws in self.weights.items()}
        s["grads"].update({k: torch.empty_like(v) for k, v in self.norms.items()})
        return s

    def forward(self, s, parts, h0):
        w, n = self.weights, self.norms
        self.first.forward(parts, h0, n["pre1"], s["z"], s["h1"], post_weight=n["post1"], total=s["total"], rstd=s["rstd1"])
        self.keep_sum.store(s["total"], *s["total1"])
        self.keep_stream.store(s["h1"], *s["stream1"])
        self.ffn.forward(s["z"], w["gate"], w["up"], w["down"], s["hidden"], s["parts"], s["gate"], s["up"],
                         s["gate_scales"], s["up_scales"])
        self.last.forward(s["parts"], s["h1"], n["pre2"], s["y"], s["h2"], post_weight=n["post2"], total=s["total"],
                          rstd=s["rstd2"])
        self.keep_sum.store(s["total"], *s["total2"])
        self.keep_stream.store(s["h2"], *s["stream2"])
        return s["y"][0], s["h2"]

    def backward(self, s, grad_y, grad_h2):
        """The gradients of the layer before's partial products and of h0; the
        parameters' in s["grads"].  From the codes alone: every other buffer of forward's may have been used for something else."""
        w, n, g = self.weights, self.norms, s["grads"]
        self.keep_sum.load(*s["total2"], s["total"])
        self.keep_stream.load(*s["stream2"], s["h2"])
        self.last.backward([grad_y], grad_h2, s["h2"], s["rstd2"], n["pre2"], s["grad_part"], s["grad_h"], g["pre2"],
                           post_weight=n["post2"], total=s["total"], grad_post_weight=g["post2"])
        # the stream between, with the normalised rows that the projections took
        self.keep_stream.load(*s["stream1"], s["h1"], s["rstd1"][1], n["pre1"], s["z"][0])
        self.ffn.backward(s["grad_part"], s["z"], w["gate"], w["up"], w["down"], s["gate"], s["up"], s["hidden"],
                          s["grad_gate"], s["grad_up"], s["grad_z"], g["gate"], g["up"], g["down"], s["gate_scales"],
                          s["up_scales"])
        self.keep_sum.load(*s["total1"], s["total"])
        self.first.backward(s["grad_z"], s["grad_h"], s["h1"], s["rstd1"], n["pre1"], s["grad_part"], s["grad_h"],
                            g["pre1"], post_weight=n["post1"], total=s["total"], grad_post_weight=g["post1"])
        return s["grad_part"][0], s["grad_h"]


def batch(seed):
    """Partial products of the layer before, the residual stream, and a target for the output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    return (r(RANKS, TOKENS, DIM) * RANKS ** -0.5).to(DT), r(TOKENS, DIM), r(TOKENS, DIM)


def train(steps=10, rate=0.2):
    """Mean squared distance of y from the target before every step."""
    block = Block()
    s = block.buffers(TOKENS)
    parts, h0, target = batch(1)
    losses = []
    for _ in range(steps):
        y, _ = block.forward(s, parts, h0)
        off = y.float() - target
        losses.append(off.square().mean())
        block.backward(s, (off * (2.0 / off.numel())).to(DT), None)
        for k, ws in block.weights.items():
            for p, d in zip(ws, s["grads"][k]):
                p.sub_((d * (rate * DIM)).to(DT))
        for k, p in block.norms.items():
            p.sub_(s["grads"][k], alpha=rate * DIM)
    return [v.item() for v in losses]


def main():
    for i, v in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 10)):
        print(f"step {i:3d}  loss {v:.4f}")


if __name__ == "__main__":
    main()
