"""What is measured of the model operators: the block end (BlockNorm) and the
vocabulary-parallel head (VocabHead: log probabilities, distillation).

A case is a dict of plain values.  ``prepare`` makes what a program has in hand
before the call (activations, logits, weights, output buffers and, where
``own`` is set, the operator's handle); ``run`` is one pass.  Where ``own`` is
false the pass is the operator's plain form in elementary torch operations, in
32 bits and rounded once at the end; ``exact`` is the definition in 64 bits.
"""

import math

import torch

own = False

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-6
_SCALE = 0.5          # residual scale of the block ends
_HANDLES = {}         # one handle per configuration, as a program keeps it


def listed():
    return [
        # One new token of a served model: R = 8 partial products of the output projection summed,
        # normalised before and after; latency alone counts.
        dict(name="norm_token", op="norm", R=8, T=1, D=4096, dtype="bf16", residual="bf16", param="bf16",
             post=True, groups=0, copies=1, save=False),
        # Training forward over one micro-batch with a 32-bit residual stream and a learned gate per
        # channel; every rank gets its own copy of the normalised rows, the sum is kept for backward.
        dict(name="norm_train", op="norm", R=4, T=8192, D=4096, dtype="bf16", residual="f32", param="f32",
             post=True, groups=1, copies=4, save=True),
        # Rows of odd width and count: no row starts on a vector boundary; one gate row per sequence.
        dict(name="norm_odd", op="norm", R=3, T=1023, D=5001, dtype="f32", residual="f32", param="f32",
             post=True, groups=33, copies=1, save=True),
        # Backward of a wide block end: eight partial gradients summed, weight and gate gradients.
        dict(name="norm_backward", op="norm_backward", R=8, T=4096, D=8192, dtype="bf16", residual="bf16",
             param="bf16", post=True, groups=1, copies=1),
        # Backward of a short ragged batch in half precision, gated per sequence.
        dict(name="norm_backward_small", op="norm_backward", R=2, T=96, D=1538, dtype="f16", residual="f32",
             param="f32", post=True, groups=8, copies=2),
        # One sampled token: log probability, entropy and 20 alternatives over eight vocabulary shards.
        dict(name="logprobs_token", op="logprobs", R=8, T=1, V=131072, dtype="bf16", top=20, tau=1.0, masked=False),
        # Scoring given text: many rows, a few alternatives each.
        dict(name="logprobs_score", op="logprobs", R=8, T=4096, V=131072, dtype="bf16", top=5, tau=1.0, masked=False),
        # Constrained decoding of a small batch: logits in 32 bits, odd vocabulary, most of it masked in
        # some rows, all of it in a few.
        dict(name="logprobs_masked", op="logprobs", R=3, T=61, V=50021, dtype="f32", top=32, tau=0.7, masked=True),
        # Policy gradient: gradients of the log probability and the entropy for every logit.
        dict(name="logprobs_backward", op="logprobs_backward", R=4, T=2048, V=65536, dtype="f16", tau=1.0,
             masked=True),
        # Distillation of a batch, loss and normaliser.
        dict(name="distill", op="distill", R=8, T=4096, V=131072, dtype="bf16", K=64, tau=2.0),
        # The logits' gradient of a batch with an odd vocabulary, whose rows start off the vector boundary.
        dict(name="distill_backward", op="distill_backward", R=8, T=4096, V=100003, dtype="bf16", K=64, tau=2.0),
        # A whole small training step, loss and gradient, odd everywhere.
        dict(name="distill_step", op="distill_step", R=5, T=129, V=32003, dtype="f16", K=16, tau=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    op = rng.choice(["norm", "norm_backward", "logprobs", "logprobs_backward", "distill", "distill_backward",
                     "distill_step"])
    R = _log_int(rng, 1, 32)
    if op.startswith("norm"):
        D = _log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            D = (D + 63) // 64 * 64
        G = rng.choice([0, 1, 1, _log_int(rng, 2, 64)])
        most = 5e8 / (_BYTES[dtype] * (R + 6) * D)
        T = _log_int(rng, 1, max(1, min(65536, int(most))))
        if G > 1:
            T = max(1, T // G) * G
        case = dict(op=op, R=R, T=T, D=D, dtype=dtype, residual=rng.choice([dtype, "f32"]),
                    param=rng.choice([dtype, "f32"]), post=rng.random() < 0.7, groups=G,
                    copies=rng.choice([1, R]) if R <= 8 else 1)
        if op == "norm":
            case["save"] = rng.random() < 0.5
        return case
    V = _log_int(rng, max(64, R), 200000)
    if rng.random() < 0.5:
        V = (V + 127) // 128 * 128
    T = _log_int(rng, 1, max(1, min(8192, int(5e8 / (_BYTES[dtype] * V)))))
    case = dict(op=op, R=R, T=T, V=V, dtype=dtype, tau=rng.choice([1.0, 1.0, 0.7, 2.0]))
    if op.startswith("logprobs"):
        case["masked"] = rng.random() < 0.5
        if op == "logprobs":
            case["top"] = rng.choice([0, 1, 5, 20, 32])
    else:
        case["K"] = min(V, _log_int(rng, 1, 256))
    return case


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 12345)
    return g


def _normal(g, shape, dtype, sigma=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma + mean).to(dtype)


def _shards(full, R):
    """The column shards that R ranks hold: shard r is [r C, min((r + 1) C, V)), C = ceil(V / R)."""
    V = full.shape[1]
    C = -(-V // R)
    return [full[:, min(r * C, V):min((r + 1) * C, V)].contiguous() for r in range(R)]


def _handle(key, make):
    if key not in _HANDLES:
        _HANDLES[key] = make()
    return _HANDLES[key]


def _norm_handle(c):
    from ring_allreduce_gb300 import BlockNorm
    key = ("norm", c["R"], c["D"], c["dtype"], c["residual"], c["param"])
    return _handle(key, lambda: BlockNorm(c["R"], c["D"], c["dtype"], residual_dtype=c["residual"],
                                          param_dtype=c["param"], eps=_EPS, scale=_SCALE))


def _vocab_handle(c):
    from ring_allreduce_gb300 import VocabHead
    key = ("vocab", c["R"], c["V"], c["dtype"], c["tau"])
    return _handle(key, lambda: VocabHead(c["R"], c["V"], c["dtype"], temperature=c["tau"]))


def _prepare_norm(c, g):
    R, T, D, G = c["R"], c["T"], c["D"], c["groups"]
    dt, rdt, pdt = _TORCH[c["dtype"]], _TORCH[c["residual"]], _TORCH[c["param"]]
    s = dict(case=c, pre=_normal(g, (D,), pdt, 0.1, 1.0), post=_normal(g, (D,), pdt, 0.1, 1.0) if c["post"] else None,
             gate=_normal(g, (G, D), pdt, 0.3, 0.5) if G else None)
    # one allocation for the ranks' buffers, one row range per rank
    if c["op"] == "norm":
        s["parts"] = torch.empty((R, T, D), dtype=dt, device="cuda")
        for r in range(R):
            s["parts"][r] = _normal(g, (T, D), dt, 1.0 / math.sqrt(R))
        s["residual"] = _normal(g, (T, D), rdt, 2.0)
        s["z"] = torch.empty((c["copies"], T, D), dtype=dt, device="cuda")
        s["residual_out"] = torch.empty((T, D), dtype=rdt, device="cuda")
        s["total"] = torch.empty((T, D), dtype=dt, device="cuda") if c["save"] else None
        s["rstd"] = torch.empty((2, T), dtype=torch.float32, device="cuda") if c["save"] else None
    else:
        s["grad_parts"] = torch.empty((R, T, D), dtype=dt, device="cuda")
        for r in range(R):
            s["grad_parts"][r] = _normal(g, (T, D), dt, 1.0 / math.sqrt(R))
        s["grad_residual_out"] = _normal(g, (T, D), rdt)
        s["total"] = _normal(g, (T, D), dt)
        s["residual_out"] = _normal(g, (T, D), rdt, 2.0)
        s["rstd"] = torch.empty((2, T), dtype=torch.float32, device="cuda")
        s["rstd"][0] = (s["total"].float().square().mean(1) + _EPS).rsqrt()
        s["rstd"][1] = (s["residual_out"].float().square().mean(1) + _EPS).rsqrt()
        s["grad_in"] = torch.empty((c["copies"], T, D), dtype=dt, device="cuda")
        s["grad_residual"] = torch.empty((T, D), dtype=rdt, device="cuda")
        s["grad_pre"] = torch.empty(D, dtype=torch.float32, device="cuda")
        s["grad_post"] = torch.empty(D, dtype=torch.float32, device="cuda") if c["post"] else None
        s["grad_gate"] = torch.empty((G, D), dtype=torch.float32, device="cuda") if G else None
    if own:
        s["op"] = _norm_handle(c)
    return s


def _logits(c, g):
    """Rows of logits: a broad normal bulk, with a few tokens per row that stand out."""
    T, V = c["T"], c["V"]
    x = torch.randn((T, V), generator=g, device="cuda").mul_(2.0)
    hot = torch.randint(V, (T, 16), generator=g, device="cuda")
    x.scatter_(1, hot, torch.randn((T, 16), generator=g, device="cuda") * 2.0 + 11.0)
    return x, hot


def _prepare_logprobs(c, g):
    T, V, dt = c["T"], c["V"], _TORCH[c["dtype"]]
    x, hot = _logits(c, g)
    targets = torch.where(torch.rand(T, generator=g, device="cuda") < 0.8, hot[:, 0],
                          torch.randint(V, (T,), generator=g, device="cuda"))
    if c["masked"]:
        # a third of the rows allow only a narrow band of tokens, every 20th row none at all; some
        # positions have no target
        rows = torch.arange(T, device="cuda")
        start = torch.randint(V, (T, 1), generator=g, device="cuda")
        j = torch.arange(V, device="cuda")
        away = ((j - start) % V >= 1 + V // 500) & (rows % 3 == 0)[:, None] | (rows % 20 == 7)[:, None]
        x.masked_fill_(away, -math.inf)
        targets = torch.where(rows % 11 == 4, torch.full_like(targets, -1), targets)
    shards = _shards(x.to(dt), c["R"])
    del x
    s = dict(case=c, shards=shards, targets=targets)
    f32 = dict(dtype=torch.float32, device="cuda")
    if c["op"] == "logprobs":
        K = c["top"]
        s.update(logprob=torch.empty(T, **f32), lse=torch.empty(T, **f32), entropy=torch.empty(T, **f32),
                 top_ids=torch.empty((T, K), dtype=torch.int64, device="cuda") if K else None,
                 top_logprobs=torch.empty((T, K), **f32) if K else None)
    else:
        lse, entropy = [], []
        for k in range(0, T, 512):
            lp, l, h = _plain_logp([q[k:k + 512] for q in shards], c["tau"])
            lse.append(l)
            entropy.append(h)
        s.update(lse=torch.cat(lse), entropy=torch.cat(entropy), grad_logprob=_normal(g, (T,), torch.float32),
                 grad_entropy=_normal(g, (T,), torch.float32, 0.1), grads=[torch.empty_like(q) for q in shards])
    if own:
        s["op"] = _vocab_handle(c)
    return s


def _prepare_distill(c, g):
    T, V, K, dt = c["T"], c["V"], c["K"], _TORCH[c["dtype"]]
    x, _ = _logits(c, g)
    # the teacher's K tokens: distinct ids, falling logits; the student half agrees with them
    ids = (torch.randint(V, (T, 1), generator=g, device="cuda") +
           torch.randint(1, V // K + 1, (T, K), generator=g, device="cuda").cumsum(1)) % V
    teacher = 14.0 - torch.rand((T, K), generator=g, device="cuda").mul_(-1).add_(1).log_().neg_().cumsum(1)
    x.scatter_(1, ids, teacher * 0.8 + torch.randn((T, K), generator=g, device="cuda"))
    rows = torch.arange(T, device="cuda")
    ids = torch.where((rows % 17 == 5)[:, None], torch.full_like(ids, -1), ids)   # padding rows: no teacher
    shards = _shards(x.to(dt), c["R"])
    s = dict(case=c, shards=shards, ids=ids, teacher=teacher)
    f32 = dict(dtype=torch.float32, device="cuda")
    if c["op"] != "distill_backward":
        s.update(loss=torch.empty(T, **f32), lse=torch.empty(T, **f32))
    else:
        s["lse"] = torch.cat([_plain_logp([q[k:k + 512] for q in shards], c["tau"])[1] for k in range(0, T, 512)])
    if c["op"] != "distill":
        s.update(grad_loss=_normal(g, (T,), torch.float32, 0.1, 1.0), grads=[torch.empty_like(q) for q in shards])
    if own:
        s["op"] = _vocab_handle(c)
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"].startswith("norm"):
        return _prepare_norm(case, g)
    if case["op"].startswith("logprobs"):
        return _prepare_logprobs(case, g)
    return _prepare_distill(case, g)


# ------------------------------------------------------- one pass, both forms

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_norm(s):
    s["op"].forward(s["parts"], s["residual"], s["pre"], s["z"], s["residual_out"], post_weight=s["post"],
                    gate=s["gate"], total=s["total"], rstd=s["rstd"])
    return s["z"], s["residual_out"], s["total"], s["rstd"]


def _own_norm_backward(s):
    s["op"].backward(s["grad_parts"], s["grad_residual_out"], s["residual_out"], s["rstd"], s["pre"], s["grad_in"],
                     s["grad_residual"], s["grad_pre"], post_weight=s["post"], gate=s["gate"], total=s["total"],
                     grad_post_weight=s["grad_post"], grad_gate=s["grad_gate"])
    return s["grad_in"], s["grad_residual"], s["grad_pre"], s["grad_post"], s["grad_gate"]


def _own_logprobs(s):
    s["op"].logprobs(s["shards"], s["targets"], s["logprob"], s["lse"], s["entropy"], s["top_ids"],
                     s["top_logprobs"])
    return s["logprob"], s["lse"], s["entropy"], s["top_ids"], s["top_logprobs"]


def _own_logprobs_backward(s):
    s["op"].logprobs_backward(s["shards"], s["targets"], s["lse"], s["grad_logprob"], s["grads"],
                              entropy=s["entropy"], grad_entropy=s["grad_entropy"])
    return s["grads"]


def _own_distill(s):
    s["op"].distill(s["shards"], s["ids"], s["teacher"], s["loss"], s["lse"])
    return s["loss"], s["lse"]


def _own_distill_backward(s):
    s["op"].distill_backward(s["shards"], s["ids"], s["teacher"], s["lse"], s["grad_loss"], s["grads"])
    return s["grads"]


def _own_distill_step(s):
    return _own_distill(s), _own_distill_backward(s)


def _rms(x):
    return (x.square().mean(1) + _EPS).rsqrt()


def _gate_rows(s, T):
    return s["gate"].float().repeat_interleave(T // s["gate"].shape[0], 0) if s["gate"] is not None else 1.0


def _plain_norm(s):
    c = s["case"]
    dt, rdt = _TORCH[c["dtype"]], _TORCH[c["residual"]]
    total = s["parts"].float().sum(0)
    r1 = _rms(total) if c["post"] else torch.zeros(c["T"], device="cuda")
    y = total * r1[:, None] * s["post"].float() if c["post"] else total
    h = s["residual"].float() + _SCALE * _gate_rows(s, c["T"]) * y
    r2 = _rms(h)
    z = (h * r2[:, None] * s["pre"].float()).to(dt)
    saved = (total.to(dt), torch.stack([r1, r2])) if c["save"] else (None, None)
    return (z.expand(c["copies"], -1, -1).contiguous(), h.to(rdt)) + saved


def _plain_norm_backward(s):
    c = s["case"]
    dt, rdt = _TORCH[c["dtype"]], _TORCH[c["residual"]]
    r1, r2 = s["rstd"][0][:, None], s["rstd"][1][:, None]
    dz, x2, total = s["grad_parts"].float().sum(0), s["residual_out"].float() * r2, s["total"].float()
    wdz = dz * s["pre"].float()
    e = s["grad_residual_out"].float() + r2 * (wdz - x2 * (wdz * x2).mean(1, keepdim=True))
    dy = e * (_SCALE * _gate_rows(s, c["T"]))
    grad_post = None
    y, ds = total, dy
    if c["post"]:
        x1 = total * r1
        y = x1 * s["post"].float()
        wdy = dy * s["post"].float()
        ds = r1 * (wdy - x1 * (wdy * x1).mean(1, keepdim=True))
        grad_post = (dy * x1).sum(0)
    G = c["groups"]
    grad_gate = (_SCALE * y * e).view(G, -1, c["D"]).sum(1) if G else None
    return (ds.to(dt).expand(c["copies"], -1, -1).contiguous(), e.to(rdt), (dz * x2).sum(0), grad_post, grad_gate)


def _plain_logp(shards, tau):
    """log p [T, V], lse and entropy; a row with nothing left has lse -inf, log p -inf and entropy 0."""
    x = torch.cat(shards, 1).float().div_(tau)
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    total = (x - m).exp_().sum(1, keepdim=True)
    lse = m + total.log()
    # the logarithm of a whole row's sum is taken apart from its largest logit
    logp = torch.where(lse == -math.inf, -math.inf, (x - m) - total.log())
    p = logp.exp()
    entropy = -(p * torch.where(p > 0, logp, 0.0)).sum(1)
    return logp, lse[:, 0], entropy


def _top(x, K):
    """The K greatest of each row, ties to the lowest index: a whole number that orders by value, then by index."""
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64) * (1 << 32)
    order += (1 << 31) - 1 - torch.arange(x.shape[1], device=x.device)
    return (1 << 31) - 1 - (order.topk(K, dim=1).values & 0xFFFFFFFF)


def _plain_logprobs(s):
    c = s["case"]
    logp, lse, entropy = _plain_logp(s["shards"], c["tau"])
    known = s["targets"] >= 0
    logprob = torch.where(known, logp.gather(1, s["targets"].clamp(min=0)[:, None])[:, 0], 0.0)
    if not c["top"]:
        return logprob, lse, entropy, None, None
    ids = _top(torch.cat(s["shards"], 1).float(), c["top"])
    return logprob, lse, entropy, ids, logp.gather(1, ids)


def _split(grad, shards):
    return list(x.to(shards[0].dtype).contiguous() for x in grad.split([q.shape[1] for q in shards], 1))


def _plain_p(s):
    x = torch.cat(s["shards"], 1).float().div_(s["case"]["tau"])
    lse = s["lse"][:, None]
    logp = x - torch.where(lse == -math.inf, 0.0, lse)
    return logp, logp.exp(), lse > -math.inf


def _plain_logprobs_backward(s):
    logp, p, some = _plain_p(s)
    g, gh = s["grad_logprob"][:, None], s["grad_entropy"][:, None]
    known = (s["targets"] >= 0)[:, None]
    g = torch.where(known, g, 0.0)
    grad = -(p * (g + gh * (torch.where(p > 0, logp, 0.0) + s["entropy"][:, None])))
    grad.scatter_add_(1, s["targets"].clamp(min=0)[:, None], g)
    grad = torch.where(some, grad, 0.0).div_(s["case"]["tau"])
    return _split(grad, s["shards"])


def _plain_q(s):
    tau, ids = s["case"]["tau"], s["ids"]
    t = torch.where(ids >= 0, s["teacher"].float() / tau, -math.inf)
    m = t.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = (t - m).exp()
    total = e.sum(1, keepdim=True)
    some = total > 0
    return torch.where(some, e / total, 0.0), torch.where(some, t - m - total.log(), 0.0), some


def _plain_distill(s):
    logp, lse, _ = _plain_logp(s["shards"], s["case"]["tau"])
    q, logq, _ = _plain_q(s)
    at = logp.gather(1, s["ids"].clamp(min=0))
    loss = torch.where(q > 0, q * (logq - at), 0.0).sum(1) * s["case"]["tau"] ** 2
    return loss, lse


def _plain_distill_backward(s):
    _, p, some = _plain_p(s)
    q, _, taught = _plain_q(s)
    grad = torch.where(taught, p, 0.0).scatter_add_(1, s["ids"].clamp(min=0), -q)
    grad = torch.where(some, grad, 0.0).mul_(s["grad_loss"][:, None] * s["case"]["tau"])
    return _split(grad, s["shards"])


def _plain_distill_step(s):
    loss, lse = _plain_distill(s)
    return (loss, lse), _plain_distill_backward(dict(s, lse=lse))


_own = dict(norm=_own_norm, norm_backward=_own_norm_backward, logprobs=_own_logprobs,
            logprobs_backward=_own_logprobs_backward, distill=_own_distill, distill_backward=_own_distill_backward,
            distill_step=_own_distill_step)
_plain = dict(norm=_plain_norm, norm_backward=_plain_norm_backward, logprobs=_plain_logprobs,
              logprobs_backward=_plain_logprobs_backward, distill=_plain_distill,
              distill_backward=_plain_distill_backward, distill_step=_plain_distill_step)


# ------------------------------------------------------------------- work

def work(case):
    """Bytes that a pass cannot do without (every input read once, every output written once) and its operations."""
    c = case
    b = _BYTES[c["dtype"]]
    if c["op"].startswith("norm"):
        n, rb, pb = c["T"] * c["D"], _BYTES[c["residual"]], _BYTES[c["param"]]
        params = c["D"] * (1 + c["post"] + c["groups"])
        if c["op"] == "norm":
            moved = n * b * (c["R"] + c["copies"] + c["save"]) + 2 * n * rb + 8 * c["T"] * c["save"]
            return dict(bytes=moved + params * pb, flops=n * (c["R"] + 13))
        need = c["post"] or c["groups"] > 0
        moved = n * b * (c["R"] + c["copies"] + need) + 3 * n * rb + 8 * c["T"]
        return dict(bytes=moved + params * (pb + 4), flops=n * (c["R"] + 26))
    n, T = c["T"] * c["V"], c["T"]
    if c["op"] == "logprobs":
        return dict(bytes=n * b + T * (8 + 12 + 12 * c["top"]), flops=6 * n)
    if c["op"] == "logprobs_backward":
        return dict(bytes=2 * n * b + T * (8 + 16), flops=7 * n)
    if c["op"] == "distill":
        return dict(bytes=n * b + T * (12 * c["K"] + 8), flops=3 * n)
    if c["op"] == "distill_backward":
        return dict(bytes=2 * n * b + T * (12 * c["K"] + 8), flops=4 * n)
    return dict(bytes=3 * n * b + T * (24 * c["K"] + 16), flops=7 * n)


# ------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "norm_backward":
        return _exact_norm_backward(s)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    if case["op"] == "logprobs_backward":
        return _exact_logprobs_backward(s)
    if case["op"] == "distill":
        return _exact_distill(s)
    if case["op"] == "distill_backward":
        return _exact_distill_backward(s, s["lse"].double())
    loss, lse = _exact_distill(s)
    return (loss, lse), _exact_distill_backward(s, lse)


def _exact_norm(s):
    c = s["case"]
    T, D, G = c["T"], c["D"], c["groups"]
    total = torch.zeros((T, D), dtype=torch.float64, device="cuda")
    for r in range(c["R"]):
        total += s["parts"][r].double()
    r1 = torch.zeros(T, dtype=torch.float64, device="cuda")
    y = total.clone()
    if c["post"]:
        r1 = 1.0 / torch.sqrt((total ** 2).sum(1) / D + _EPS)
        y = y * r1.unsqueeze(1) * s["post"].double()
    if G:
        y = (y.reshape(G, T // G, D) * s["gate"].double().unsqueeze(1)).reshape(T, D)
    h = s["residual"].double() + _SCALE * y
    r2 = 1.0 / torch.sqrt((h ** 2).sum(1) / D + _EPS)
    z = h * s["pre"].double() * r2.unsqueeze(1)
    out = (torch.stack([z] * c["copies"]), h)
    return out + ((total, torch.stack([r1, r2])) if c["save"] else (None, None))


def _exact_norm_backward(s):
    c = s["case"]
    T, D, G = c["T"], c["D"], c["groups"]
    dz = torch.zeros((T, D), dtype=torch.float64, device="cuda")
    for r in range(c["R"]):
        dz += s["grad_parts"][r].double()
    r1, r2 = (s["rstd"][k].double().unsqueeze(1) for k in (0, 1))
    x2 = s["residual_out"].double() * r2
    a = dz * s["pre"].double()
    e = s["grad_residual_out"].double() + r2 * a - r2 * x2 * ((a * x2).sum(1, keepdim=True) / D)
    gate = s["gate"].double().unsqueeze(1).expand(G, T // G, D).reshape(T, D) if G else 1.0
    total = s["total"].double()
    dy = _SCALE * gate * e
    grad_post, branch, ds = None, total, dy
    if c["post"]:
        x1 = total * r1
        branch = x1 * s["post"].double()
        b = dy * s["post"].double()
        ds = r1 * b - r1 * x1 * ((b * x1).sum(1, keepdim=True) / D)
        grad_post = (dy * x1).sum(0)
    grad_gate = (_SCALE * branch * e).reshape(G, T // G, D).sum(1) if G else None
    return torch.stack([ds] * c["copies"]), e, (dz * x2).sum(0), grad_post, grad_gate


def _blocks(s):
    """The rows in blocks that fit 64-bit copies: (first row, last row, logits / tau)."""
    T, V = s["case"]["T"], s["case"]["V"]
    step = max(1, (1 << 27) // V)
    for k in range(0, T, step):
        yield k, min(T, k + step), torch.cat([q[k:k + step].double() for q in s["shards"]], 1) / s["case"]["tau"]


def _exact_logprobs(s):
    K, got = s["case"]["top"], []
    for lo, hi, x in _blocks(s):
        lse = torch.logsumexp(x, 1)
        empty = torch.isinf(lse)
        lp = torch.where(empty[:, None], -math.inf, x - lse[:, None])
        H = -torch.nan_to_num(lp.exp() * lp, nan=0.0).sum(1)
        t = s["targets"][lo:hi]
        at = torch.where(t < 0, 0.0, lp.gather(1, t.clamp(min=0)[:, None]).squeeze(1))
        best = torch.sort(lp, 1, descending=True).values[:, :K] if K else None
        got.append((at, lse, H, best))
    cols = [torch.cat(v) if v[0] is not None else None for v in zip(*got)]
    return cols[0], cols[1], cols[2], None, cols[3]


def _cut(rows, s):
    grad = torch.cat(rows)
    C = -(-s["case"]["V"] // s["case"]["R"])
    edges = [min(r * C, grad.shape[1]) for r in range(s["case"]["R"] + 1)]
    return [grad[:, a:b] for a, b in zip(edges, edges[1:])]


def _exact_logprobs_backward(s):
    rows = []
    for lo, hi, x in _blocks(s):
        lse, H, t = s["lse"][lo:hi].double(), s["entropy"][lo:hi].double(), s["targets"][lo:hi]
        g, gh = s["grad_logprob"][lo:hi].double(), s["grad_entropy"][lo:hi].double()
        g = torch.where(t < 0, 0.0, g)
        empty = torch.isinf(lse)
        lp = x - torch.where(empty, 0.0, lse)[:, None]
        p = lp.exp()
        grad = -g[:, None] * p - gh[:, None] * (torch.nan_to_num(p * lp, nan=0.0) + p * H[:, None])
        grad[torch.arange(hi - lo, device="cuda"), t.clamp(min=0)] += g
        rows.append((grad / s["case"]["tau"]).masked_fill_(empty[:, None], 0.0))
    return _cut(rows, s)


def _exact_q(s, lo, hi):
    ids = s["ids"][lo:hi]
    t = (s["teacher"][lo:hi].double() / s["case"]["tau"]).masked_fill(ids < 0, -math.inf)
    return ids, torch.nan_to_num(torch.softmax(t, 1), nan=0.0)


def _exact_distill(s):
    loss, lse = [], []
    for lo, hi, x in _blocks(s):
        ids, q = _exact_q(s, lo, hi)
        z = torch.logsumexp(x, 1)
        at = x.gather(1, ids.clamp(min=0)) - z[:, None]
        loss.append(s["case"]["tau"] ** 2 * (torch.xlogy(q, q) - torch.where(q > 0, q * at, 0.0)).sum(1))
        lse.append(z)
    return torch.cat(loss), torch.cat(lse)


def _exact_distill_backward(s, lse):
    rows = []
    for lo, hi, x in _blocks(s):
        ids, q = _exact_q(s, lo, hi)
        grad = (x - lse[lo:hi, None]).exp()
        grad = grad * (q.sum(1, keepdim=True) > 0)
        grad.scatter_add_(1, ids.clamp(min=0), -q)
        rows.append(grad * (s["grad_loss"][lo:hi].double() * s["case"]["tau"])[:, None])
    return _cut(rows, s)
