"""What is measured of the feed-forward block between two block ends
(FeedForward: gated projections, product, projection back; forward and
backward) and of rows kept in 8 bits (Checkpoint).

A case is a dict of plain values.  ``prepare`` makes what a program has in hand
before the call (activations, weights, kept codes, output buffers and, where
``own`` is set, the operator's handle); ``run`` is one pass.  Where ``own`` is
false the pass is the operator's plain form in elementary torch operations, in
32 bits and rounded once at the end; ``exact`` is the definition in 64 bits.
"""

import math

import torch

own = False

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_GROUP = 128          # columns that share a scale
_LOWEST = 2.0 ** -110  # groups with no magnitude above this are kept as zeros
_HANDLES = {}         # one handle per configuration, as a program keeps it


def listed():
    return [
        # One new token of a small model in two ranks: 25 MB of weights, so latency counts.
        dict(name="forward_token_small", op="forward", R=2, T=1, D=1024, F=4096, dtype="bf16", act="silu",
             copies=1),
        # One new token of a served model in eight ranks: 403 MB of weights read once.
        dict(name="forward_token", op="forward", R=8, T=1, D=4096, F=16384, dtype="bf16", act="silu", copies=8),
        # A decoding batch of odd size.
        dict(name="forward_batch", op="forward", R=8, T=37, D=4096, F=16384, dtype="bf16", act="silu", copies=1),
        # A prompt of odd length in three ranks, whose shards are odd and unequal.
        dict(name="forward_ragged", op="forward", R=3, T=777, D=1544, F=5005, dtype="f16", act="gelu", copies=1),
        # Scoring or a long prompt: bound by the matrix products.
        dict(name="forward_prompt", op="forward", R=4, T=8192, D=4096, F=16384, dtype="bf16", act="silu", copies=1),
        # Backward of a micro-batch from kept 8-bit activations; all gradients.
        dict(name="backward_train", op="backward", R=4, T=4096, D=4096, F=16384, dtype="bf16", act="silu", copies=1),
        # Backward of a short ragged batch in half precision.
        dict(name="backward_ragged", op="backward", R=3, T=321, D=1032, F=2999, dtype="f16", act="gelu", copies=3),
        # Forward, its activations kept in 8 bits, and backward: a whole training step of the block.
        dict(name="step_train", op="step", R=2, T=4096, D=2048, F=8192, dtype="bf16", act="silu", copies=1),
        # The same of a small model, where launches count.
        dict(name="step_small", op="step", R=2, T=200, D=512, F=1400, dtype="bf16", act="gelu", copies=2),
        # A residual stream in 32 bits kept in 8, and brought back with the normalised rows.
        dict(name="keep_train", op="keep", T=16384, D=8192, dtype="f32", normed="bf16", param="f32"),
        # A few rows of odd width.
        dict(name="keep_odd", op="keep", T=333, D=1538, dtype="f16", normed="f16", param="f16"),
        # Kept partial sums brought back for a backward pass.
        dict(name="load_train", op="load", T=8192, D=5120, dtype="bf16", normed="", param="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "forward", "backward", "backward", "step", "keep", "load"])
    if op in ("keep", "load"):
        D = _log_int(rng, 40, 16384)
        if rng.random() < 0.5:
            D = (D + 127) // 128 * 128
        T = _log_int(rng, 1, max(1, min(65536, (1 << 27) // D)))
        dtype = rng.choice(["bf16", "f16", "f32", "f32"])
        return dict(op=op, T=T, D=D, dtype=dtype, normed=rng.choice(["", dtype, "bf16" if dtype == "f32" else dtype]),
                    param=rng.choice([dtype, "f32"]))
    R = _log_int(rng, 1, 8) if rng.random() < 0.9 else _log_int(rng, 9, 32 if op == "forward" else 16)
    D = _log_int(rng, 8, 1024) * 8
    F = _log_int(rng, 64, 28000)
    if rng.random() < 0.6:
        F = (F + 127) // 128 * 128
    most = 5.4e11 / {"forward": 1, "backward": 2, "step": 3}[op] / (D * F)
    T = _log_int(rng, 1, max(1, min(8192, int(most))))
    return dict(op=op, R=R, T=T, D=D, F=F, dtype=rng.choice(["bf16", "bf16", "f16"]),
                act=rng.choice(["silu", "silu", "gelu"]), copies=rng.choice([1, R]))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 12345)
    return g


def _normal(g, shape, dtype, sigma=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(sigma).add_(mean).to(dtype)


def _widths(F, R):
    """Columns of the inner dimension that each rank holds: [r C, min((r + 1) C, F)), C = ceil(F / R)."""
    C = -(-F // R)
    return [max(0, min((r + 1) * C, F) - r * C) for r in range(R)]


def _rows(T, width, dtype, like=torch.empty):
    """[T, width] whose rows start on 16-byte boundaries."""
    return like((T, (width + 7) // 8 * 8), dtype=dtype, device="cuda")[:, :width]


def _handle(key, make):
    if key not in _HANDLES:
        _HANDLES[key] = make()
    return _HANDLES[key]


def _ffn_handle(c):
    from ring_allreduce_gb300 import FeedForward
    key = ("ffn", c["R"], c["D"], c["F"], c["dtype"], c["act"])
    return _handle(key, lambda: FeedForward(c["R"], c["D"], c["F"], c["dtype"], activation=c["act"]))


def _checkpoint_handle(c):
    from ring_allreduce_gb300 import Checkpoint
    key = ("keep", c["D"], c["dtype"], c["normed"], c["param"])
    return _handle(key, lambda: Checkpoint(c["D"], c["dtype"], normed_dtype=c["normed"] or None,
                                           param_dtype=c["param"]))


def _prepare_ffn(c, g):
    R, T, D, F, dt = c["R"], c["T"], c["D"], c["F"], _TORCH[c["dtype"]]
    widths = _widths(F, R)
    s = dict(case=c, x=_normal(g, (T, D), dt))
    s["xs"] = s["x"].expand(c["copies"], T, D).contiguous()   # every rank's copy of the normalised rows
    # outliers: a few channels of the projections are larger, as trained ones are
    loud = 1.0 + 4.0 * (torch.rand((F, 1), generator=g, device="cuda") < 0.01)
    s["w_gate"], s["w_up"], s["w_down"] = (
        list((_normal(g, (F, D), torch.float32, sigma) * louder).to(dt).split(widths))
        for sigma, louder in ((D ** -0.5, loud), (D ** -0.5, loud), (F ** -0.5, 1.0)))
    new = lambda: [_rows(T, w, dt) for w in widths]   # noqa: E731
    s["hidden"] = new()
    if c["op"] != "backward":
        s["parts"] = torch.empty((R, T, D), dtype=dt, device="cuda")
    if c["op"] == "forward":
        s["op"] = _ffn_handle(c) if own else None
        return s
    # the block end's gradient for every rank's partial product
    s["grad_parts"] = _normal(g, (T, D), dt, 0.5).expand(c["copies"], T, D).contiguous()
    groups = [-(-w // _GROUP) for w in widths]
    s["codes"], s["scales"] = [], []
    for _ in range(2):
        codes = [_rows(T, w, torch.int8) for w in widths]
        scales = [torch.empty((T, n), device="cuda") for n in groups]
        if c["op"] == "backward":
            # what forward kept: the codes of rows of a unit normal
            for q, f, w in zip(codes, scales, widths):
                if w:
                    a, b = _codes(_normal(g, (T, w), torch.float32))
                    q.copy_(a)
                    f.copy_(b)
        s["codes"].append(codes)
        s["scales"].append(scales)
    s["grad_gate"], s["grad_up"] = new(), new()
    s["grad_xs"] = torch.empty((R, T, D), dtype=dt, device="cuda")
    s["grad_w"] = [[torch.empty_like(w) for w in s[k]] for k in ("w_gate", "w_up", "w_down")]
    s["op"] = _ffn_handle(c) if own else None
    return s


def _prepare_keep(c, g):
    T, D = c["T"], c["D"]
    dt, pdt = _TORCH[c["dtype"]], _TORCH[c["param"]]
    x = torch.randn((T, D), generator=g, device="cuda") * 2.0
    x *= 1.0 + 9.0 * (torch.rand(D, generator=g, device="cuda") < 0.005)   # loud channels
    s = dict(case=c, rows=x.to(dt), codes=torch.empty((T, D), dtype=torch.int8, device="cuda"),
             scales=torch.empty((T, -(-D // _GROUP)), device="cuda"), restored=torch.empty((T, D), dtype=dt, device="cuda"))
    s["rstd"] = s["weight"] = s["normed"] = None
    if c["normed"]:
        s.update(rstd=(x.square().mean(1) + 1e-6).rsqrt(), weight=_normal(g, (D,), pdt, 0.1, 1.0),
                 normed=torch.empty((T, D), dtype=_TORCH[c["normed"]], device="cuda"))
    if c["op"] == "load":
        s["codes"], s["scales"] = _codes(s.pop("rows").float())
    s["op"] = _checkpoint_handle(c) if own else None
    return s


def prepare(case, seed):
    g = _generator(seed)
    return (_prepare_keep if case["op"] in ("keep", "load") else _prepare_ffn)(case, g)


# ------------------------------------------------------- one pass, both forms

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_forward(s):
    s["op"].forward(s["xs"], s["w_gate"], s["w_up"], s["w_down"], s["hidden"], s["parts"])
    return s["parts"]


def _own_backward(s):
    s["op"].backward(s["grad_parts"], s["xs"], s["w_gate"], s["w_up"], s["w_down"], *s["codes"], s["hidden"],
                     s["grad_gate"], s["grad_up"], s["grad_xs"], *s["grad_w"], gate_scales=s["scales"][0],
                     up_scales=s["scales"][1])
    return s["grad_xs"], s["grad_w"]


def _own_step(s):
    s["op"].forward(s["xs"], s["w_gate"], s["w_up"], s["w_down"], s["hidden"], s["parts"], *s["codes"], *s["scales"])
    return s["parts"], _own_backward(s)


def _own_keep(s):
    s["op"].store(s["rows"], s["codes"], s["scales"])
    return _own_load(s)


def _own_load(s):
    s["op"].load(s["codes"], s["scales"], s["restored"], s["rstd"], s["weight"], s["normed"])
    return s["restored"], s["normed"]


def _act(a, kind):
    return a * torch.sigmoid(a) if kind == "silu" else 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5)))


def _slope(a, kind):
    """The activation's derivative."""
    if kind == "silu":
        p = torch.sigmoid(a)
        return p * (1.0 + a * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5))) + a * (-0.5 * a * a).exp() * (1.0 / math.sqrt(2.0 * math.pi))


def _codes(v):
    """Rows of 32-bit values as 8-bit codes, and the scale of each group of 128 columns: the largest magnitude is 127."""
    T, n = v.shape
    groups = -(-n // _GROUP)
    x = torch.nn.functional.pad(v, (0, groups * _GROUP - n)).view(T, groups, _GROUP)
    most = x.abs().amax(2)
    some = most > _LOWEST
    top = torch.full_like(most, 127.0)   # as a tensor: quotients with a plain number are rounded twice
    q = (x * torch.where(some, top / most, 0.0).unsqueeze(2)).round()
    return q.view(T, -1)[:, :n].to(torch.int8), torch.where(some, most / top, 0.0)


def _values(q, scales):
    """The values that codes stand for, in 32 bits."""
    return q.float() * scales.repeat_interleave(_GROUP, 1)[:, :q.shape[1]]


def _plain_projections(s):
    x = s["x"].float()
    return [x @ w.float().T for w in s["w_gate"]], [x @ w.float().T for w in s["w_up"]]


def _plain_parts(s, gate, up):
    c = s["case"]
    dt = _TORCH[c["dtype"]]
    return torch.stack([((_act(a, c["act"]) * b) @ w.float()).to(dt) for a, b, w in zip(gate, up, s["w_down"])])


def _plain_forward(s):
    return _plain_parts(s, *_plain_projections(s))


def _plain_gradients(s, gate, up):
    c = s["case"]
    dt, kind = _TORCH[c["dtype"]], c["act"]
    dy, x = s["grad_parts"][0].float(), s["x"].float()
    dh = [dy @ w.float().T for w in s["w_down"]]
    da = [d * b * _slope(a, kind) for d, a, b in zip(dh, gate, up)]
    db = [d * _act(a, kind) for d, a in zip(dh, gate)]
    dx = torch.stack([(a @ wg.float() + b @ wu.float()).to(dt)
                      for a, b, wg, wu in zip(da, db, s["w_gate"], s["w_up"])])
    return dx, [[(a.T @ x).to(dt) for a in da], [(b.T @ x).to(dt) for b in db],
                [((_act(a, kind) * b).T @ dy).to(dt) for a, b in zip(gate, up)]]


def _plain_backward(s):
    return _plain_gradients(s, *([_values(q, f) for q, f in zip(*kept)] for kept in zip(s["codes"], s["scales"])))


def _plain_step(s):
    gate, up = _plain_projections(s)
    parts = _plain_parts(s, gate, up)
    return parts, _plain_gradients(s, *([_values(*_codes(v)) for v in kept] for kept in (gate, up)))


def _plain_keep(s):
    return _plain_load(dict(s, **dict(zip(("codes", "scales"), _codes(s["rows"].float())))))


def _plain_load(s):
    c = s["case"]
    v = _values(s["codes"], s["scales"])
    normed = (v * s["rstd"][:, None] * s["weight"].float()).to(_TORCH[c["normed"]]) if c["normed"] else None
    return v.to(_TORCH[c["dtype"]]), normed


_own = dict(forward=_own_forward, backward=_own_backward, step=_own_step, keep=_own_keep, load=_own_load)
_plain = dict(forward=_plain_forward, backward=_plain_backward, step=_plain_step, keep=_plain_keep, load=_plain_load)


# ------------------------------------------------------------------- work

def work(case):
    """Bytes that a pass cannot do without (every input read once, every output written once) and its operations."""
    c = case
    if c["op"] in ("keep", "load"):
        n = c["T"] * c["D"]
        coded = n + 4 * c["T"] * -(-c["D"] // _GROUP)
        restored = n * _BYTES[c["dtype"]] + (n * _BYTES[c["normed"]] + 4 * c["T"] + c["D"] * _BYTES[c["param"]]
                                             if c["normed"] else 0)
        if c["op"] == "load":
            return dict(bytes=coded + restored, flops=3 * n)
        return dict(bytes=n * _BYTES[c["dtype"]] + 2 * coded + restored, flops=6 * n)
    R, T, D, F = (c[k] for k in "RTDF")
    product = 2 * T * D * F
    rows, weights = 2 * T * D, 2 * 3 * D * F
    forward = dict(bytes=rows * (1 + R) + weights, flops=3 * product)
    if c["op"] == "forward":
        return forward
    kept = 2 * T * F + 8 * T * -(-F // _GROUP)
    backward = dict(bytes=rows * (2 + R) + 2 * weights + kept, flops=6 * product)
    if c["op"] == "backward":
        return backward
    # what forward keeps is written once more than backward reads it; the rest is read anew by each
    return {k: forward[k] + backward[k] + (kept if k == "bytes" else 0) for k in forward}


# ------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("keep", "load"):
        return _exact_load(s, *(_exact_codes(s["rows"].double()) if case["op"] == "keep" else (s["codes"], s["scales"])))
    gelu = case["act"] == "gelu"
    x = s["x"].double()
    parts, grads_x, grads = [], [], [[], [], []]
    for r, width in enumerate(_widths(case["F"], case["R"])):
        wg, wu, wd = (s[k][r].double() for k in ("w_gate", "w_up", "w_down"))
        if case["op"] != "backward":
            a, b = torch.mm(x, wg.t()), torch.mm(x, wu.t())
            parts.append(torch.mm((a * _cdf(a) if gelu else a / (1.0 + torch.exp(-a))) * b, wd))
        if case["op"] == "forward":
            continue
        if case["op"] == "step":
            a, b = (_exact_values(*_exact_codes(v.float().double())) for v in (a, b))
        else:
            a, b = (_exact_values(s["codes"][k][r], s["scales"][k][r]) for k in (0, 1))
        dy = s["grad_parts"][0].double()
        dh = torch.mm(dy, wd.t())
        if gelu:
            act, slope = a * _cdf(a), _cdf(a) + a * torch.exp(-a * a / 2.0) / math.sqrt(2.0 * math.pi)
        else:
            p = 1.0 / (1.0 + torch.exp(-a))
            act, slope = a * p, p + a * p * (1.0 - p)
        da, db = dh * slope * b, dh * act
        grads_x.append(torch.mm(da, wg) + torch.mm(db, wu))
        for k, d, y in ((0, da, x), (1, db, x), (2, act * b, dy)):
            grads[k].append(torch.mm(d.t(), y))
    if case["op"] == "forward":
        return torch.stack(parts)
    grads = torch.stack(grads_x), grads
    return grads if case["op"] == "backward" else (torch.stack(parts), grads)


def _cdf(a):
    """The normal distribution function."""
    return torch.special.ndtr(a)


def _exact_codes(v):
    """The codes' definition: 127 over the largest magnitude, and its product with a value, are numbers of binary32."""
    T, n = v.shape
    scales, codes = [], []
    for lo in range(0, n, _GROUP):
        x = v[:, lo:lo + _GROUP]
        most = x.abs().max(1, keepdim=True).values
        by = torch.where(most > _LOWEST, (127.0 / most).float().double(), 0.0)
        codes.append(torch.round((x * by).float()).to(torch.int8))
        scales.append(torch.where(most > _LOWEST, (most / 127.0).float(), 0.0))
    if not codes:
        return torch.empty((T, 0), dtype=torch.int8, device="cuda"), torch.empty((T, 0), device="cuda")
    return torch.cat(codes, 1), torch.cat(scales, 1)


def _exact_values(q, scales):
    if not q.shape[1]:
        return q.double()
    return torch.cat([q[:, _GROUP * k:_GROUP * (k + 1)].double() * scales[:, k:k + 1].double()
                      for k in range(scales.shape[1])], 1)


def _exact_load(s, q, scales):
    v = _exact_values(q, scales)
    return v, v * s["weight"].double() * s["rstd"].double()[:, None] if s["case"]["normed"] else None
