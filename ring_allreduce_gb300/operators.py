"""Model operators around the sums over ranks (``ra_norm_*`` and ``ra_vocab_*``
of include/ra.h), on torch CUDA tensors.

``BlockNorm``: the end of a tensor-parallel block.  The R ranks' partial
products are summed, normalised, gated, added to the residual stream and
normalised for the next block, in one pass; and the gradient of that.

``VocabHead``: the vocabulary-parallel head on R column shards of the logits
(shard r: columns [r C, min((r + 1) C, V)), C = ceil(V / R), as
``ra_chunk_plan(R, V)`` lays them out): log probabilities of given tokens with
entropy and top alternatives, distillation from a teacher's top logits, and
the gradients of both.

The caller owns every buffer, outputs included.  Where R rank buffers are
asked for, a list of R tensors or one tensor with a leading axis of R will do.
Rows may be strided; the last axis is contiguous.  Calls run on the current
stream, or on `stream`.  A wrong shape, type, device or stride raises
ValueError, what the library refuses raises RAError; nothing is launched then.
"""

import ctypes

import torch

from . import binding
from .binding import RAError, Status, _lib, _ST, _SZ, _P

__all__ = ["BlockNorm", "VocabHead"]

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 3}
_CODE_OF = {k: _CODE[v] for k, v in _TORCH.items()}


class _NormForward(ctypes.Structure):
    _fields_ = [("rows", _SZ), ("in_", _P), ("in_stride", _SZ), ("residual", _P), ("residual_stride", _SZ),
                ("weight", _P), ("post_weight", _P), ("gate", _P), ("gate_rows", _SZ), ("out", _P),
                ("out_stride", _SZ), ("outs", _ST), ("residual_out", _P), ("residual_out_stride", _SZ),
                ("total", _P), ("total_stride", _SZ), ("rstd", _P)]


class _NormBackward(ctypes.Structure):
    _fields_ = [("rows", _SZ), ("grad_out", _P), ("grad_out_stride", _SZ), ("grads", _ST),
                ("grad_residual_out", _P), ("grad_residual_out_stride", _SZ), ("residual_out", _P),
                ("residual_out_stride", _SZ), ("total", _P), ("total_stride", _SZ), ("rstd", _P), ("weight", _P),
                ("post_weight", _P), ("gate", _P), ("gate_rows", _SZ), ("grad_in", _P), ("grad_in_stride", _SZ),
                ("outs", _ST), ("grad_residual", _P), ("grad_residual_stride", _SZ), ("grad_weight", _P),
                ("grad_post_weight", _P), ("grad_gate", _P)]


class _Logprobs(ctypes.Structure):
    _fields_ = [("rows", _SZ), ("shards", _P), ("strides", _P), ("targets", _P), ("logprob", _P), ("lse", _P),
                ("entropy", _P), ("top", _ST), ("top_ids", _P), ("top_logprobs", _P)]


class _LogprobsBackward(ctypes.Structure):
    _fields_ = [("rows", _SZ), ("shards", _P), ("strides", _P), ("targets", _P), ("lse", _P), ("entropy", _P),
                ("grad_logprob", _P), ("grad_entropy", _P), ("grads", _P), ("grad_strides", _P)]


class _Distill(ctypes.Structure):
    _fields_ = [("rows", _SZ), ("shards", _P), ("strides", _P), ("teacher_k", _ST), ("teacher_ids", _P),
                ("teacher_logits", _P), ("teacher_dtype", _ST), ("loss", _P), ("lse", _P)]


class _DistillBackward(ctypes.Structure):
    _fields_ = [("rows", _SZ), ("shards", _P), ("strides", _P), ("teacher_k", _ST), ("teacher_ids", _P),
                ("teacher_logits", _P), ("teacher_dtype", _ST), ("lse", _P), ("grad_loss", _P), ("grads", _P),
                ("grad_strides", _P)]


def _fail(name, t, want):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a torch tensor is expected, got {type(t).__name__}")
    raise ValueError(f"{name}: {want} is expected, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on "
                     f"{t.device}")


class _Handle:
    """What the operators share: the device, the checks and the call."""

    def __init__(self, dtype):
        self._h = None
        if dtype not in _TORCH:
            raise ValueError(f"dtype {dtype!r}: one of {sorted(_TORCH)} is expected")
        self.dtype = _TORCH[dtype]
        self.device = torch.cuda.current_device() if torch.cuda.is_available() else -1

    def _flat(self, name, t, shape, dtype):
        """Address of a contiguous tensor."""
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and t.get_device() == self.device):
            _fail(name, t, f"a contiguous {dtype} {tuple(shape)} on cuda:{self.device}")
        return t.data_ptr()

    def _rows(self, name, t, shape, dtype):
        """Address and row stride of a tensor [rows, width] whose rows are contiguous."""
        if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                and t.get_device() == self.device):
            _fail(name, t, f"{dtype} {tuple(shape)} on cuda:{self.device}")
        st = t.stride()
        if st[1] != 1 and shape[1] > 1:
            _fail(name, t, "a contiguous last axis")
        return t.data_ptr(), st[0]

    def _ranks(self, name, t, counts, shape, dtype):
        """C array of rank buffers [rows, width], their common row stride and
        their number (one of `counts`)."""
        if isinstance(t, torch.Tensor):
            if t.dim() != 3 or t.shape[0] not in counts:
                _fail(name, t, f"{' or '.join(map(str, counts))} rank buffers {tuple(shape)}")
            n = t.shape[0]
            step = t.stride(0) * t.element_size() if n > 1 else 0
            base, stride = self._rows(name, t[0], shape, dtype)
            return (_P * n)(*[base + r * step for r in range(n)]), stride, n
        if len(t) not in counts:
            raise ValueError(f"{name}: {' or '.join(map(str, counts))} rank buffers are expected, got {len(t)}")
        got = [self._rows(f"{name}[{r}]", x, shape, dtype) for r, x in enumerate(t)]
        if shape[0] > 1 and any(s != got[0][1] for _, s in got):
            raise ValueError(f"{name}: the rank buffers' rows have different strides")
        return (_P * len(got))(*[p for p, _ in got]), got[0][1], len(got)

    def _call(self, fn, args, stream, tensors):
        if self._h is None:
            raise ValueError("the handle is closed")
        if stream is None:
            # the raw handle of torch's current stream on the handle's device
            raw = torch.cuda.current_stream(self.device).cuda_stream
        else:
            raw = binding._stream(stream)
            _keep(tensors, stream, self.device)
        st = fn(self._h, ctypes.addressof(args), raw)
        if st != Status.OK:
            raise RAError(st, binding.ra_last_error())

    def close(self):
        if self._h is not None:
            h, self._h = self._h, None
            binding._check(self._destroy(h))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _keep(tensors, stream, device):
    """Tell torch's allocator that a stream of the caller's choice uses the
    tensors, so that their memory is not handed out again before it is done."""
    if isinstance(stream, int):
        if stream == 0:
            stream = torch.cuda.default_stream(device)
        else:
            stream = torch.cuda.ExternalStream(stream, device=device)
    for t in tensors:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
        elif t is not None:
            for x in t:
                x.record_stream(stream)


class BlockNorm(_Handle):
    """The end of a block of `dim` columns over R ranks.

    dtype: the partials' and the normalised rows' type; residual_dtype,
    param_dtype: the residual stream's and the weights' (and the gate's), "f32"
    or dtype, which is their default.  eps is added to the mean square; scale
    multiplies the block's contribution to the residual stream."""

    _destroy = staticmethod(_lib.ra_norm_destroy)

    def __init__(self, R, dim, dtype="bf16", residual_dtype=None, param_dtype=None, eps=1e-6, scale=1.0):
        super().__init__(dtype)
        residual_dtype, param_dtype = residual_dtype or dtype, param_dtype or dtype
        for name, d in (("residual_dtype", residual_dtype), ("param_dtype", param_dtype)):
            if d not in _TORCH:
                raise ValueError(f"{name} {d!r}: one of {sorted(_TORCH)} is expected")
        self.R, self.dim, self.eps, self.scale = int(R), int(dim), float(eps), float(scale)
        self.residual_dtype, self.param_dtype = _TORCH[residual_dtype], _TORCH[param_dtype]
        h = _P()
        binding._check(_lib.ra_norm_create(self.R, self.dim, _CODE_OF[dtype], _CODE_OF[residual_dtype],
                                           _CODE_OF[param_dtype], self.eps, self.scale, ctypes.byref(h)))
        self._h = h

    def _params(self, a, rows, weight, post_weight, gate):
        one = (self.dim,)
        a.weight = self._flat("weight", weight, one, self.param_dtype)
        if post_weight is not None:
            a.post_weight = self._flat("post_weight", post_weight, one, self.param_dtype)
        if gate is not None:
            a.gate_rows = gate.shape[0] if isinstance(gate, torch.Tensor) and gate.dim() == 2 else 0
            a.gate = self._flat("gate", gate, (a.gate_rows, self.dim), self.param_dtype)

    def forward(self, parts, residual, weight, outs, residual_out, post_weight=None, gate=None, total=None,
                rstd=None, stream=None):
        """S = sum of parts; y = S / rms(S) * post_weight (y = S without it);
        residual_out = residual + scale * gate * y;
        outs = residual_out / rms(residual_out) * weight.

        parts: R x [T, dim]; outs: 1 or R x [T, dim], each gets the same;
        residual, residual_out: [T, dim], may be one tensor; gate: [G, dim], G
        divides T, row t is gated by row t // (T / G).  total [T, dim] and rstd
        [2, T] (float32) keep what backward reads: S, and the two norms' factors."""
        if not isinstance(residual, torch.Tensor) or residual.dim() != 2:
            raise ValueError(f"residual: a tensor [rows, {self.dim}] is expected")
        T = residual.shape[0]
        shape = (T, self.dim)
        a = _NormForward(rows=T)
        # the arrays stay referenced until the call has returned
        ins, a.in_stride, _ = self._ranks("parts", parts, (self.R,), shape, self.dtype)
        to, a.out_stride, a.outs = self._ranks("outs", outs, (1, self.R), shape, self.dtype)
        a.in_, a.out = ctypes.addressof(ins), ctypes.addressof(to)
        a.residual, a.residual_stride = self._rows("residual", residual, shape, self.residual_dtype)
        a.residual_out, a.residual_out_stride = self._rows("residual_out", residual_out, shape, self.residual_dtype)
        self._params(a, T, weight, post_weight, gate)
        if total is not None:
            a.total, a.total_stride = self._rows("total", total, shape, self.dtype)
        if rstd is not None:
            a.rstd = self._flat("rstd", rstd, (2, T), torch.float32)
        self._call(_lib.ra_norm_forward, a, stream,
                   (parts, residual, weight, outs, residual_out, post_weight, gate, total, rstd))

    def backward(self, grad_outs, grad_residual_out, residual_out, rstd, weight, grad_ins, grad_residual,
                 grad_weight=None, post_weight=None, gate=None, total=None, grad_post_weight=None, grad_gate=None,
                 stream=None):
        """The gradient of forward.

        grad_outs: 1 or R x [T, dim], the ranks' partial gradients of the
        normalised rows, summed here; grad_residual_out: that of residual_out, or None for zero.
        residual_out, rstd, total: what forward wrote (total only with
        post_weight or grad_gate).  Writes grad_ins, 1 or R x [T, dim] (the
        gradient of every rank's partial), grad_residual [T, dim], and, in
        float32, grad_weight [dim], grad_post_weight [dim] and grad_gate
        [G, dim] where given.  grad_residual may be grad_residual_out, and
        grad_ins may be grad_outs."""
        if not isinstance(residual_out, torch.Tensor) or residual_out.dim() != 2:
            raise ValueError(f"residual_out: a tensor [rows, {self.dim}] is expected")
        T = residual_out.shape[0]
        shape, one = (T, self.dim), (self.dim,)
        a = _NormBackward(rows=T)
        ins, a.grad_out_stride, a.grads = self._ranks("grad_outs", grad_outs, (1, self.R), shape, self.dtype)
        to, a.grad_in_stride, a.outs = self._ranks("grad_ins", grad_ins, (1, self.R), shape, self.dtype)
        a.grad_out, a.grad_in = ctypes.addressof(ins), ctypes.addressof(to)
        if grad_residual_out is not None:
            a.grad_residual_out, a.grad_residual_out_stride = self._rows(
                "grad_residual_out", grad_residual_out, shape, self.residual_dtype)
        a.residual_out, a.residual_out_stride = self._rows("residual_out", residual_out, shape, self.residual_dtype)
        a.grad_residual, a.grad_residual_stride = self._rows("grad_residual", grad_residual, shape,
                                                             self.residual_dtype)
        self._params(a, T, weight, post_weight, gate)
        if total is not None:
            a.total, a.total_stride = self._rows("total", total, shape, self.dtype)
        a.rstd = self._flat("rstd", rstd, (2, T), torch.float32)
        if grad_weight is not None:
            a.grad_weight = self._flat("grad_weight", grad_weight, one, torch.float32)
        if grad_post_weight is not None:
            a.grad_post_weight = self._flat("grad_post_weight", grad_post_weight, one, torch.float32)
        if grad_gate is not None:
            a.grad_gate = self._flat("grad_gate", grad_gate, (a.gate_rows, self.dim), torch.float32)
        self._call(_lib.ra_norm_backward, a, stream,
                   (grad_outs, grad_residual_out, residual_out, rstd, weight, grad_ins, grad_residual, grad_weight,
                    post_weight, gate, total, grad_post_weight, grad_gate))


class VocabHead(_Handle):
    """A head of `vocab` columns over R ranks; every call divides the logits by `temperature`."""

    _destroy = staticmethod(_lib.ra_vocab_destroy)

    def __init__(self, R, vocab, dtype="bf16", temperature=1.0):
        super().__init__(dtype)
        self.R, self.vocab, self.temperature = int(R), int(vocab), float(temperature)
        if self.vocab < 0:
            raise ValueError(f"vocab {vocab}")
        h = _P()
        binding._check(_lib.ra_vocab_create(self.R, self.vocab, _CODE_OF[dtype], self.temperature, ctypes.byref(h)))
        self._h = h
        #: columns of each rank's shard
        self.widths = [n for _, n in binding.ra_chunk_plan(self.R, self.vocab)]

    def _shards(self, name, t, T):
        """C arrays of the shards' addresses and row strides."""
        if len(t) != self.R:
            raise ValueError(f"{name}: {self.R} shards are expected, got {len(t)}")
        ptrs, strides = [], []
        for r, (x, w) in enumerate(zip(t, self.widths)):
            if w:
                p, s = self._rows(f"{name}[{r}]", x, (T, w), self.dtype)
            else:
                p, s = None, 0      # a shard without columns: nothing to look at
            ptrs.append(p)
            strides.append(s)
        return (_P * self.R)(*ptrs), (_SZ * self.R)(*strides)

    @staticmethod
    def _count(name, t):
        if not isinstance(t, torch.Tensor) or t.dim() != 1:
            raise ValueError(f"{name}: a tensor [rows] is expected")
        return t.shape[0]

    def logprobs(self, shards, targets, logprob, lse, entropy=None, top_ids=None, top_logprobs=None, stream=None):
        """Per row of the logits: logprob = log p of targets (int64; 0 where
        negative, NaN where beyond the vocabulary), lse = log sum exp, entropy,
        and the K = top_ids.shape[1] largest logits' columns (int64, equal ones
        lowest first) with their log probabilities, K at most 32."""
        T = self._count("targets", targets)
        one = (T,)
        a = _Logprobs(rows=T)
        p, s = self._shards("shards", shards, T)
        a.shards, a.strides = ctypes.addressof(p), ctypes.addressof(s)
        a.targets = self._flat("targets", targets, one, torch.int64)
        a.logprob = self._flat("logprob", logprob, one, torch.float32)
        a.lse = self._flat("lse", lse, one, torch.float32)
        if entropy is not None:
            a.entropy = self._flat("entropy", entropy, one, torch.float32)
        if (top_ids is None) != (top_logprobs is None):
            raise ValueError("top_ids and top_logprobs go together")
        if top_ids is not None:
            K = top_ids.shape[1] if isinstance(top_ids, torch.Tensor) and top_ids.dim() == 2 else 0
            a.top = K
            a.top_ids = self._flat("top_ids", top_ids, (T, K), torch.int64)
            a.top_logprobs = self._flat("top_logprobs", top_logprobs, (T, K), torch.float32)
        self._call(_lib.ra_vocab_logprobs, a, stream,
                   (shards, targets, logprob, lse, entropy, top_ids, top_logprobs))

    def logprobs_backward(self, shards, targets, lse, grad_logprob, grads, entropy=None, grad_entropy=None,
                          stream=None):
        """grads (R shards, may be the logits' own) = the logits' gradient of
        sum(grad_logprob * logprob) + sum(grad_entropy * entropy); lse and
        entropy are what logprobs wrote."""
        T = self._count("targets", targets)
        one = (T,)
        a = _LogprobsBackward(rows=T)
        p, s = self._shards("shards", shards, T)
        gp, gs = self._shards("grads", grads, T)
        a.shards, a.strides = ctypes.addressof(p), ctypes.addressof(s)
        a.grads, a.grad_strides = ctypes.addressof(gp), ctypes.addressof(gs)
        a.targets = self._flat("targets", targets, one, torch.int64)
        a.lse = self._flat("lse", lse, one, torch.float32)
        a.grad_logprob = self._flat("grad_logprob", grad_logprob, one, torch.float32)
        if grad_entropy is not None:
            a.grad_entropy = self._flat("grad_entropy", grad_entropy, one, torch.float32)
            a.entropy = self._flat("entropy", entropy, one, torch.float32)
        self._call(_lib.ra_vocab_logprobs_backward, a, stream,
                   (shards, targets, lse, grad_logprob, grads, entropy, grad_entropy))

    def _teacher(self, a, teacher_ids, teacher_logits):
        if not isinstance(teacher_ids, torch.Tensor) or teacher_ids.dim() != 2:
            raise ValueError("teacher_ids: a tensor [rows, K] is expected")
        T, K = teacher_ids.shape
        a.rows, a.teacher_k = T, K
        a.teacher_ids = self._flat("teacher_ids", teacher_ids, (T, K), torch.int64)
        dt = torch.float32 if isinstance(teacher_logits, torch.Tensor) and teacher_logits.dtype is torch.float32 \
            else self.dtype
        a.teacher_logits = self._flat("teacher_logits", teacher_logits, (T, K), dt)
        a.teacher_dtype = _CODE[dt]
        return T

    def distill(self, shards, teacher_ids, teacher_logits, loss, lse, stream=None):
        """Per row: q = softmax(teacher_logits / temperature) over the row's K
        tokens (at most 256; a negative id or one beyond the vocabulary is absent),
        loss = temperature^2 sum q (log q - log p), lse = log sum exp of the
        student's logits / temperature.  teacher_ids: int64 [T, K];
        teacher_logits: float32 or the logits' type."""
        a = _Distill()
        T = self._teacher(a, teacher_ids, teacher_logits)
        p, s = self._shards("shards", shards, T)
        a.shards, a.strides = ctypes.addressof(p), ctypes.addressof(s)
        a.loss = self._flat("loss", loss, (T,), torch.float32)
        a.lse = self._flat("lse", lse, (T,), torch.float32)
        self._call(_lib.ra_vocab_distill, a, stream, (shards, teacher_ids, teacher_logits, loss, lse))

    def distill_backward(self, shards, teacher_ids, teacher_logits, lse, grad_loss, grads, stream=None):
        """grads (R shards, may be the logits' own) = the logits' gradient of
        sum(grad_loss * loss); lse is what distill wrote."""
        a = _DistillBackward()
        T = self._teacher(a, teacher_ids, teacher_logits)
        p, s = self._shards("shards", shards, T)
        gp, gs = self._shards("grads", grads, T)
        a.shards, a.strides = ctypes.addressof(p), ctypes.addressof(s)
        a.grads, a.grad_strides = ctypes.addressof(gp), ctypes.addressof(gs)
        a.lse = self._flat("lse", lse, (T,), torch.float32)
        a.grad_loss = self._flat("grad_loss", grad_loss, (T,), torch.float32)
        self._call(_lib.ra_vocab_distill_backward, a, stream,
                   (shards, teacher_ids, teacher_logits, lse, grad_loss, grads))
