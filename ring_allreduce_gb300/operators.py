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
from array import array

import torch

from . import binding
from .binding import RAError, _lib, _ST, _SZ, _P

__all__ = ["BlockNorm", "VocabHead"]

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 3}
_CODE_OF = {k: _CODE[v] for k, v in _TORCH.items()}
_byref = ctypes.byref
_current_stream = torch._C._cuda_getCurrentRawStream   # the raw handle of torch's current stream on a device


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

    # A call's checks run before every launch, for a few microseconds in all: a
    # decode step is hardly longer.  So the common case (a contiguous tensor)
    # is asked for first, and texts are made only for an error.

    def _flat(self, name, t, shape, dtype):
        """Address of a contiguous tensor."""
        if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous() \
                and t.get_device() == self.device:
            return t.data_ptr()
        _fail(name, t, f"a contiguous {dtype} {tuple(shape)} on cuda:{self.device}")

    def _rows(self, name, t, shape, dtype):
        """Address and row stride of a tensor [rows, width] whose rows are contiguous."""
        if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == self.device:
            if t.is_contiguous():
                return t.data_ptr(), shape[1]
            step, one = t.stride()
            if one == 1 or shape[1] <= 1:
                return t.data_ptr(), step
        _fail(name, t, f"{dtype} {tuple(shape)}, its last axis contiguous, on cuda:{self.device}")

    def _ranks(self, name, t, shape, dtype, only=None):
        """The addresses of rank buffers [rows, width] as a C array (which has
        to stay referenced until the call has returned) and where it is, their
        common row stride and their number: R, or also 1 where `only` is not R."""
        n, rows, width = len(t), *shape
        if n != self.R and (n != 1 or only == self.R):
            raise ValueError(f"{name}: {'' if only == self.R else '1 or '}{self.R} rank buffers are expected, got {n}")
        if isinstance(t, torch.Tensor):
            if t.dtype is dtype and t.shape == (n, rows, width) and t.get_device() == self.device:
                base, rank, stride = t.data_ptr(), rows * width, width
                if not t.is_contiguous():
                    rank, stride, one = t.stride()
                    if one != 1 and width > 1:
                        _fail(name, t, "a contiguous last axis")
                step = rank * dtype.itemsize
                ptrs = array("Q", range(base, base + n * step, step) if step else [base] * n)
                return ptrs, ptrs.buffer_info()[0], stride, n
            _fail(name, t, f"{n} x {dtype} {tuple(shape)} on cuda:{self.device}")
        got = [self._rows(name, x, shape, dtype) for x in t]
        stride = got[0][1]
        if rows > 1:
            for _, s in got:
                if s != stride:
                    raise ValueError(f"{name}: the rank buffers' rows have different strides")
        ptrs = array("Q", [p for p, _ in got])
        return ptrs, ptrs.buffer_info()[0], stride, n

    def _call(self, fn, args, stream, tensors):
        if self._h is None:
            raise ValueError("the handle is closed")
        if stream is None:
            raw = _current_stream(self.device)
        else:
            raw = binding._stream(stream)
            _keep(tensors, stream, self.device)
        status = fn(self._h, _byref(args), raw)
        if status:
            raise RAError(status, binding.ra_last_error())

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

    def _gate(self, gate):
        """Address and rows of the gate (0, 0 without one)."""
        if gate is None:
            return None, 0
        rows = gate.shape[0] if isinstance(gate, torch.Tensor) and gate.dim() == 2 else 0
        return self._flat("gate", gate, (rows, self.dim), self.param_dtype), rows

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
        T, one, dt, rdt = residual.shape[0], (self.dim,), self.dtype, self.residual_dtype
        shape = (T, self.dim)
        ins, ins_at, in_stride, _ = self._ranks("parts", parts, shape, dt, self.R)
        to, to_at, out_stride, n = self._ranks("outs", outs, shape, dt)
        res, res_stride = self._rows("residual", residual, shape, rdt)
        res_out, res_out_stride = self._rows("residual_out", residual_out, shape, rdt)
        g, gate_rows = self._gate(gate)
        tot, tot_stride = (None, 0) if total is None else self._rows("total", total, shape, dt)
        self._call(_lib.ra_norm_forward, _NormForward(
            T, ins_at, in_stride, res, res_stride, self._flat("weight", weight, one, self.param_dtype),
            None if post_weight is None else self._flat("post_weight", post_weight, one, self.param_dtype),
            g, gate_rows, to_at, out_stride, n, res_out, res_out_stride, tot, tot_stride,
            None if rstd is None else self._flat("rstd", rstd, (2, T), torch.float32)), stream,
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
        T, one, dt, rdt, f32 = residual_out.shape[0], (self.dim,), self.dtype, self.residual_dtype, torch.float32
        shape = (T, self.dim)
        ins, ins_at, in_stride, grads = self._ranks("grad_outs", grad_outs, shape, dt)
        to, to_at, out_stride, n = self._ranks("grad_ins", grad_ins, shape, dt)
        gro, gro_stride = (None, 0) if grad_residual_out is None else \
            self._rows("grad_residual_out", grad_residual_out, shape, rdt)
        ro, ro_stride = self._rows("residual_out", residual_out, shape, rdt)
        gr, gr_stride = self._rows("grad_residual", grad_residual, shape, rdt)
        g, gate_rows = self._gate(gate)
        tot, tot_stride = (None, 0) if total is None else self._rows("total", total, shape, dt)
        self._call(_lib.ra_norm_backward, _NormBackward(
            T, ins_at, in_stride, grads, gro, gro_stride, ro, ro_stride, tot, tot_stride,
            self._flat("rstd", rstd, (2, T), f32), self._flat("weight", weight, one, self.param_dtype),
            None if post_weight is None else self._flat("post_weight", post_weight, one, self.param_dtype),
            g, gate_rows, to_at, out_stride, n, gr, gr_stride,
            None if grad_weight is None else self._flat("grad_weight", grad_weight, one, f32),
            None if grad_post_weight is None else self._flat("grad_post_weight", grad_post_weight, one, f32),
            None if grad_gate is None else self._flat("grad_gate", grad_gate, (gate_rows, self.dim), f32)), stream,
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
        self._widths = array("Q", [0] * self.R + self.widths)   # addresses and strides of contiguous shards

    def _shards(self, name, t, T):
        """C array of the shards' addresses, then of their row strides, and
        where the two are."""
        R, dt, device = self.R, self.dtype, self.device
        if len(t) != R:
            raise ValueError(f"{name}: {R} shards are expected, got {len(t)}")
        both = array("Q", self._widths)
        for r, x in enumerate(t):
            shape = (T, self.widths[r])
            if shape[1]:      # a shard without columns is not looked at
                if isinstance(x, torch.Tensor) and x.dtype is dt and x.shape == shape and x.is_contiguous() \
                        and x.get_device() == device:
                    both[r] = x.data_ptr()
                else:
                    both[r], both[R + r] = self._rows(name, x, shape, dt)
        at = both.buffer_info()[0]
        return both, at, at + 8 * R

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
        T, f32 = self._count("targets", targets), torch.float32
        one, K, ti, tl = (T,), 0, None, None
        x, x_at, x_strides = self._shards("shards", shards, T)
        if (top_ids is None) != (top_logprobs is None):
            raise ValueError("top_ids and top_logprobs go together")
        if top_ids is not None:
            K = top_ids.shape[1] if isinstance(top_ids, torch.Tensor) and top_ids.dim() == 2 else 0
            ti = self._flat("top_ids", top_ids, (T, K), torch.int64)
            tl = self._flat("top_logprobs", top_logprobs, (T, K), f32)
        self._call(_lib.ra_vocab_logprobs, _Logprobs(
            T, x_at, x_strides, self._flat("targets", targets, one, torch.int64),
            self._flat("logprob", logprob, one, f32), self._flat("lse", lse, one, f32),
            None if entropy is None else self._flat("entropy", entropy, one, f32), K, ti, tl), stream,
            (shards, targets, logprob, lse, entropy, top_ids, top_logprobs))

    def logprobs_backward(self, shards, targets, lse, grad_logprob, grads, entropy=None, grad_entropy=None,
                          stream=None):
        """grads (R shards, may be the logits' own) = the logits' gradient of
        sum(grad_logprob * logprob) + sum(grad_entropy * entropy); lse and
        entropy are what logprobs wrote."""
        T, f32 = self._count("targets", targets), torch.float32
        one, H, gh = (T,), None, None
        x, x_at, x_strides = self._shards("shards", shards, T)
        g, g_at, g_strides = self._shards("grads", grads, T)
        if grad_entropy is not None:
            gh = self._flat("grad_entropy", grad_entropy, one, f32)
            H = self._flat("entropy", entropy, one, f32)
        self._call(_lib.ra_vocab_logprobs_backward, _LogprobsBackward(
            T, x_at, x_strides, self._flat("targets", targets, one, torch.int64),
            self._flat("lse", lse, one, f32), H, self._flat("grad_logprob", grad_logprob, one, f32), gh,
            g_at, g_strides), stream,
            (shards, targets, lse, grad_logprob, grads, entropy, grad_entropy))

    def _teacher(self, teacher_ids, teacher_logits):
        """Rows, tokens per row, the two addresses and the type's code."""
        if not isinstance(teacher_ids, torch.Tensor) or teacher_ids.dim() != 2:
            raise ValueError("teacher_ids: a tensor [rows, K] is expected")
        shape = teacher_ids.shape
        dt = torch.float32 if getattr(teacher_logits, "dtype", None) is torch.float32 else self.dtype
        return (*shape, self._flat("teacher_ids", teacher_ids, shape, torch.int64),
                self._flat("teacher_logits", teacher_logits, shape, dt), _CODE[dt])

    def distill(self, shards, teacher_ids, teacher_logits, loss, lse, stream=None):
        """Per row: q = softmax(teacher_logits / temperature) over the row's K
        tokens (at most 256; a negative id or one beyond the vocabulary is absent),
        loss = temperature^2 sum q (log q - log p), lse = log sum exp of the
        student's logits / temperature.  teacher_ids: int64 [T, K];
        teacher_logits: float32 or the logits' type."""
        T, K, ids, logits, code = self._teacher(teacher_ids, teacher_logits)
        x, x_at, x_strides = self._shards("shards", shards, T)
        self._call(_lib.ra_vocab_distill, _Distill(
            T, x_at, x_strides, K, ids, logits, code, self._flat("loss", loss, (T,), torch.float32),
            self._flat("lse", lse, (T,), torch.float32)), stream, (shards, teacher_ids, teacher_logits, loss, lse))

    def distill_backward(self, shards, teacher_ids, teacher_logits, lse, grad_loss, grads, stream=None):
        """grads (R shards, may be the logits' own) = the logits' gradient of
        sum(grad_loss * loss); lse is what distill wrote."""
        T, K, ids, logits, code = self._teacher(teacher_ids, teacher_logits)
        x, x_at, x_strides = self._shards("shards", shards, T)
        g, g_at, g_strides = self._shards("grads", grads, T)
        self._call(_lib.ra_vocab_distill_backward, _DistillBackward(
            T, x_at, x_strides, K, ids, logits, code, self._flat("lse", lse, (T,), torch.float32),
            self._flat("grad_loss", grad_loss, (T,), torch.float32), g_at, g_strides), stream,
            (shards, teacher_ids, teacher_logits, lse, grad_loss, grads))
