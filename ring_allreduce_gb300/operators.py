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
stream, or on `stream`; what one call writes and another reads or writes is the
caller's to order between streams.  A wrong shape, type, device or stride raises
ValueError, what the library refuses raises RAError; nothing is launched then.
"""

import ctypes
import importlib
import os

import torch

from . import binding
from . import build as _build
from .binding import RAError, _lib, _P

__all__ = ["BlockNorm", "VocabHead"]

_CODE = {"f32": 0, "bf16": 1, "f16": 3}     # ra_dtype


def _load():
    """The extension that checks and marshals the tensors (after torch, whose
    libraries it uses), bound to the loaded library's functions."""
    if not os.path.exists(_build.TORCH_EXT_PATH):
        raise ImportError(f"{_build.TORCH_EXT}.so is not built ({_build.TORCH_EXT_PATH}); run "
                          "`python -m ring_allreduce_gb300.build` (or __graft_entry__.build())")
    ext = importlib.import_module("." + _build.TORCH_EXT, __package__)
    ext.bind(*(ctypes.cast(f, _P).value for f in (
        _lib.ra_norm_forward, _lib.ra_norm_backward, _lib.ra_vocab_logprobs, _lib.ra_vocab_logprobs_backward,
        _lib.ra_vocab_distill, _lib.ra_vocab_distill_backward)))
    return ext


_ext = _load()
_current_stream = torch._C._cuda_getCurrentRawStream   # the raw handle of torch's current stream on a device


class _Handle:
    """What the operators share: the handle, its device and the calls' streams."""

    def __init__(self, dtype):
        self._config = None
        _code("dtype", dtype)
        self.device = torch.cuda.current_device() if torch.cuda.is_available() else -1

    def _opened(self, h, R, *config):
        """The handle and what the extension's checks go by."""
        # the extension has seen every tensor to be on the device
        binding._check(self._set_option(h, binding.Option.CHECK_POINTERS, 0))
        self._config = (h.value, self.device, R, *config)

    def _call(self, fn, stream, *args):
        if self._config is None:
            raise ValueError("the handle is closed")
        if stream is None:
            status = fn(*self._config, *args, _current_stream(self.device))
        else:
            args = [_listed(a) for a in args]
            status = fn(*self._config, *args, binding._stream(stream))
            if not status:
                _keep(args, stream, self.device)   # now that the extension has seen that they are tensors that fit
        if status:
            raise RAError(status, binding.ra_last_error())

    def close(self):
        if self._config is not None:
            h, self._config = self._config[0], None
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


def _code(name, dtype):
    if dtype not in _CODE:
        raise ValueError(f"{name} {dtype!r}: one of {sorted(_CODE)} is expected")
    return _CODE[dtype]


def _listed(arg):
    """An argument that can be gone through twice."""
    if arg is None or isinstance(arg, (torch.Tensor, list, tuple)):
        return arg
    try:
        return tuple(arg)
    except TypeError:
        return arg


def _keep(args, stream, device):
    """Tell torch's allocator that a stream of the caller's choice uses the
    tensors, so that their memory is not handed out again before it is done."""
    if isinstance(stream, int):
        if stream == 0:
            stream = torch.cuda.default_stream(device)
        else:
            stream = torch.cuda.ExternalStream(stream, device=device)
    for arg in args:
        for t in arg if isinstance(arg, (list, tuple)) else (arg,):
            if isinstance(t, torch.Tensor) and t.is_cuda:   # what a call does not look at may be anything
                t.record_stream(stream)


class BlockNorm(_Handle):
    """The end of a block of `dim` columns over R ranks.

    dtype: the partials' and the normalised rows' type; residual_dtype,
    param_dtype: the residual stream's and the weights' (and the gate's), "f32"
    or dtype, which is their default.  eps is added to the mean square; scale
    multiplies the block's contribution to the residual stream.

    backward calls of one BlockNorm share its workspace: calls on several
    streams, and replays of graphs that captured one, have to be ordered (by
    events or wait_stream) as dependent work is; for backward passes that
    overlap, take a BlockNorm each.  forward calls may overlap.  The first
    backward call allocates the workspace and cannot be captured; a graph that
    captured a later one may be replayed when the BlockNorm is closed."""

    _destroy, _set_option = staticmethod(_lib.ra_norm_destroy), staticmethod(_lib.ra_norm_set_option)

    def __init__(self, R, dim, dtype="bf16", residual_dtype=None, param_dtype=None, eps=1e-6, scale=1.0):
        super().__init__(dtype)
        self.R, self.dim, self.eps, self.scale = int(R), int(dim), float(eps), float(scale)
        codes = (_code("dtype", dtype), _code("residual_dtype", residual_dtype or dtype),
                 _code("param_dtype", param_dtype or dtype))
        h = _P()
        binding._check(_lib.ra_norm_create(self.R, self.dim, *codes, self.eps, self.scale, ctypes.byref(h)))
        self._opened(h, self.R, self.dim, *codes)

    def forward(self, parts, residual, weight, outs, residual_out, post_weight=None, gate=None, total=None,
                rstd=None, stream=None):
        """S = sum of parts; y = S / rms(S) * post_weight (y = S without it);
        residual_out = residual + scale * gate * y;
        outs = residual_out / rms(residual_out) * weight.

        parts: R x [T, dim]; outs: 1 or R x [T, dim], each gets the same;
        residual, residual_out: [T, dim], may be one tensor; gate: [G, dim], G
        divides T, row t is gated by row t // (T / G).  total [T, dim] and rstd
        [2, T] (float32) keep what backward reads: S, and the two norms' factors."""
        self._call(_ext.norm_forward, stream, parts, residual, weight, outs, residual_out, post_weight, gate, total, rstd)

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
        [G, dim] where given: sums over the rows, zero where T is 0.  grad_residual may be grad_residual_out, and
        grad_ins may be grad_outs."""
        self._call(_ext.norm_backward, stream, grad_outs, grad_residual_out, residual_out, rstd, weight, grad_ins,
                   grad_residual, grad_weight, post_weight, gate, total, grad_post_weight, grad_gate)


class VocabHead(_Handle):
    """A head of `vocab` columns over R ranks; every call divides the logits by `temperature`."""

    _destroy, _set_option = staticmethod(_lib.ra_vocab_destroy), staticmethod(_lib.ra_vocab_set_option)

    def __init__(self, R, vocab, dtype="bf16", temperature=1.0):
        super().__init__(dtype)
        self.R, self.vocab, self.temperature = int(R), int(vocab), float(temperature)
        if self.vocab < 0:
            raise ValueError(f"vocab {vocab}")
        code = _code("dtype", dtype)
        h = _P()
        binding._check(_lib.ra_vocab_create(self.R, self.vocab, code, self.temperature, ctypes.byref(h)))
        self._opened(h, self.R, self.vocab, code)
        #: columns of each rank's shard
        self.widths = [n for _, n in binding.ra_chunk_plan(self.R, self.vocab)]

    def logprobs(self, shards, targets, logprob, lse, entropy=None, top_ids=None, top_logprobs=None, stream=None):
        """Per row of the logits: logprob = log p of targets (int64; 0 where
        negative, NaN where beyond the vocabulary), lse = log sum exp, entropy,
        and the K = top_ids.shape[1] largest logits' columns (int64, equal ones
        lowest first) with their log probabilities, K at most 32."""
        self._call(_ext.logprobs, stream, shards, targets, logprob, lse, entropy, top_ids, top_logprobs)

    def logprobs_backward(self, shards, targets, lse, grad_logprob, grads, entropy=None, grad_entropy=None,
                          stream=None):
        """grads (R shards, may be the logits' own) = the logits' gradient of
        sum(grad_logprob * logprob) + sum(grad_entropy * entropy); lse and
        entropy are what logprobs wrote."""
        self._call(_ext.logprobs_backward, stream, shards, targets, lse, grad_logprob, grads, entropy, grad_entropy)

    def distill(self, shards, teacher_ids, teacher_logits, loss, lse, stream=None):
        """Per row: q = softmax(teacher_logits / temperature) over the row's K
        tokens (at most 256; a negative id or one beyond the vocabulary is absent),
        loss = temperature^2 sum q (log q - log p), lse = log sum exp of the
        student's logits / temperature.  teacher_ids: int64 [T, K];
        teacher_logits: float32 or the logits' type."""
        self._call(_ext.distill, stream, shards, teacher_ids, teacher_logits, loss, lse)

    def distill_backward(self, shards, teacher_ids, teacher_logits, lse, grad_loss, grads, stream=None):
        """grads (R shards, may be the logits' own) = the logits' gradient of
        sum(grad_loss * loss); lse is what distill wrote."""
        self._call(_ext.distill_backward, stream, shards, teacher_ids, teacher_logits, lse, grad_loss, grads)
