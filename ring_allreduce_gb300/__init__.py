"""Ring AllReduce for R ranks held as R buffers in one GB300's HBM.

The compute path is the CUDA library ``libra_gb300.so`` (``include/ra.h``);
this package is its thin Python binding (ctypes marshalling, torch for device
memory and streams).  ``BlockNorm``, ``VocabHead``, ``FeedForward`` and
``Checkpoint`` (``operators.py``) are the model operators around those sums: a
block's end with its norms, the vocabulary-parallel head's log probabilities
and distillation, the gated feed-forward block between two block ends, and
rows kept in 8 bits for the backward pass.
The binding is loaded on first use of one of its names,
so ``ring_allreduce_gb300.inputs`` can be imported on a machine where the
library has not been built.  Using the binding without the built library
raises ImportError: there is no CPU fallback.
"""

_BINDING_NAMES = {
    "ra_create", "ra_destroy", "ra_reduce_scatter", "ra_all_gather", "ra_allreduce",
    "ra_reduce_scatter_compact", "ra_all_gather_compact",
    "ra_chunk_plan", "ra_owned_chunk", "ra_set_option", "ra_get_option",
    "ra_get_device_status", "ra_read_signals", "ra_read_shadows", "ra_allreduce_noalloc", "ra_last_error", "ra_status_string",
    "RingAllReduce", "PreparedCall", "RAError", "Status", "DType", "Op", "Variant", "Barrier", "Option",
    "DeviceError", "load_library", "library_path",
}
_OPERATOR_NAMES = {"BlockNorm", "VocabHead", "FeedForward", "Checkpoint"}


def __getattr__(name):
    if name in _BINDING_NAMES:
        from . import binding
        return getattr(binding, name)
    if name in _OPERATOR_NAMES:
        from . import operators
        globals().update({n: getattr(operators, n) for n in _OPERATOR_NAMES})   # found directly from now on
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
