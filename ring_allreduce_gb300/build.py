"""Build the CUDA library libra_gb300.so in-tree, for sm_103a only.

``python -m ring_allreduce_gb300.build`` (or ``build()``) compiles every
translation unit under ``csrc/`` with nvcc in parallel into ``_build/`` and
links ``libra_gb300.so`` next to this file.  Nothing is rebuilt when the
library is newer than every source and header and the flags are unchanged.
Set RA_PTXAS_VERBOSE=1 to print ptxas register / spill / shared-memory use.
``build(debug=True)`` builds ``libra_gb300_debug.so`` from the same sources
with -DRA_DEBUG_BOUNDS (into ``_build_debug/``): every global access of every
kernel is checked against the byte ranges registered for the call, and
violations are counted and skipped (``ra_debug_bounds_report``).
"""

import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libra_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
TORCH_EXT = "_ra_torch"   # the Python extension that marshals torch tensors for the model operators
TORCH_EXT_PATH = os.path.join(HERE, TORCH_EXT + ".so")
DEBUG_BUILD_DIR = os.path.join(HERE, "_build_debug")
DEBUG_LIB_PATH = os.path.join(HERE, "libra_gb300_debug.so")

SOURCES = ["ra_host.cpp", "ra_direct.cu", "ra_round.cu", "ra_persistent.cu", "ra_pipelined.cu", "ra_compact.cu",
           "ra_bcast.cu", "ra_static.cu", "ra_local.cu", "ra_ll.cu", "ra_ops_host.cpp", "ra_norm.cu", "ra_vocab.cu",
           "ra_ffn_host.cpp", "ra_ffn_simple.cu", "ra_ckpt.cu"]
# (source, object stem, preprocessor definitions): ra_direct_inst.cu is
# compiled once per dtype so its instantiations build in parallel
DTYPES = ["RA_F32", "RA_BF16", "RA_I32", "RA_F16", "RA_F64", "RA_I64"]
# ... and ra_norm_inst.cu per pair of activations' and residual stream's types
NORM_TYPES = [("DF32", "DF32"), ("DBF16", "DBF16"), ("DBF16", "DF32"), ("DF16", "DF16"), ("DF16", "DF32")]
UNITS = ([(src, os.path.splitext(src)[0], {}) for src in SOURCES] +
         [("ra_direct_inst.cu", "ra_direct_" + dt[3:].lower(), {"RA_INST_DTYPE": dt}) for dt in DTYPES] +
         [("ra_ffn_mma_inst.cu", "ra_ffn_mma_" + dt[3:].lower(), {"RA_INST_DTYPE": dt}) for dt in ("RA_BF16", "RA_F16")] +
         [("ra_norm_inst.cu", f"ra_norm_{d}_{rd}".lower(), {"RA_INST_D": d, "RA_INST_RD": rd})
          for d, rd in NORM_TYPES])
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# IEEE arithmetic throughout: no fast-math, no flush to zero, no contraction.
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-ftz=false",
         "-prec-div=true", "-prec-sqrt=true", "-fmad=false"]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libra_gb300.so")
    return cand


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "ra.h"))
    files.append(os.path.abspath(__file__))
    return sorted(f for f in files if os.path.isfile(f))


# The files each kernel's device code is built from.
KERNEL_SOURCES = {
    "direct": ["ra_direct.cu", "ra_direct.cuh", "ra_direct_inst.cu", "ra_device.cuh", "ra_internal.h"],
    "round": ["ra_round.cu", "ra_device.cuh", "ra_internal.h"],
    "persistent": ["ra_persistent.cu", "ra_signal.cuh", "ra_device.cuh", "ra_internal.h"],
    "pipelined": ["ra_pipelined.cu", "ra_signal.cuh", "ra_device.cuh", "ra_internal.h"],
    "compact": ["ra_compact.cu", "ra_device.cuh", "ra_internal.h"],
    "bcast": ["ra_bcast.cu", "ra_device.cuh", "ra_internal.h"],
    "local": ["ra_local.cu", "ra_device.cuh", "ra_internal.h"],
    "ll": ["ra_ll.cu", "ra_ll.h", "ra_device.cuh", "ra_internal.h"],
    "norm": ["ra_norm.cu", "ra_norm.cuh", "ra_norm_inst.cu", "ra_ops.cuh", "ra_ops.h", "ra_device.cuh", "ra_internal.h"],
    "vocab": ["ra_vocab.cu", "ra_ops.cuh", "ra_ops.h", "ra_device.cuh", "ra_internal.h"],
    "ffn": ["ra_ffn_mma_inst.cu", "ra_ffn_few.cuh", "ra_ffn_mma.cuh", "ra_ffn_mma.h", "ra_tensor.cuh", "ra_ffn_simple.cu", "ra_ffn.cuh",
            "ra_ffn.h", "ra_ops.cuh", "ra_ops.h", "ra_device.cuh", "ra_internal.h"],
    "ckpt": ["ra_ckpt.cu", "ra_ffn.cuh", "ra_ffn.h", "ra_ops.cuh", "ra_ops.h", "ra_device.cuh", "ra_internal.h"],
}


def kernel_source_hash(kernel=None):
    """Short hash of the sources of one kernel (``KERNEL_SOURCES``), or of
    every CUDA / C++ source and the public header when ``kernel`` is None.
    A profile summary taken on another hash describes a different kernel."""
    h = hashlib.sha256()
    files = KERNEL_SOURCES[kernel] if kernel else sorted(os.listdir(CSRC))
    for f in files:
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(f.encode() + b"\0" + fh.read())
    if kernel is None:
        with open(os.path.join(INCLUDE, "ra.h"), "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


def _stamp(extra):
    h = hashlib.sha256(" ".join(ARCH + FLAGS + extra).encode())
    for f in _inputs():
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def _torch_dir():
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    return spec.submodule_search_locations[0]


def _build_torch_ext(force=False):
    """Compile _ra_torch.so against the installed torch; its own stamp, since
    that is what it depends on beside its source."""
    import importlib.metadata
    src = os.path.join(CSRC, "ra_torch.cpp")
    torch_dir = _torch_dir()
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"),
           "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), src,
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-Wl,-rpath," + os.path.join(torch_dir, "lib")]
    h = hashlib.sha256(" ".join(cmd + [sys.version, importlib.metadata.version("torch")]).encode())
    for f in (src, os.path.join(INCLUDE, "ra.h")):
        with open(f, "rb") as fh:
            h.update(fh.read())
    os.makedirs(BUILD_DIR, exist_ok=True)
    stamp_file = os.path.join(BUILD_DIR, "stamp_torch")
    if not force and os.path.exists(TORCH_EXT_PATH) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read().strip() == h.hexdigest():
                return
    tmp = TORCH_EXT_PATH + ".tmp"
    res = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("the compiler failed\n" + res.stdout + res.stderr)
    os.replace(tmp, TORCH_EXT_PATH)
    with open(stamp_file, "w") as f:
        f.write(h.hexdigest())


def _try_torch_ext(force=False):
    """Build the extension; why it could not be, or None.  The library serves C
    callers too and needs neither torch nor Python's headers; an extension of
    another header is worse than none."""
    try:
        _build_torch_ext(force)
        return None
    except Exception as e:
        if os.path.exists(TORCH_EXT_PATH):
            os.remove(TORCH_EXT_PATH)
        return f"{TORCH_EXT}.so (for the model operators on torch tensors) was not built: {e}\n"


def build(force=False, verbose=None, jobs=None, debug=False):
    """Compile and link the library (the bounds-checked one with debug=True);
    returns its path.  The Python extension is built beside it; that it could
    not be is written to stderr, and importing the operators then fails."""
    verbose = os.environ.get("RA_PTXAS_VERBOSE") == "1" if verbose is None else verbose
    extra = (["-Xptxas", "-v"] if verbose else []) + (["-DRA_DEBUG_BOUNDS"] if debug else [])
    build_dir, lib_path = (DEBUG_BUILD_DIR, DEBUG_LIB_PATH) if debug else (BUILD_DIR, LIB_PATH)
    stamp = _stamp(extra)
    stamp_file = os.path.join(build_dir, "stamp")
    if not force and os.path.exists(lib_path) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read().strip() == stamp:
                sys.stderr.write(_try_torch_ext() or "")
                return lib_path
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(unit):
        src, stem, defs = unit
        obj = os.path.join(build_dir, stem + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, *[f"-D{k}={v}" for k, v in defs.items()],
               "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        return stem, obj, res

    with ThreadPoolExecutor(max_workers=jobs or min(len(UNITS) + 1, os.cpu_count() or 4)) as ex:
        ext = ex.submit(_try_torch_ext, force)
        results = list(ex.map(compile_one, UNITS))
        sys.stderr.write(ext.result() or "")
    failed = [(s, r) for s, _, r in results if r.returncode != 0]
    for s, _, r in results:
        if verbose or r.returncode != 0:
            sys.stderr.write(f"--- {s}\n{r.stdout}{r.stderr}")
    if failed:
        raise RuntimeError("nvcc failed for " + ", ".join(s for s, _ in failed))
    objs = [o for _, o, _ in results]
    tmp = lib_path + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"link of {os.path.basename(lib_path)} failed")
    os.replace(tmp, lib_path)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
