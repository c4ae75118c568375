"""The model operators without a GPU: argument structures of the binding match
the header's, and refusals that come before any device call."""

import ctypes
import os
import re

import pytest

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "ra.h")


@pytest.fixture(scope="module")
def ops():
    from ring_allreduce_gb300 import build
    build.build()
    from ring_allreduce_gb300 import operators
    return operators


def _struct_fields(name):
    """Field names of a struct of ra.h, in order, with a size and kind each."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, flags=re.S).group(1)
    out = []
    for decl in body.split(";"):
        decl = " ".join(decl.split())
        if decl:
            kind = "pointer" if "*" in decl else "size" if decl.startswith("size_t") else "int"
            out.append((re.search(r"(\w+)$", decl).group(1), kind))
    return out


@pytest.mark.parametrize("name,cls", [
    ("ra_norm_forward_args", "_NormForward"), ("ra_norm_backward_args", "_NormBackward"),
    ("ra_vocab_logprobs_args", "_Logprobs"), ("ra_vocab_logprobs_backward_args", "_LogprobsBackward"),
    ("ra_vocab_distill_args", "_Distill"), ("ra_vocab_distill_backward_args", "_DistillBackward")])
def test_structures_match_the_header(ops, name, cls):
    kinds = {ctypes.c_void_p: "pointer", ctypes.c_size_t: "size", ctypes.c_int: "int"}
    got = [(n.rstrip("_"), kinds[t]) for n, t in getattr(ops, cls)._fields_]
    assert got == _struct_fields(name)


def test_null_handles_and_arguments(ops):
    lib = ops._lib
    for fn in (lib.ra_norm_forward, lib.ra_norm_backward, lib.ra_vocab_logprobs, lib.ra_vocab_logprobs_backward,
               lib.ra_vocab_distill, lib.ra_vocab_distill_backward):
        assert fn(None, None, None) == 1
    assert lib.ra_norm_destroy(None) == 0 and lib.ra_vocab_destroy(None) == 0
    assert lib.ra_norm_create(2, 64, 0, 0, 0, 1e-6, 1.0, None) == 1
    assert lib.ra_vocab_create(2, 64, 0, 1.0, None) == 1


@pytest.mark.parametrize("args,status", [
    ((0, 64, 0, 0, 0, 1e-6, 1.0), 1), ((33, 64, 0, 0, 0, 1e-6, 1.0), 1), ((2, 0, 0, 0, 0, 1e-6, 1.0), 1),
    ((2, 16385, 0, 0, 0, 1e-6, 1.0), 4), ((2, 64, 2, 2, 2, 1e-6, 1.0), 4), ((2, 64, 1, 3, 0, 1e-6, 1.0), 4),
    ((2, 64, 1, 0, 3, 1e-6, 1.0), 4), ((2, 64, 0, 0, 0, -1.0, 1.0), 1), ((2, 64, 0, 0, 0, float("nan"), 1.0), 1),
    ((2, 64, 0, 0, 0, 1e-6, float("inf")), 1)])
def test_norm_create_refuses(ops, args, status):
    h = ctypes.c_void_p()
    assert ops._lib.ra_norm_create(*args, ctypes.byref(h)) == status
    assert not h.value


@pytest.mark.parametrize("args,status", [
    ((0, 64, 0, 1.0), 1), ((33, 64, 0, 1.0), 1), ((2, 0, 0, 1.0), 1), ((2, 2 ** 30 + 1, 0, 1.0), 1),
    ((2, 64, 2, 1.0), 4), ((2, 64, 0, 0.0), 1), ((2, 64, 0, -2.0), 1), ((2, 64, 0, float("nan")), 1),
    ((2, 64, 0, float("inf")), 1)])
def test_vocab_create_refuses(ops, args, status):
    h = ctypes.c_void_p()
    assert ops._lib.ra_vocab_create(*args, ctypes.byref(h)) == status
    assert not h.value
