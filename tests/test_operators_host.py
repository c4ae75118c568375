"""The model operators without a GPU: the extension's checks of tensors, and
refusals that come before any device call."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def ops():
    from ring_allreduce_gb300 import build
    build.build()
    from ring_allreduce_gb300 import operators
    return operators


def test_extension_refuses_what_is_no_tensor(ops):
    """The extension's own checks, on CPU tensors and things that are none: ValueError, and nothing is called."""
    import torch
    ext = ops._ext
    x, w = torch.zeros(3, 8), torch.ones(8)
    norm = (0, 0, 2, 8, 0, 0, 0)      # a NULL handle on device 0
    for args in ((), norm, ("a",) * 17, norm + ([x, x], x, w, [x], x, None, None, None, None, 0),
                 norm + ([x, x], 5, w, [x], x, None, None, None, None, 0),
                 norm + ([x, 7], x, w, [x], x, None, None, None, None, 0),
                 norm + (3, x, w, [x], x, None, None, None, None, 0)):
        with pytest.raises(ValueError):
            ext.norm_forward(*args)
    # device -1 is the CPU: a fitting call goes through to the library, which refuses the NULL handle
    cpu = (0, -1, 2, 8, 0, 0, 0)
    assert ext.norm_forward(*cpu, [x, x], x, w, [x], x, None, None, None, None, 0) == 1
    assert ext.norm_forward(*cpu, torch.zeros(2, 3, 8), x, w, torch.zeros(1, 3, 8), x, w, None, None, None, 0) == 1
    for bad in ((torch.zeros(3, 3, 8), x), (torch.zeros(2, 3, 8).double(), x), (torch.zeros(2, 4, 8), x),
                ([x], x), ([x, x.t().contiguous().t()], x), ([x, torch.zeros(3, 16)[:, :8]], x),
                ([x, x], x.to_sparse()), ([x, x], torch.zeros(8))):
        with pytest.raises(ValueError):
            ext.norm_forward(*cpu, bad[0], bad[1], w, [x], x, None, None, None, None, 0)
    head = (0, -1, 2, 5, 0)
    s = [torch.zeros(3, 3), torch.zeros(3, 2)]
    t, f = torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    assert ext.logprobs(*head, s, t, f, f, None, None, None, 0) == 1
    for bad in ((s[:1], t, f, f, None, None, None), (s, t.int(), f, f, None, None, None), (s, t, f, x, None, None, None),
                (s, t, f, f, None, torch.zeros(3, 2, dtype=torch.int64), None)):
        with pytest.raises(ValueError):
            ext.logprobs(*head, *bad, 0)


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


@pytest.mark.parametrize("tau,status", [(4e-39, 1), (2.9e-39, 1)])
def test_vocab_create_refuses_a_temperature_whose_factor_is_infinite(ops, tau, status):
    """log2(e) / temperature has to be a binary32 number, not 1 / temperature alone."""
    h = ctypes.c_void_p()
    assert ops._lib.ra_vocab_create(2, 64, 0, tau, ctypes.byref(h)) == status
    assert not h.value
