"""FeedForward and Checkpoint without a GPU: the extension's checks of tensors,
and refusals that come before any device call."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def ops():
    from ring_allreduce_gb300 import build
    build.build()
    from ring_allreduce_gb300 import operators
    return operators


def ffn_tensors(R=2, T=3, D=8, F=5):
    import torch
    dt = torch.bfloat16
    widths = [3, 2]
    return dict(xs=[torch.zeros(T, D, dtype=dt)], wg=[torch.zeros(n, D, dtype=dt) for n in widths],
                wu=[torch.zeros(n, D, dtype=dt) for n in widths], wd=[torch.zeros(n, D, dtype=dt) for n in widths],
                hidden=[torch.zeros(T, n, dtype=dt) for n in widths], parts=[torch.zeros(T, D, dtype=dt) for _ in range(R)],
                codes=[torch.zeros(T, n, dtype=torch.int8) for n in widths], scales=[torch.zeros(T, 1) for _ in widths])


# device -1 is the CPU: a fitting call goes through to the library, which refuses the NULL handle
CONFIG = (0, -1, 2, 8, 5, 1, 1)


def test_extension_checks_feed_forward(ops):
    import torch
    ext, t = ops._ext, ffn_tensors()
    ok = [t[k] for k in ("xs", "wg", "wu", "wd", "hidden", "parts")]
    none = [None] * 4
    kept = [t["codes"], t["codes"], t["scales"], t["scales"]]
    assert ext.ffn_forward(*CONFIG, *ok, *none, 0) == 1
    assert ext.ffn_forward(*CONFIG, *ok, *kept, 0) == 1
    assert ext.ffn_forward(*CONFIG, *ok, t["hidden"], t["hidden"], None, None, 0) == 1
    # a tensor with a leading axis, generators and tuples
    assert ext.ffn_forward(*CONFIG, torch.zeros(2, 3, 8, dtype=torch.bfloat16), (w for w in t["wg"]), tuple(t["wu"]),
                           *ok[3:], *kept, 0) == 1
    for k, bad in ((0, []), (0, 5), (0, None), (0, [torch.zeros(3, 8)]), (0, [torch.zeros(3, 9, dtype=torch.bfloat16)]),
                   (0, [t["xs"][0]] * 3), (1, t["wg"][:1]), (1, t["wg"][::-1]), (1, [t["wg"][0], 4]), (2, None),
                   (3, [w.t().contiguous().t() for w in t["wd"]]), (4, t["parts"]), (4, [h[:2] for h in t["hidden"]]),
                   (5, t["parts"][:1]), (5, [p.float() for p in t["parts"]])):
        with pytest.raises(ValueError):
            ext.ffn_forward(*CONFIG, *ok[:k], bad, *ok[k + 1:], *none, 0)
    for bad in ((t["codes"], None, None, None), (None, t["codes"], None, None), (t["codes"], t["codes"], None, None),
                (t["codes"], t["codes"], t["scales"], t["scales"][:1]), (t["codes"], t["hidden"], t["scales"], t["scales"]),
                (t["hidden"], t["hidden"], t["scales"], None), (None, None, t["scales"], t["scales"]), (3, 3, None, None)):
        with pytest.raises(ValueError):
            ext.ffn_forward(*CONFIG, *ok, *bad, 0)
    for args in ((), CONFIG, CONFIG + tuple(ok), ("a",) * 18):
        with pytest.raises(ValueError):
            ext.ffn_forward(*args)


def test_extension_checks_feed_forward_gradient(ops):
    ext, t = ops._ext, ffn_tensors()
    new = lambda: [h.clone() for h in t["hidden"]]   # noqa: E731
    args = dict(dy=[t["parts"][0]], xs=t["xs"], wg=t["wg"], wu=t["wu"], wd=t["wd"], gate=t["codes"], up=t["codes"],
                hidden=new(), dg=new(), du=new(), dx=t["parts"], gwg=t["wg"], gwu=t["wu"], gwd=t["wd"], gs=t["scales"],
                us=t["scales"])
    call = lambda **kw: ext.ffn_backward(*CONFIG, *{**args, **kw}.values(), 0)   # noqa: E731
    assert call() == 1
    # what is not wanted, and what only that needs, is not looked at
    assert call(dx=None, wg=None, wu=7, gwg=None, gwu=None, xs="x", gwd=None, hidden=None) == 1
    for bad in (dict(dy=None), dict(gate=None, up=None), dict(up=None), dict(wd=None), dict(dg=None), dict(du=t["codes"]),
                dict(wg=None), dict(xs=None), dict(gs=None), dict(us=t["scales"][:1]), dict(hidden=t["parts"]),
                dict(dx=t["parts"][:1]), dict(gwg=[w.float() for w in t["wg"]]), dict(gwd=[w.t() for w in t["wd"]])):
        with pytest.raises(ValueError):
            call(**bad)


def test_extension_checks_kept_rows(ops):
    import torch
    ext, x = ops._ext, torch.zeros(3, 200)
    config = (0, -1, 200, 0, 0, 0)
    q, s, r, w = torch.zeros(3, 200, dtype=torch.int8), torch.zeros(3, 2), torch.zeros(3), torch.zeros(200)
    assert ext.ckpt_store(*config, x, q, s, 0) == 1
    assert ext.ckpt_load(*config, q, s, x, r, w, x, 0) == 1
    assert ext.ckpt_load(*config, q, s, x, "not", "looked at", None, 0) == 1
    for bad in ((x.half(), q, s), (x, x, s), (x, q, s[:, :1]), (x, q[:2], s), (x.t(), q, s), (None, q, s), (x, q, None)):
        with pytest.raises(ValueError):
            ext.ckpt_store(*config, *bad, 0)
    for bad in ((q, s, x, None, w, x), (q, s, x, r, None, x), (q, s.double(), x, r, w, x), (q, s, x[:, :1], r, w, x),
                (q, s, x, r, w, x.half())):
        with pytest.raises(ValueError):
            ext.ckpt_load(*config, *bad, 0)


def test_null_handles_and_arguments(ops):
    lib = ops._lib
    for fn in (lib.ra_ffn_forward, lib.ra_ffn_backward, lib.ra_ckpt_store, lib.ra_ckpt_load):
        assert fn(None, None, None) == 1
    assert lib.ra_ffn_destroy(None) == 0 and lib.ra_ckpt_destroy(None) == 0
    assert lib.ra_ffn_create(2, 64, 64, 1, 0, 1, None) == 1
    assert lib.ra_ckpt_create(64, 0, 0, 0, None) == 1
    assert lib.ra_ffn_get_device_status(None, None, None) == 1
    assert lib.ra_ffn_set_option(None, 4, 1) == 1 and lib.ra_ckpt_set_option(None, 4, 1) == 1


@pytest.mark.parametrize("args,status", [
    ((0, 64, 64, 1, 0, 1), 1), ((33, 64, 64, 1, 0, 1), 1), ((2, 0, 64, 1, 0, 1), 1), ((2, 2 ** 20 + 1, 64, 1, 0, 1), 1),
    ((2, 64, 0, 1, 0, 1), 1), ((2, 64, 2 ** 24 + 1, 1, 0, 1), 1), ((2, 64, 64, 0, 0, 0), 4), ((2, 64, 64, 2, 0, 2), 4),
    ((2, 64, 64, 1, 0, 3), 4), ((2, 64, 64, 1, 2, 1), 1), ((2, 64, 64, 1, -1, 1), 1)])
def test_ffn_create_refuses(ops, args, status):
    h = ctypes.c_void_p()
    assert ops._lib.ra_ffn_create(*args, ctypes.byref(h)) == status
    assert not h.value


@pytest.mark.parametrize("args,status", [
    ((0, 0, 0, 0), 1), ((2 ** 24 + 1, 0, 0, 0), 1), ((64, 2, 0, 0), 4), ((64, 0, 2, 2), 4), ((64, 0, 1, 3), 4)])
def test_ckpt_create_refuses(ops, args, status):
    h = ctypes.c_void_p()
    assert ops._lib.ra_ckpt_create(*args, ctypes.byref(h)) == status
    assert not h.value


def test_python_arguments(ops):
    for kw in (dict(activation="tanh"), dict(dtype="f64"), dict(grad_dtype="i32"), dict(inner=-1)):
        with pytest.raises(ValueError):
            ops.FeedForward(**{**dict(R=2, dim=64, inner=64), **kw})
    for kw in (dict(dtype="i64"), dict(normed_dtype="f64"), dict(param_dtype="i32")):
        with pytest.raises(ValueError):
            ops.Checkpoint(64, **kw)
