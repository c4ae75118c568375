"""How the model operators may be called."""

import ctypes
import gc
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_gb300 import build
    build.build()
    from ring_allreduce_gb300 import operators
    return operators


@pytest.mark.parametrize("captured", [False, True])
def test_gradients_of_no_rows_are_zero(ops, captured):
    """A micro-batch without tokens: the sums over its rows are written, as zeros."""
    D, G = 72, 3
    op = ops.BlockNorm(2, D, "bf16")
    e, r = torch.empty((0, D), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 0), device="cuda")
    w, gate = torch.ones(D, dtype=torch.bfloat16, device="cuda"), torch.ones((G, D), dtype=torch.bfloat16, device="cuda")
    sums = [torch.full(s, 9.0, device="cuda") for s in ((D + 2,), (D + 2,), (G + 1, D))]
    gw, gp, gg = sums[0][1:-1], sums[1][1:-1], sums[2][:G]   # what lies beside them stays

    def call():
        op.backward([e, e], e, e, r, w, [e], e, gw, post_weight=w, gate=gate, total=e, grad_post_weight=gp, grad_gate=gg)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        assert all((s == 9).all() for s in sums)
        graph.replay()
    else:
        call()
    for s in (gw, gp, gg):
        assert (s == 0).all()
    assert (sums[0][[0, -1]] == 9).all() and (sums[1][[0, -1]] == 9).all() and (sums[2][G] == 9).all()
    op.backward([e, e], None, e, r, w, [e], e)   # none asked for


def test_refusals_without_rows(ops):
    from ring_allreduce_gb300 import RAError, Status
    op = ops.BlockNorm(1, 8, "f32")
    e, r, w = torch.empty((0, 8), device="cuda"), torch.empty((2, 0), device="cuda"), torch.ones(8, device="cuda")
    for kw in (dict(grad_post_weight=torch.ones(8, device="cuda")), dict(grad_weight=w, post_weight=w, grad_post_weight=w)):
        with pytest.raises(RAError) as err:
            op.backward([e], None, e, r, w, [e], e, **kw)
        assert err.value.status == Status.ERR_INVALID


class ForwardArgs(ctypes.Structure):   # ra_norm_forward_args
    _fields_ = [(n, ctypes.c_int if n == "outs" else ctypes.c_size_t if n == "rows" or n.endswith("stride") or
                 n == "gate_rows" else ctypes.c_void_p) for n in
                ("rows in in_stride residual residual_stride weight post_weight gate gate_rows out out_stride outs "
                 "residual_out residual_out_stride total total_stride rstd").split()]


def test_widths_from_two_host_threads(ops):
    """Handles of one type and two widths, each called from a host thread of its own through the C entries: their
    launches need different amounts of shared memory of one kernel."""
    from ring_allreduce_gb300 import binding
    lib, T = binding._lib, 320
    failures = []

    def work(dim):
        h, st = ctypes.c_void_p(), torch.cuda.Stream()
        assert lib.ra_norm_create(1, dim, 1, 1, 1, 1e-6, 1.0, ctypes.byref(h)) == 0
        with torch.cuda.stream(st):
            b = [torch.ones((T, dim), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
            w = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
        st.synchronize()
        ins, outs = (ctypes.c_void_p * 1)(b[0].data_ptr()), (ctypes.c_void_p * 1)(b[1].data_ptr())
        a = ForwardArgs(rows=T, in_stride=dim, residual=b[2].data_ptr(), residual_stride=dim, weight=w.data_ptr(),
                        out=ctypes.addressof(outs), out_stride=dim, outs=1, residual_out=b[3].data_ptr(),
                        residual_out_stride=dim)
        setattr(a, "in", ctypes.addressof(ins))
        for _ in range(3000):
            status = lib.ra_norm_forward(h, ctypes.addressof(a), st.cuda_stream)
            if status:
                failures.append((dim, status, binding.ra_last_error()))
                break
        st.synchronize()
        if not (b[3] == 2).all():
            failures.append((dim, "residual_out"))
        lib.ra_norm_destroy(h)

    threads = [threading.Thread(target=work, args=(dim,)) for dim in (8192, 16384, 12288)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures


def backward_case(R, T, D):
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    return ([r(T, D) for _ in range(R)], r(T, D), r(T, D), r(2, T).abs(), r(D)), ([r(T, D)], r(T, D), r(D))


def test_a_graph_outlives_its_handle(ops):
    """A captured backward pass keeps the handle's workspace: the handle may be closed, and other handles made."""
    args, want = backward_case(2, 700, 512)
    outs = [want[0][0], want[1], want[2]]
    got = [torch.zeros_like(o) for o in outs]
    op = ops.BlockNorm(2, 512, "f32")
    op.backward(*args, want[0], want[1], want[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.backward(*args, [got[0]], got[1], got[2])
    op.close()
    del op
    gc.collect()
    other = ops.BlockNorm(2, 512, "f32")
    sums = torch.zeros_like(want[2])
    for _ in range(3):
        for t in got:
            t.fill_(9.0)
        graph.replay()
        other.backward(*[[2 * p for p in args[0]], *args[1:]], [torch.empty_like(want[1])], torch.empty_like(want[1]), sums)
        for a, b in zip(got, outs):
            assert torch.equal(a, b)


def test_workspaces_are_given_back(ops):
    """Closed handles and dropped graphs leave no device memory behind (a workspace here has 40 MB)."""
    args, (gin, gh, gw) = backward_case(1, 4, 16384)
    graph = None

    def one():
        nonlocal graph
        op = ops.BlockNorm(1, 16384, "f32")
        op.backward(*args, gin, gh, gw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op.backward(*args, gin, gh, gw)
            op.backward(*args, gin, gh, gw)
        op.close()
        graph.replay()
        torch.cuda.synchronize()

    one()
    before = torch.cuda.mem_get_info()[0]
    for _ in range(40):
        one()
    assert before - torch.cuda.mem_get_info()[0] < 400 << 20


def test_what_does_not_fit_beside_a_stream(ops):
    """ValueError whether or not the caller names a stream; what a call does not look at may be anything."""
    op = ops.BlockNorm(2, 64, "f32")
    x, y, z, h = (torch.zeros((6, 64), device="cuda") for _ in range(4))
    w = torch.ones(64, device="cuda")
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        for bad in ([x, 7], [x, None], [x, y.cpu()], [x], 7, [x, y.half()], x.cpu()):
            with pytest.raises(ValueError):
                op.forward(bad, z, w, [h], torch.empty_like(z), stream=stream)
        with pytest.raises(ValueError):
            op.forward([x, y], z, w, [h], torch.empty_like(z), rstd=5, stream=stream)
        op.forward((t for t in (x, y)), z, w, [h], torch.empty_like(z), stream=stream)
    # five columns over four ranks: the last shard has none and is not looked at
    head = ops.VocabHead(4, 5, "f32")
    assert head.widths == [2, 2, 1, 0]
    s = [torch.zeros((6, 2), device="cuda"), torch.zeros((6, 2), device="cuda"), torch.zeros((6, 1), device="cuda")]
    t, lp, lse = torch.zeros(6, dtype=torch.int64, device="cuda"), torch.zeros(6, device="cuda"), torch.zeros(6, device="cuda")
    for last in (None, torch.zeros(6, 0), 3):
        for stream in (None, side, side.cuda_stream):
            lse.zero_()
            torch.cuda.synchronize()
            head.logprobs([*s, last], t, lp, lse, stream=stream)
            # entropy without its gradient is not looked at either
            head.logprobs_backward([*s, last], t, lse, lp, [*(torch.zeros_like(q) for q in s), last], entropy=lp.cpu(),
                                   stream=stream)
            torch.cuda.synchronize()
            assert torch.allclose(lse, torch.full_like(lse, 5.0).log())
