"""How the model operators may be called."""

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
