"""Checkpoint: rows kept in 8 bits, against the definition.  Codes and scales
are numbers that binary32 operations define, so they are compared exactly; what
comes back is rounded once."""

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -25}


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from ring_allreduce_gb300 import build
    build.build()
    from ring_allreduce_gb300 import operators
    return operators


def definition(v):
    """Codes and scales of the rows of a CPU or GPU tensor, every operation a rounding of its 64-bit result."""
    v = v.double()
    codes, scales = [], []
    for lo in range(0, v.shape[1], 128):
        x = v[:, lo:lo + 128]
        most = x.abs().amax(1, keepdim=True)
        some = most > 2.0 ** -110
        by = torch.where(some, (127.0 / most).float().double(), 0.0)
        codes.append((x * by).float().double().round())
        scales.append(torch.where(some, (most / 127.0).float(), 0.0))
    return torch.cat(codes, 1).to(torch.int8), torch.cat(scales, 1)


def padded(rows, width, dtype, pad, fill=7.0):
    big = torch.full((rows, width + pad), fill, device="cuda").to(dtype)
    return big, big[:, :width]


SHAPES = [(1, 1), (1, 128), (3, 7), (5, 129), (64, 256), (33, 1000), (300, 1538), (17, 4096), (2000, 640), (70000, 40)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("pad", [0, 3, 16])
def test_store_and_load(ops, dtype, T, D, pad):
    g = torch.Generator(device="cuda").manual_seed(T * 7 + D)
    dt = TORCH[dtype]
    _, x = padded(T, D, dt, pad)
    x.copy_(torch.randn((T, D), generator=g, device="cuda") * 3 * torch.rand((T, 1), generator=g, device="cuda"))
    x[:, D // 2] *= 20
    guard, codes = padded(T, D, torch.int8, pad)
    scales = torch.full((T, -(-D // 128)), 7.0, device="cuda")
    op = ops.Checkpoint(D, dtype)
    op.store(x, codes, scales)
    want, ws = definition(x)
    assert torch.equal(scales, ws)
    assert torch.equal(codes, want)
    assert (guard[:, D:] == 7).all()
    big, back = padded(T, D, dt, pad)
    op.load(codes, scales, back)
    v = codes.double() * scales.double().repeat_interleave(128, 1)[:, :D]
    assert ((back.double() - v).abs() <= U[dtype] * v.abs() + TINY[dtype]).all()
    assert (big[:, D:] == 7).all()
    # half a scale: the documented distance
    s = scales.double().repeat_interleave(128, 1)[:, :D]
    assert ((v - x.double()).abs() <= s * (0.5 + 127 * 3 * 2.0 ** -24)).all()


@pytest.mark.parametrize("dtype,normed,param", [("f32", "bf16", "f32"), ("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
                                                ("f16", "f16", "f32"), ("f32", "f16", "f16"), ("bf16", "f32", "f32")])
@pytest.mark.parametrize("T,D,pad", [(1, 64, 0), (77, 1032, 0), (400, 515, 5), (90, 2048, 8)])
def test_normalised_rows(ops, dtype, normed, param, T, D, pad):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    op = ops.Checkpoint(D, dtype, normed, param)
    _, codes = padded(T, D, torch.int8, pad)
    codes.copy_(torch.randint(-127, 128, (T, D), generator=g, device="cuda"))
    scales = torch.rand((T, -(-D // 128)), generator=g, device="cuda") + 0.01
    rstd = torch.rand(T, generator=g, device="cuda") + 0.1
    w = (torch.randn(D, generator=g, device="cuda") + 1).to(TORCH[param])
    v = codes.double() * scales.double().repeat_interleave(128, 1)[:, :D]
    z = v * rstd.double()[:, None] * w.double()
    for both in (True, False):
        big, got = padded(T, D, TORCH[normed], pad)
        back = padded(T, D, TORCH[dtype], pad)[1] if both else None
        op.load(codes, scales, back, rstd, w, got)
        # three products before the rounding
        assert ((got.double() - z).abs() <= (U[normed] * 1.0001 + 3 * 2.0 ** -24) * z.abs() + TINY[normed]).all()
        assert (big[:, D:] == 7).all()
        if both:
            assert ((back.double() - v).abs() <= U[dtype] * v.abs() + TINY[dtype]).all()


def test_what_a_group_cannot_hold(ops):
    """Infinities and NaN come back as NaN, in their group alone; tiny groups as zeros; the largest numbers as they are."""
    D = 300
    x = torch.randn((6, D), device="cuda")
    x[0, 5], x[1, 130], x[2, 299] = float("inf"), float("nan"), -float("inf")
    x[3, 128:256] = 2.0 ** -111
    x[4, :128] = 3.4e38
    x[5] = 0
    op = ops.Checkpoint(D, "f32")
    codes, scales = torch.empty((6, D), dtype=torch.int8, device="cuda"), torch.empty((6, 3), device="cuda")
    back = torch.empty_like(x)
    op.store(x, codes, scales)
    op.load(codes, scales, back)
    bad = torch.zeros((6, D), dtype=torch.bool, device="cuda")
    bad[0, :128] = bad[1, 128:256] = bad[2, 256:] = True
    assert torch.equal(back.isnan(), bad)
    assert (back[3, 128:256] == 0).all() and (back[5] == 0).all()
    # 127 x the rounded scale: two roundings
    assert ((back[4, :128] / 3.4e38 - 1).abs() <= 2.0 ** -22).all()
    ok = ~bad
    ok[3, 128:256] = ok[4, :128] = False
    most = torch.nn.functional.pad(x.nan_to_num(0, 0, 0).abs(), (0, 84)).view(6, 3, 128).amax(2)
    assert ((back - x).abs()[ok] <= (most / 253).repeat_interleave(128, 1)[:, :D][ok]).all()


def test_halves_go_to_even(ops):
    """Values half way between two codes."""
    x = torch.arange(-127, 1, device="cuda", dtype=torch.float32)[None] + 0.5
    x[0, 0] = 127.0
    op = ops.Checkpoint(128, "f32")
    codes, scales = torch.empty((1, 128), dtype=torch.int8, device="cuda"), torch.empty((1, 1), device="cuda")
    op.store(x, codes, scales)
    assert scales.item() == 1.0
    assert torch.equal(codes, x.round().to(torch.int8)) and codes[0, 126] == 0 and codes[0, 125] == -2


def test_offsets_beyond_32_bits(ops):
    """Rows 2^31 elements apart."""
    D, stride = 256, 2 ** 31 + 64
    big = torch.empty(2 * stride, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, D), (stride, 1))
    x.copy_(torch.randn((2, D), device="cuda"))
    space = torch.zeros(2 * stride, dtype=torch.int8, device="cuda")
    codes = space.as_strided((2, D), (stride, 1))
    scales = torch.empty((2, 2), device="cuda")
    op = ops.Checkpoint(D, "bf16")
    op.store(x, codes, scales)
    want, ws = definition(x)
    assert torch.equal(codes, want) and torch.equal(scales, ws)
    back = torch.empty((2, D), dtype=torch.bfloat16, device="cuda")
    op.load(codes, scales, back)
    v = want.double() * ws.double().repeat_interleave(128, 1)
    assert ((back.double() - v).abs() <= U["bf16"] * v.abs()).all()


def test_no_rows_and_capture(ops):
    op = ops.Checkpoint(40, "f32")
    e = torch.empty((0, 40), device="cuda")
    op.store(e, e.to(torch.int8), torch.empty((0, 1), device="cuda"))
    op.load(e.to(torch.int8), torch.empty((0, 1), device="cuda"), e)
    x, codes, scales = torch.randn((9, 40), device="cuda"), torch.zeros((9, 40), dtype=torch.int8, device="cuda"), torch.zeros((9, 1), device="cuda")
    back = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.store(x, codes, scales)
        op.load(codes, scales, back)
    x.normal_()
    op.close()
    graph.replay()
    want, ws = definition(x)
    assert torch.equal(codes, want) and torch.equal(back, (want.float() * ws))


def test_refusals(ops):
    from ring_allreduce_gb300 import RAError, Status
    op = ops.Checkpoint(64, "f32", "bf16")
    x, codes, scales = torch.zeros((4, 64), device="cuda"), torch.zeros((4, 64), dtype=torch.int8, device="cuda"), torch.zeros((4, 1), device="cuda")
    for bad in ((x.half(), codes, scales), (x, codes.to(torch.uint8), scales), (x, codes[:3], scales), (x, codes, scales.T),
                (x, codes, scales.double()), (x.cpu(), codes, scales), (x[:, :60], codes, scales), (None, codes, scales)):
        with pytest.raises(ValueError):
            op.store(*bad)
    z, r, w = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    for bad in ((x, None, w, z), (x, r, None, z), (x, r, w.float(), z), (x, r, w, z.float()), (x, r[:2], w, z)):
        with pytest.raises(ValueError):
            op.load(codes, scales, *bad)
    for args in ((codes, scales), (codes, scales, x[:1].expand(4, 64))):
        with pytest.raises(RAError) as err:
            op.load(*args)
        assert err.value.status == Status.ERR_INVALID
    big = torch.zeros((4, 64), device="cuda")
    with pytest.raises(RAError) as err:   # codes inside the values
        op.store(big, big.view(torch.int8)[:, :64], scales)
    assert err.value.status == Status.ERR_INVALID
