"""Checkpoint at the ends of binary32: groups whose largest magnitude is the
type's largest number, as masks of the type's lowest value are."""

import pytest

import test_gpu_checkpoint as c

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ops = c.ops


def test_only_the_largest_number_has_a_scale_of_its_own(ops):
    """The scale is m / 127 rounded for every other magnitude."""
    top = torch.tensor([torch.finfo(torch.float32).max])
    x = torch.cat([top, (top.view(torch.int32) - 1).view(torch.float32), (top.view(torch.int32) - 64).view(torch.float32),
                   torch.tensor([1e38, 2.0 ** -109])])[:, None].cuda()
    op = ops.Checkpoint(1, "f32")
    codes, scales = torch.empty((5, 1), dtype=torch.int8, device="cuda"), torch.empty((5, 1), device="cuda")
    op.store(x, codes, scales)
    want = (x.double() / 127).float()
    want[0, 0] = 8454659 * 2.0 ** 98
    assert torch.equal(scales, want) and (codes == 127).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [1, 128, 300, 1024])
def test_largest_numbers_come_back(ops, dtype, D):
    """Finite, and half a scale away at most, besides the roundings: the factor 127 / m, its product with the value
    and the scale (8454659 where m / 127 is 8454659.53) are off by 1, 1 and 1.06 units of 2^-24, of a code of
    127, and the result is rounded once."""
    info = torch.finfo(c.TORCH[dtype])
    x = torch.randn((4, D), device="cuda").to(c.TORCH[dtype])
    x[0, 0], x[1, -1], x[2] = info.max, info.min, info.min
    x[3] = torch.nextafter(torch.tensor(info.max).float(), torch.tensor(0.0)).to(x.dtype)
    op = ops.Checkpoint(D, dtype)
    codes, scales = torch.empty((4, D), dtype=torch.int8, device="cuda"), torch.empty((4, -(-D // 128)), device="cuda")
    back = torch.empty_like(x)
    op.store(x, codes, scales)
    op.load(codes, scales, back)
    assert torch.isfinite(back).all()
    s = scales.double().repeat_interleave(128, 1)[:, :D]
    tol = s * (0.5 + 4 * 127 * 2.0 ** -24) + c.U[dtype] * x.double().abs()
    assert ((back.double() - x.double()).abs() <= tol).all()
