"""nvfp4_global_scale and the 4-bit quantisation at the ends of float's range, as include/rmsq.h states them."""
from fractions import Fraction

import pytest
import torch

import fp4_common as F
from gpu_common import rq

gpu = pytest.mark.gpu


def global_scales(tops, dtype, count):
    """The global scale of a tensor of `count` elements whose largest magnitude is tops[i], for every i."""
    x = torch.zeros((len(tops), count), dtype=dtype, device="cuda")
    x[:, count // 3] = torch.tensor(tops, dtype=torch.float64).to(dtype).cuda()
    got = torch.cat([rq().nvfp4_global_scale(row) for row in x]).cpu()
    return x[:, count // 3].float().cpu(), got


def units_off(top, gs):
    """How far gs is from 2688 / top, in units of the exact quotient's last place (a float's)."""
    exact = Fraction(2688) / Fraction(top)
    e = 0
    while Fraction(2) ** (e + 1) <= exact:
        e += 1
    while Fraction(2) ** e > exact:
        e -= 1
    return abs(Fraction(gs) - exact) / Fraction(2) ** (max(e, -126) - 23)


@gpu
@pytest.mark.parametrize("count", [40, 70000])
def test_the_global_scale_is_near_the_quotient(count):
    """Two roundings: half a unit of the last place, and the reciprocal's half unit times the ratio of the two mantissas, which is
    1.3125 at most (2688 = 1.3125 2^11): 1.16 units. One rounding where the reciprocal would be a subnormal float: half a unit."""
    g = torch.Generator().manual_seed(5)
    mantissas = [1.0, 1.0 + 2.0 ** -23, 1.3125, 1.5, 2.0 - 2.0 ** -23] + (1 + torch.rand(40, generator=g)).tolist()
    for power in (-100, -20, 0, 7, 60, 125, 126, 127):
        top, got = global_scales([m * 2.0 ** power for m in mantissas], torch.float32, count)
        off = [units_off(a, b) for a, b in zip(top.tolist(), got.tolist())]
        assert max(off) <= (Fraction(1, 2) if power > 126 else Fraction(116, 100)), (power, float(max(off)))
    for dtype in (torch.bfloat16, torch.float32):
        m = torch.finfo(dtype).max
        top, got = global_scales([m, m / 2, m / 4], dtype, count)
        assert max(units_off(a, b) for a, b in zip(top.tolist(), got.tolist())) <= Fraction(116, 100)


@gpu
@pytest.mark.parametrize("swizzled", [False, True])
def test_a_tensor_with_an_infinity_has_no_global_scale(swizzled):
    """It is 0; under it every block has scale 0 but the infinity's, and a product is NaN throughout."""
    q, g = rq(), torch.Generator(device="cuda").manual_seed(2)
    x, w = (torch.randn((n, 64), generator=g, device="cuda").bfloat16() for n in (6, 32))
    x[2, 40] = float("-inf")
    gs = q.nvfp4_global_scale(x)
    assert float(gs) == 0.0
    c, s = q.quant_nvfp4(x, global_scale=gs, swizzled=True)
    rows = F.untiled(s.view(torch.uint8), 6, 4)[0]
    hit = torch.zeros_like(rows, dtype=torch.bool)
    hit[2, 2] = True
    assert bool((rows[hit] == 0x7F).all()) and bool((rows[~hit] == 0).all())
    w4, ws = q.quant_nvfp4(w, swizzled=True)
    assert torch.isnan(q.matmul_nvfp4(c, s, w4, ws, input_global_scale=gs)).all()


@gpu
@pytest.mark.parametrize("swizzled", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mxfp4_blocks_of_the_smallest_scale_are_zeros(dtype, swizzled):
    """Blocks up to 6 2^-127, whose scale code is 0; one step above the code is 1 and the values stay."""
    top = torch.tensor(6.0 * 2.0 ** -127, dtype=torch.float64).to(dtype).cuda()
    above = torch.nextafter(top, torch.tensor(1.0, dtype=dtype, device="cuda"))
    x = torch.zeros((5, 64), dtype=dtype, device="cuda")
    x[0, 3], x[1, 3], x[2, 3], x[3, 40] = top, above, -top, -above
    x[4, :32] = 1.0
    c, s = rq().quant_mxfp4(x, swizzled=swizzled)
    s = F.untiled(s, 5, 2)[0] if swizzled else s
    assert s.tolist() == [[0, 0], [1, 0], [0, 0], [0, 1], [125, 0]]
    want = torch.zeros((5, 64), dtype=torch.float64, device="cuda")
    want[1, 3], want[3, 40] = 3.0 * 2.0 ** -126, -3.0 * 2.0 ** -126
    want[4, :32] = 1.0
    assert torch.equal(F.decoded(c, s, "mxfp4"), want)
