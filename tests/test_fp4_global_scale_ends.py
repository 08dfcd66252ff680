"""matmul_nvfp4 under global scales from the subnormal floats to the largest one: the factor 1 / (gs_a gs_w) may be past float's
range, or below it, where the products with it are not.

Tolerance. As for ordinary scales (test_matmul_fp4.py: (K / 64 + 16) 2^-22 of the terms' magnitudes and half a step of the
output); and where results are subnormal floats, the two products with the factor's parts and their sum are each off
by at most half of 2^-149, the output's rounding by half of its own type's smallest step."""
import pytest
import torch

import fp4_common as F
from gpu_common import rq
from test_matmul_fp4 import DTYPES, call, make

gpu = pytest.mark.gpu
MOST = torch.finfo(torch.float32).max
STEP = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}        # smallest ones

# their products: about 2^-133, 2^133, 2^138, 2^139, 2^256, 2^-138, 2^-279, 2^-12, 2^101, 2^-101, 2^-98
SCALES = [(1e-20, 1e-20), (1e20, 1e20), (2.0 ** 127, 2000.0), (MOST, 2688.0), (MOST, MOST), (2.0 ** -140, 3.0),
          (2.0 ** -140, 1.5 * 2.0 ** -140), (MOST, 2.0 ** -140), (1.1 * 2.0 ** 50, 1.7 * 2.0 ** 50), (1.1 * 2.0 ** -50, 1.7 * 2.0 ** -52),
          (1.3 * 2.0 ** -30, 1.9 * 2.0 ** -69)]


def operands(m, n, k, dtype, ga, gw, bias, seed, big):
    """`big`: block scales near the largest, so that sums are near 2^24; otherwise around 4."""
    d = make(m, n, k, "nvfp4", seed, dtype=dtype, bias=bias)
    if big:
        for s, t in (("sa", "ta"), ("sw", "tw")):
            d[s] = d[s] % 8 + 0x76                       # 224 to 448, none a NaN
            d[t] = F.tiled(d[s], 0x7F)
    d["a"][m // 2] = 0                                   # a token of nothing
    d["ga"], d["gw"] = (torch.tensor([v], dtype=torch.float32, device="cuda") for v in (ga, gw))
    return d


def check(d):
    out, t, dead = call(d), d["dtype"], d["a"].shape[0] // 2
    a, w = F.decoded(d["a"], d["sa"], "nvfp4"), F.decoded(d["w"], d["sw"], "nvfp4")
    p = d["ga"].double() * d["gw"].double()
    e, size = a @ w.t() / p, a.abs() @ w.abs().t() / p
    b = torch.zeros(out.shape[1], dtype=torch.float64, device="cuda") if d["bias"] is None else d["bias"].double()
    e, size = e + b, size + b.abs()
    h, top = torch.finfo(t).eps / 2, torch.finfo(t).max
    most = (a.shape[1] / 64 + 16) * 2.0 ** -22 * size * (1 + h)
    fits = e.abs() + most < top
    off, allowed = (out.double() - e).abs(), h * e.abs() + most + STEP[t] / 2 + 1.5 * 2.0 ** -149
    assert bool((off <= allowed)[fits].all()), (float((off / allowed)[fits].max()), int((off > allowed)[fits].sum()))
    past = e.abs() * (1 - h) - most > top               # surely past the type's range: an infinity of the right sign
    assert torch.equal(out[past].double(), torch.copysign(torch.full_like(e[past], float("inf")), e[past]))
    assert torch.equal(out[dead].double(), b)           # nothing added up is 0, whatever the factor
    assert not torch.isnan(out).any() and rq().rmsq_device_status() == 0
    return int(fits.sum()), int(past.sum())


# tiles of 16, 32, 64 and 128 tokens with and without shared k, and CTA pairs
@gpu
@pytest.mark.parametrize("ga,gw", SCALES)
@pytest.mark.parametrize("m,n,k", [(2, 130, 512), (24, 200, 2048), (64, 4096, 544), (130, 384, 1024), (2048, 2100, 512)])
def test_scales_whose_product_is_far_from_one(m, n, k, ga, gw):
    for i, dtype in enumerate(DTYPES):
        check(operands(m, n, k, dtype, ga, gw, bias=(m + i) % 2 == 0, seed=m + i, big=False))


@gpu
@pytest.mark.parametrize("m", [2, 24, 130, 600])
@pytest.mark.parametrize("ga,gw", [(MOST, 2688.0), (2.0 ** 127, 2688.0), (2.0 ** 126 * 1.25, 0.75 * 2.0 ** 14), (1.7e38, 1.0)])
def test_large_sums_under_the_global_scale_of_a_small_tensor(m, ga, gw):
    """Results are ordinary floats, with all of their bits."""
    for dtype in (torch.float32, torch.bfloat16):
        fits, past = check(operands(m, 300, 1024, dtype, ga, gw, bias=False, seed=m, big=True))
        assert fits == m * 300 and past == 0


@gpu
def test_from_a_small_tensor_to_its_product():
    """quant_nvfp4 of a tensor around 2^-118, whose global scale is nearly as large as a float can be, times a weight."""
    q, g = rq(), torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((40, 512), generator=g, device="cuda") * 2.0 ** -118
    w = torch.randn((256, 512), generator=g, device="cuda") * 0.02
    x[7] = 0
    gx, gw = q.nvfp4_global_scale(x), q.nvfp4_global_scale(w)
    assert float(gx) > 2.0 ** 126
    (a, sa), (b, sb) = (q.quant_nvfp4(v, global_scale=s, swizzled=True) for v, s in ((x, gx), (w, gw)))
    rows = lambda s, n: F.untiled(s.view(torch.uint8), n, 32)[0]  # noqa: E731
    d = dict(a=a, sa=rows(sa, 40), ta=sa, w=b, sw=rows(sb, 256), tw=sb, fmt="nvfp4", dtype=torch.float32, ga=gx, gw=gw, bias=None)
    out = call(d)
    e = F.decoded(a, d["sa"], "nvfp4") @ F.decoded(b, d["sw"], "nvfp4").t() / (gx.double() * gw.double())
    size = F.decoded(a, d["sa"], "nvfp4").abs() @ F.decoded(b, d["sw"], "nvfp4").abs().t() / (gx.double() * gw.double())
    assert bool(((out.double() - e).abs() <= 2.0 ** -24 * e.abs() + 24 * 2.0 ** -22 * size + 2.0 ** -148).all())
    assert bool((out[7] == 0).all())
