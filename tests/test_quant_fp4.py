"""quant_nvfp4, quant_mxfp4 and nvfp4_global_scale against their formulas in 64 bits, exactly: a block's scale is E4M3 of the
fp32 nearest to gs * amax / 6 (UE8M0: from amax's bits), and a code the nearest to the exact quotient by that scale, ties to
even. Quotients in 64 bits are off by 2^-53 of themselves; an exact one that is not on a boundary is off it by more than
that: x gs - t s is a multiple of the product of the last places of x and gs, at least 2^-47 of it."""
import pytest
import torch

import fp4_common as F
from gpu_common import guarded, guards_intact, rq

gpu = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(rows, hidden, dtype, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, hidden), generator=g, device="cuda")
    return (x * torch.exp2(spread * torch.randn((rows, 1), generator=g, device="cuda"))).to(dtype)


def run(x, fmt, gs=None, swizzled=False, **kw):
    if fmt == "nvfp4":
        t = None if gs is None else torch.tensor([gs], dtype=torch.float32, device="cuda")
        return rq().quant_nvfp4(x, global_scale=t, swizzled=swizzled, **kw)
    return rq().quant_mxfp4(x, swizzled=swizzled, **kw)


def check(x, fmt, gs=None, swizzled=False, **kw):
    rows, hidden, block = x.shape[0], x.shape[1], F.BLOCK[fmt]
    q, s = run(x, fmt, gs, swizzled, **kw)
    s = s.view(torch.uint8)
    if swizzled:
        s = F.untiled(s, rows, hidden // block)[0]
    parts = x.double().unflatten(1, (-1, block))
    amax = parts.abs().amax(-1)
    if fmt == "nvfp4":
        g32 = torch.tensor(1.0 if gs is None else gs, dtype=torch.float32, device="cuda")
        want = (g32.double() * amax / 6.0).float().clamp(max=448.0).to(torch.float8_e4m3fn)
        each = want.double()[:, :, None]
        t = torch.where(each > 0, parts * g32.double() / each, 0.0)
        want = want.view(torch.uint8)
    else:
        e = torch.ceil(torch.log2(amax / 6.0)).clamp(-127, 128) + 127
        # log2 rounds: one step too low or high is put right by the definition itself
        e = e + (6.0 * torch.exp2(e - 127) < amax).double()
        e = e - (6.0 * torch.exp2(e - 128) >= amax).double()
        e = torch.where(amax > 0, e, 0.0).clamp(0, 255)
        want = e.to(torch.uint8)
        t = torch.where(e[:, :, None] > 0, parts * torch.exp2(127.0 - e)[:, :, None], 0.0)
    assert torch.equal(s, want)
    value, got = F.nearest(t.flatten(1)), F.e2m1_values(q)
    assert torch.equal(got, value), int((got != value).sum())
    assert rq().rmsq_device_status() == 0
    return q, s


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("swizzled", [False, True])
@pytest.mark.parametrize("rows,blocks", [(1, 1), (1, 512), (2, 3), (31, 5), (128, 4), (129, 7), (300, 33), (257, 64), (1000, 18)])
def test_sizes(fmt, dtype, swizzled, rows, blocks):
    x = make(rows, blocks * F.BLOCK[fmt], dtype, rows + blocks)
    check(x, fmt, gs=2688.0 / float(x.float().abs().max()) if fmt == "nvfp4" else None, swizzled=swizzled)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gs", [None, 1.0, 64.0, 3.7, 0.013, 1e6])
def test_global_scales(dtype, gs):
    # far too small (blocks of scale 0) and far too large (scales that saturate) among them
    check(make(64, 512, dtype, 5, spread=4.0), "nvfp4", gs=gs)


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_ties(fmt, dtype):
    # every 16-bit value up to 6 beside a 6: with scale 1 the midpoints themselves, and what lies next to them
    bits = torch.arange(0, 32768, dtype=torch.int32, device="cuda").to(torch.int16)
    v = bits.view(dtype)
    v = v[torch.isfinite(v) & (v <= 6)]
    block = F.BLOCK[fmt]
    v = v[: v.numel() // (block - 1) * (block - 1)].reshape(-1, block - 1)
    x = torch.cat((torch.full((v.shape[0], 1), 6.0, dtype=dtype, device="cuda"), v * torch.where(
        torch.arange(block - 1, device="cuda") % 2 == 0, 1.0, -1.0).to(dtype)), 1)
    for f in (1.0, 0.25, 3.0, 5.0):        # scales of other mantissas
        check((x * f).contiguous(), fmt, gs=1.0)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("top", [1.0, 1.125, 2.625, 2.75, 3.0, 4.25, 5.25, 6.5625, 10.5, 21.0, 43.0])
def test_quotients_a_rounding_of_the_global_scale_off_a_boundary(dtype, top):
    # gs = 2688 / amax: quotients by it are ratios of small numbers, off by gs's rounding; tops whose mantissas share a
    # factor with 2688 make many of them boundaries, and many block scales too
    x = make(256, 2048, torch.bfloat16, 11).float().clamp(-top, top)
    x[0, 0] = top
    x = x.to(dtype)
    gs = float(rq().nvfp4_global_scale(x))
    assert gs == float(2688.0 * (torch.tensor(1.0) / top))
    for g in {gs, float(torch.tensor(2688.0) / torch.tensor(top))}:
        check(x, "nvfp4", gs=g)
        check(x, "nvfp4", gs=g, swizzled=True)


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_zeros_and_extremes(fmt, dtype):
    info = torch.finfo(dtype)
    x = torch.zeros((6, 64), dtype=dtype, device="cuda")
    x[1, 3] = info.max
    x[2, 40] = info.tiny
    x[3, :] = info.smallest_normal / 4            # subnormal
    x[4, ::2] = -info.max
    x[5, 0], x[5, 33] = 1.0, -1e-3
    check(x, fmt)


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("swizzled", [False, True])
def test_blocks_that_are_not_finite(fmt, dtype, swizzled):
    x = make(40, 256, dtype, 3)
    block = F.BLOCK[fmt]
    want, ws = run(x, fmt, 2.0, swizzled)
    x[3, 5], x[17, 70], x[39, 255] = float("nan"), float("inf"), float("-inf")
    q, s = run(x, fmt, 2.0, swizzled)
    s, ws = (F.untiled(t.view(torch.uint8), 40, 256 // block)[0] if swizzled else t.view(torch.uint8) for t in (s, ws))
    hit = torch.zeros((40, 256 // block), dtype=torch.bool, device="cuda")
    hit[3, 5 // block] = hit[17, 70 // block] = hit[39, 255 // block] = True
    assert bool((s[hit] == (0x7F if fmt == "nvfp4" else 255)).all()) and torch.equal(s[~hit], ws[~hit])
    same = ~hit.repeat_interleave(block // 2, 1)
    assert torch.equal(q[same], want[same])


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("power", [-105, -118, -124, -128])
def test_tensors_at_the_small_end_of_float(dtype, power):
    """Their global scale is as large as a float can be, and blocks below the normal floats have zeros among their elements."""
    g = torch.Generator(device="cuda").manual_seed(-power)
    x = torch.randn((64, 512), generator=g, device="cuda", dtype=torch.float64)
    x = x * torch.exp2(-8.0 * torch.rand((64, 32), generator=g, device="cuda", dtype=torch.float64)).repeat_interleave(16, 1)
    x[:, ::5] = 0.0
    x = (x * 2.0 ** power).float().to(dtype)
    assert bool((x != 0).any())
    check(x, "nvfp4", float(rq().nvfp4_global_scale(x)))
    check(x, "nvfp4", float(rq().nvfp4_global_scale(x)), swizzled=True)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_global_scale_below_the_normal_floats(dtype):
    x = make(64, 512, torch.float32, 6)
    x = (x / x.abs().max() * 2.0 ** 127).to(dtype)
    for gs in (1e-38, 3e-39, 2.0 ** -130 * 1.25):
        check(x, "nvfp4", gs)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_the_global_scale_of_a_tensor_with_a_nan(dtype):
    x = make(40, 256, dtype, 4)
    x[7, 9] = float("nan")
    gs = rq().nvfp4_global_scale(x)
    assert torch.isnan(gs).all()
    s = rq().quant_nvfp4(x, global_scale=gs)[1]
    assert bool((s.view(torch.uint8) == 0x7F).all())


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,blocks", [(5, 3), (130, 6), (128, 8)])
def test_nothing_else_is_written(fmt, rows, blocks):
    block = F.BLOCK[fmt]
    x = make(rows, blocks * block, torch.bfloat16, 1)
    for swizzled in (False, True):
        n = rq().swizzled_scale_numel(rows, blocks * block, block) if swizzled else rows * blocks
        out, raw1 = guarded(rows * blocks * block // 2, torch.uint8)
        scale, raw2 = guarded(n, torch.uint8)
        check(x, fmt, swizzled=swizzled, output=out.view(rows, -1), block_scale=scale if swizzled else scale.view(rows, -1))
        assert guards_intact([raw1, raw2])
        if swizzled:
            assert bool((F.untiled(scale, rows, blocks)[1] == 0x5A).all())       # the padding stays


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_past_32_bits(fmt):
    rows, hidden = 70000, 65536                       # over 2^32 elements
    x = torch.ones((rows, hidden), dtype=torch.bfloat16, device="cuda")
    tail = make(7, hidden, torch.bfloat16, 8)
    x[-7:] = tail
    q, s = run(x, fmt, 2.0, False)
    want, ws = run(tail, fmt, 2.0, False)
    assert torch.equal(q[-7:], want) and torch.equal(s[-7:].view(torch.uint8), ws.view(torch.uint8))
    q, s = run(x, fmt, 2.0, True)
    block = F.BLOCK[fmt]
    tiles = s.view(torch.uint8).reshape(-1, hidden // block // 4 * 512)[-1:].reshape(-1)
    assert torch.equal(F.untiled(tiles, 128, hidden // block)[0][(rows - 7) % 128:(rows - 1) % 128 + 1], ws.view(torch.uint8))
    assert torch.equal(q[-7:], want)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("count", [1, 3, 7, 8, 9, 1000, 4099, 65536, 65537, 131072, 131080, 1000003, 40000001])
def test_global_scale(dtype, count):
    x = make(1, count, dtype, count)[0]
    x[count // 2] = -77.0
    x[-1] = 80.0
    for _ in range(2):
        gs = rq().nvfp4_global_scale(x)
        assert float(gs) == float(2688.0 * (torch.tensor(1.0) / x.float().abs().max().cpu()))
        x[-1] = 0.5


@gpu
def test_global_scale_special_values():
    f = rq().nvfp4_global_scale
    for n in (24, 300000):
        x = torch.zeros(n, device="cuda")
        assert float(f(x)) == 1.0
        x[5] = 1e-42
        assert float(f(x)) == torch.finfo(torch.float32).max
        x[5] = float("inf")
        assert float(f(x)) == 0.0
        x[n - 1] = float("nan")
        assert torch.isnan(f(x)).all()
    assert float(f(torch.empty(0, device="cuda"))) == 1.0
    # what the workspace held before does not matter
    x, ws = torch.full((300000,), 3.0, device="cuda"), torch.full((4096,), 0xFF, dtype=torch.uint8, device="cuda")
    assert float(f(x, workspace=ws)) == 896.0
    assert float(f(x * 2, workspace=ws)) == 448.0


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_stream_graph_and_shapes(fmt):
    x = make(96, 512, torch.bfloat16, 2)

    def call(x, stream=None):
        if fmt == "mxfp4":
            return rq().quant_mxfp4(x, swizzled=True, stream=stream)
        gs = rq().nvfp4_global_scale(x, stream=stream)
        return rq().quant_nvfp4(x, global_scale=gs, swizzled=True, stream=stream)

    def same(got, w):            # codes and scales; the padding is nobody's
        a, b = (F.untiled(t[1].view(torch.uint8), 96, 512 // F.BLOCK[fmt])[0] for t in (got, w))
        return torch.equal(got[0], w[0]) and torch.equal(a, b)

    want, other = call(x), call(x * 3)
    q, s = call(x.view(2, 48, 512))
    assert q.shape == (2, 48, 256) and torch.equal(q.view(96, 256), want[0])
    x3 = x * 3
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        a, b = call(x, one), call(x3, two)
    torch.cuda.synchronize()
    assert same(a, want) and same(b, other)
    buf, graph = x.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(buf)
    for f, w in ((3.0, other), (1.0, want)):
        buf.copy_(x * f)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, w)


@gpu
def test_empty_calls_launch_nothing():
    before = rq().rmsq_launch_count()
    q, s = rq().quant_nvfp4(torch.empty((0, 64), device="cuda"), swizzled=True)
    assert q.shape == (0, 32) and s.numel() == 0
    assert rq().rmsq_launch_count() == before


def test_refusals_without_a_gpu():
    lib, A = rq().lib(), 1 << 20      # fake 16-byte aligned addresses: never dereferenced here

    def nv(x=A, rows=4, hidden=64, dt=0, gs=A, out=A, scale=A, layout=0):
        return lib.quant_nvfp4(x, rows, hidden, dt, gs, out, scale, layout, None)

    def mx(x=A, rows=4, hidden=64, dt=0, out=A, scale=A, layout=0):
        return lib.quant_mxfp4(x, rows, hidden, dt, out, scale, layout, None)

    for f in (nv, mx):
        assert all(f(**{a: None}) == 1 for a in ("x", "out", "scale"))
        assert f(rows=-1) == 2 and f(hidden=0) == 2 and f(hidden=72) == 2 and f(hidden=2 ** 31) == 2
        assert all(f(**{a: A + 8}) == 3 for a in ("x", "out", "scale"))
        assert f(dt=3) == 4 and f(layout=2) == 4
        assert f(rows=0, x=None) == 0
    assert nv(gs=A + 2) == 3 and mx(hidden=48) == 2

    def gs(x=A, n=100000, dt=0, out=A, ws=A, size=1 << 20):
        return lib.nvfp4_global_scale(x, n, dt, out, ws, size, None)

    assert all(gs(**{a: None}) == 1 for a in ("x", "out", "ws"))
    assert gs(n=-1) == 2 and gs(size=lib.nvfp4_global_scale_workspace(100000) - 1) == 2 and gs(dt=7) == 4
    assert gs(x=A + 4) == 3 and gs(ws=A + 4) == 3 and gs(out=A + 2) == 3
    assert lib.nvfp4_global_scale_workspace(0) == 0 and lib.nvfp4_global_scale_workspace(64) == 0


@gpu
def test_python_refusals():
    x, q = make(4, 64, torch.bfloat16, 0), rq()
    bad = [lambda: q.quant_nvfp4(x[:, :8].contiguous()), lambda: q.quant_mxfp4(x[:, :48].contiguous()),
           lambda: q.quant_nvfp4(x[:, ::2]), lambda: q.quant_nvfp4(x, output=torch.empty((4, 31), dtype=torch.uint8, device="cuda")),
           lambda: q.quant_mxfp4(x, block_scale=torch.empty(7, dtype=torch.uint8, device="cuda")),
           lambda: q.quant_nvfp4(x, global_scale=torch.ones(2, device="cuda")),
           lambda: q.quant_nvfp4(x, global_scale=torch.ones(1)), lambda: q.quant_nvfp4(x.cpu()),
           lambda: q.nvfp4_global_scale(x[:, ::2]), lambda: q.nvfp4_global_scale(x, out=torch.empty(2, device="cuda"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: q.quant_nvfp4(x.double()), lambda: q.nvfp4_global_scale(x.long())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(q.RmsqError):
        q.nvfp4_global_scale(torch.ones(100000, device="cuda"), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
