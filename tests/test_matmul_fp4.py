"""matmul_nvfp4 and matmul_mxfp4 against the product of the decoded operands in 64 bits, at token counts where the
kernel changes, at ragged sizes, and at lengths that end inside an MMA's 64 elements with a padding of NaN scales.

Tolerance. Products of codes and scales are exact. Taking an MMA of 64 elements to be off by at most 2^-22 of the sum of
what it adds, its accumulator among it (four units of fp32 for its inner additions), a sum of K / 64 of them, at
most 8 parts, two factors (each formed with two roundings) and a bias is off by at most (K / 64 + 16) 2^-22 size, where
size is the sum of the terms' magnitudes; the output's rounding adds half a step h."""
import threading

import pytest
import torch

import fp4_common as F
from gpu_common import guarded, guards_intact, rq

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
FORMATS = ["nvfp4", "mxfp4"]
gpu = pytest.mark.gpu


def operand(rows, k, fmt, g, spread=1.0):
    packed = torch.randint(0, 256, (rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    wide = torch.randn((rows, k // F.BLOCK[fmt]), generator=g, device="cuda") * spread
    if fmt == "nvfp4":
        scale = (torch.exp2(wide) * 4).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        scale = (wide + 127).round().clamp(0, 254).to(torch.uint8)
    return packed, scale, F.tiled(scale, 0x7F if fmt == "nvfp4" else 0xFF)          # the padding: NaN


def make(m, n, k, fmt, seed, dtype=torch.bfloat16, bias=True, globals_=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a, sa, ta = operand(m, k, fmt, g)
    w, sw, tw = operand(n, k, fmt, g)
    one = lambda v: torch.tensor([v], device="cuda") if globals_ and fmt == "nvfp4" else None  # noqa: E731
    return dict(a=a, sa=sa, ta=ta, w=w, sw=sw, tw=tw, fmt=fmt, dtype=dtype, ga=one(37.5), gw=one(0.3),
                bias=torch.randn(n, generator=g, device="cuda").to(dtype) if bias else None)


def call(d, **kw):
    kw = dict(bias=d["bias"], out_dtype=d["dtype"], **kw)
    if d["fmt"] == "mxfp4":
        return rq().matmul_mxfp4(d["a"], d["ta"], d["w"], d["tw"], **kw)
    return rq().matmul_nvfp4(d["a"], d["ta"], d["w"], d["tw"], input_global_scale=d["ga"], weight_global_scale=d["gw"], **kw)


def check(d, **kw):
    out, t = call(d, **kw), d["dtype"]
    a, w = F.decoded(d["a"], d["sa"], d["fmt"]), F.decoded(d["w"], d["sw"], d["fmt"])
    e, size = a @ w.t(), a.abs() @ w.abs().t()
    if d["ga"] is not None:
        f = 1.0 / (d["ga"].double() * d["gw"].double())
        e, size = e * f, size * f
    if d["bias"] is not None:
        e = e + d["bias"].double()
        size = size + d["bias"].double().abs()
    h = torch.finfo(t).eps / 2
    low = 2.0 ** -25 if t == torch.float16 else 0.0
    fits = e.abs() < torch.finfo(t).max
    off, most = (out.double() - e).abs(), h * e.abs() + (a.shape[1] / 64 + 16) * 2.0 ** -22 * size * (1 + h) + low
    assert bool((off <= most)[fits].all()), (float((off - most)[fits].max()), int((off > most)[fits].sum()), off.numel())
    assert rq().rmsq_device_status() == 0
    return out


TOKENS = [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300, 513, 1000]


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", TOKENS)
@pytest.mark.parametrize("n,k", [(256, 512), (1000, 1056), (129, 96)])
def test_token_counts(fmt, m, n, k):
    check(make(m, n, k, fmt, seed=m + n, dtype=DTYPES[m % 3], bias=m % 2 == 0))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [1, 40, 200, 700])
@pytest.mark.parametrize("k", [32, 64, 96, 128, 160, 192, 224, 256, 288, 320, 416, 480, 512, 544, 1024, 2880, 4096, 4128, 16384])
def test_lengths(fmt, m, k):
    check(make(m, 384, k, fmt, seed=k, dtype=torch.float32))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [1, 20, 260])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 127, 128, 130, 255, 256, 257, 1001, 7168])
@pytest.mark.parametrize("dtype", DTYPES)
def test_channel_counts(fmt, m, n, dtype):
    check(make(m, n, 288, fmt, seed=n, dtype=dtype))


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", [(1, 300, 8192), (30, 300, 4096), (100, 200, 2048), (300, 520, 1024), (2, 130, 131072)])
def test_whole_numbers_are_exact(fmt, m, n, k):
    """Unit scales, codes of -1, 0 and 1 but for one column: sums are whole numbers below 2^24, in any order."""
    d = make(m, n, k, fmt, seed=7, dtype=torch.float32, bias=False, globals_=False)
    g = torch.Generator(device="cuda").manual_seed(1)
    for x in ("a", "w"):
        nibble = torch.tensor([0, 2, 10], device="cuda", dtype=torch.uint8)
        pick = nibble[torch.randint(0, 3, (*d[x].shape, 2), generator=g, device="cuda")]
        pick[:, 0, 0] = 7                                        # 6
        d[x] = pick[:, :, 0] + 16 * pick[:, :, 1]
    one = 0x38 if fmt == "nvfp4" else 127
    for s, t in (("sa", "ta"), ("sw", "tw")):
        d[s] = torch.full_like(d[s], one)
        d[t] = F.tiled(d[s], 0x7F if fmt == "nvfp4" else 0xFF)
    want = F.e2m1_values(d["a"]) @ F.e2m1_values(d["w"]).t()
    assert torch.equal(call(d).double(), want)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [1, 33, 300])
def test_each_block_has_its_own_scale(fmt, m):
    """One block at a time is not zero: what it gives shows which scales were taken."""
    n, k, block = 130, 512, F.BLOCK[fmt]
    d = make(m, n, k, fmt, seed=2, dtype=torch.float32, bias=False)
    a, w = d["a"], d["w"]
    for b in (0, 1, 3, 5, k // block - 1):
        d["a"], d["w"] = torch.zeros_like(a), torch.zeros_like(w)
        at = slice(b * block // 2, (b + 1) * block // 2)
        d["a"][:, at], d["w"][:, at] = a[:, at], w[:, at]
        check(d)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [2, 40, 130, 400])
def test_a_row_that_is_not_finite(fmt, m):
    d = make(m, 200, 544, fmt, seed=m)
    want = call(d)
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    d["sa"][m // 2, 3] = nan
    d["ta"] = F.tiled(d["sa"], nan)
    out = call(d)
    assert torch.isnan(out[m // 2]).all()
    rest = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(out[rest], want[rest])


@gpu
def test_scales_at_the_ends_of_their_range():
    d = make(20, 200, 512, "mxfp4", seed=1, dtype=torch.float32, bias=False)
    for low_a, low_w in ((0, 254), (254, 0), (30, 224), (127, 127)):
        d["sa"].fill_(low_a)
        d["sw"].fill_(low_w)
        d["ta"], d["tw"] = F.tiled(d["sa"], 255), F.tiled(d["sw"], 255)
        check(d)
    d = make(20, 200, 512, "nvfp4", seed=1, dtype=torch.float32, bias=False)
    for low_a, low_w in ((1, 126), (126, 1), (126, 126), (0, 5), (7, 8)):        # subnormal, largest, zero
        d["sa"].fill_(low_a)
        d["sw"].fill_(low_w)
        d["ta"], d["tw"] = F.tiled(d["sa"], 127), F.tiled(d["sw"], 127)
        check(d)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m", [1, 40, 130, 400])
def test_sums_past_the_range_of_float(m, dtype):
    """Scales of 2^100: every sum is 2^200 or more, of one sign per token."""
    d = make(m, 200, 512, "mxfp4", seed=m, dtype=dtype)
    d["w"] = (d["w"] | 0x11) & 0x77                        # at least 0.5, and positive
    d["a"] = (d["a"] | 0x11) & 0x77
    d["a"][::2] |= 0x88
    d["sa"].fill_(227)
    d["sw"].fill_(227)
    d["ta"], d["tw"] = F.tiled(d["sa"], 255), F.tiled(d["sw"], 255)
    out = call(d).float()
    assert (out[::2] == float("-inf")).all() and (out[1::2] == float("inf")).all()


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_large(fmt):
    check(make(2048, 4096, 4096, fmt, seed=4))
    check(make(2051, 5001, 1184, fmt, seed=5, dtype=torch.float16))


@gpu
@pytest.mark.parametrize("m", [65, 150, 260, 500, 1100])
@pytest.mark.parametrize("n,k", [(2100, 544), (5000, 1056), (11003, 288), (130, 2080)])
def test_many_tokens(m, n, k):
    check(make(m, n, k, FORMATS[m % 2], seed=m + n))


@gpu
@pytest.mark.parametrize("m", [1, 24, 60, 100, 300])
def test_first_call_of_a_thread(m):
    # a thread with no CUDA call of its own before; every tensor made elsewhere
    d = make(m, 500, 192, "nvfp4", seed=9)
    want = call(d)
    out = torch.zeros_like(want)
    errors = []

    def go():
        try:
            call(d, output=out)
        except Exception as e:
            errors.append(e)

    thread = threading.Thread(target=go)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not errors and torch.equal(out, want)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n", [(70000, 32768), (300, 8000000), (12, 3125000)])
def test_outputs_and_weights_past_32_bits(fmt, m, n):
    # rows and channels at the far end against a small call of the same tiles' rows
    k = 64
    d = make(m, n, k, fmt, seed=6, bias=False)
    out = call(d)
    rows, far = slice(m - 5, m), slice(n - 130, n)
    part = dict(d, a=d["a"][rows].contiguous(), sa=d["sa"][rows], w=d["w"][far].contiguous(), sw=d["sw"][far])
    part["ta"], part["tw"] = F.tiled(part["sa"], 0), F.tiled(part["sw"], 0)
    assert torch.equal(out[rows, far], call(part))       # one MMA of 64 elements either way


@gpu
@pytest.mark.parametrize("m", [1, 24, 100, 300])
def test_guard_bytes_and_leading_dimensions(m):
    d = make(m, 333, 224, "nvfp4", seed=9)
    out, raw = guarded(m * 333, torch.bfloat16)
    check(d, output=out.view(m, 333))
    assert guards_intact([raw])
    split = call(dict(d, a=d["a"].view(1, m, 112)))
    assert split.shape == (1, m, 333) and torch.equal(split[0], call(d))


@gpu
@pytest.mark.parametrize("m", [1, 50, 300])
def test_global_scales_are_read_on_the_device(m):
    d = make(m, 140, 256, "nvfp4", seed=3, dtype=torch.float32, bias=False)
    graph = torch.cuda.CUDAGraph()
    first = call(d)
    with torch.cuda.graph(graph):
        out = call(d)
    d["ga"].mul_(2)
    d["gw"].mul_(4)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out * 8, first)
    d["ga"] = d["gw"] = None
    check(d)


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [1, 24, 150, 520])
@pytest.mark.parametrize("first", ["norm", "quant"])
def test_quantise_then_product_eager_streams_and_graph(fmt, m, first):
    """A projection as a served model runs it, behind a norm with its residual or behind an attention: on two streams at
    once, and captured and replayed on new inputs."""
    k, n, q = 1056, 640, rq()
    g = torch.Generator(device="cuda").manual_seed(m)
    x, r = (torch.randn((m, k), generator=g, device="cuda").bfloat16() for _ in range(2))
    gamma = torch.ones(k, device="cuda").bfloat16()
    d = make(m, n, k, fmt, seed=m)
    fixed = torch.tensor([300.0], device="cuda")

    def chain(x, stream=None):
        kw = dict(stream=stream, swizzled=True)
        gs = None
        if fmt == "nvfp4":
            gs = fixed if first == "norm" else q.nvfp4_global_scale(x, stream=stream)
            kw["global_scale"] = gs
        norm = q.rmsnorm_quant_nvfp4 if fmt == "nvfp4" else q.rmsnorm_quant_mxfp4
        quant = q.quant_nvfp4 if fmt == "nvfp4" else q.quant_mxfp4
        c, s = norm(x, gamma, residual=r, **kw)[:2] if first == "norm" else quant(x, **kw)
        if fmt == "nvfp4":
            return c, s, q.matmul_nvfp4(c, s, d["w"], d["tw"], input_global_scale=gs, weight_global_scale=d["gw"],
                                        bias=d["bias"], stream=stream), gs
        return c, s, q.matmul_mxfp4(c, s, d["w"], d["tw"], bias=d["bias"], stream=stream), gs

    want = chain(x)
    rows = F.untiled(want[1].view(torch.uint8), m, k // F.BLOCK[fmt])[0]
    check(dict(d, a=want[0], sa=rows, ta=want[1], ga=want[3]))
    other, x2 = chain(x * 2), x * 2
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        a, b = chain(x, one), chain(x2, two)
    torch.cuda.synchronize()
    assert torch.equal(a[2], want[2]) and torch.equal(b[2], other[2])
    buf, graph = x.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(buf)
    for f, w in ((2.0, other), (1.0, want)):
        buf.copy_(x * f)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[2], w[2])
    assert q.rmsq_device_status() == 0


@gpu
def test_the_same_call_gives_the_same_bits():
    for m in (1, 48, 128, 600):
        d = make(m, 2000, 4096, "nvfp4", seed=m, dtype=torch.float32)
        first = call(d)
        for _ in range(5):
            assert torch.equal(call(d), first)


@gpu
def test_empty_calls_launch_nothing():
    d = make(4, 8, 32, "mxfp4", seed=0, bias=False)
    before = rq().rmsq_launch_count()
    assert rq().matmul_mxfp4(d["a"][:0], d["ta"][:0], d["w"], d["tw"]).shape == (0, 8)
    assert rq().matmul_mxfp4(d["a"], d["ta"], d["w"][:0], d["tw"][:0]).shape == (4, 0)
    assert rq().rmsq_launch_count() == before


def test_refusals_without_a_gpu():
    lib, A = rq().lib(), 1 << 20      # fake 16-byte aligned addresses: never dereferenced here

    def nv(a=A, sa=A, ga=A, w=A, sw=A, gw=A, b=None, m=4, n=8, k=32, out=A, dt=0):
        return lib.matmul_nvfp4(a, sa, ga, w, sw, gw, b, m, n, k, out, dt, None)

    def mx(a=A, sa=A, w=A, sw=A, b=None, m=4, n=8, k=32, out=A, dt=0):
        return lib.matmul_mxfp4(a, sa, w, sw, b, m, n, k, out, dt, None)

    for mm in (nv, mx):
        assert all(mm(**{x: None}) == 1 for x in ("a", "sa", "w", "sw", "out"))
        assert mm(k=0) == 2 and mm(k=16) == 2 and mm(k=48) == 2 and mm(k=131104) == 2 and mm(m=-1) == 2 and mm(n=-1) == 2
        assert mm(m=8388609) == 2 and mm(n=8388609) == 2
        assert all(mm(**{x: A + 8}) == 3 for x in ("a", "sa", "w", "sw", "b", "out"))
        assert mm(dt=3) == 4
        assert mm(m=0, a=None) == 0 and mm(n=0, w=None) == 0
    assert nv(ga=A + 2) == 3 and nv(gw=A + 1) == 3


@gpu
def test_python_refusals():
    d, q = make(4, 8, 64, "nvfp4", seed=0), rq()
    a, ta, w, tw = d["a"], d["ta"], d["w"], d["tw"]
    nv = q.matmul_nvfp4
    bad = [lambda: nv(a, ta, w[:, :16], tw), lambda: nv(a, ta[:-1], w, tw), lambda: nv(a, ta, w, tw[:-16]),
           lambda: nv(a, ta.float(), w, tw), lambda: nv(a, ta, w, tw, bias=torch.ones(8, device="cuda")),
           lambda: nv(a, ta, w.t().contiguous().t(), tw), lambda: nv(a.t().contiguous().t(), ta, w, tw),
           lambda: nv(a, ta, w, tw, input_global_scale=torch.ones(1)),
           lambda: nv(a, ta, w, tw, weight_global_scale=torch.ones(1, device="cuda").half()),
           lambda: nv(a, ta, w, tw, output=torch.empty(4, 7, dtype=torch.bfloat16, device="cuda")),
           lambda: nv(a, ta, w, tw, output=torch.empty(4, 8, dtype=torch.float16, device="cuda")),
           lambda: q.matmul_mxfp4(a, torch.cat((ta, ta)), w, tw)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        nv(a.view(torch.int8), ta, w, tw)
    with pytest.raises(TypeError):
        nv(a, ta, w, tw, out_dtype=torch.float64)
    with pytest.raises(q.RmsqError):
        nv(a[:, :8].contiguous(), ta, w[:, :8].contiguous(), tw)
