"""matmul_int8 against the product in 64-bit integers, at token counts where the kernel changes, at
ragged sizes, and with codes whose sums are as large as they get.

Tolerance. The integer sum is exact; it is rounded to fp32 once, multiplied by two scales and the
bias added (four roundings of u = 2^-24), then rounded to the output's type (half a step h):
|out - exact| <= h |exact| + 4 u (|exact - bias| + |bias|) (1 + h), and half an fp16 subnormal step."""
import threading

import pytest
import torch

from gpu_common import guarded, guards_intact, rq

U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
gpu = pytest.mark.gpu


def make(m, n, k, seed, dtype=torch.bfloat16, bias=True, codes="random"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    a, w = r(m, k), r(n, k)
    if codes == "lowest":
        a.fill_(-128)
        w.fill_(-128)
    elif codes == "highest":
        a.fill_(127)
        w.fill_(-128)
    elif codes == "odd_ends":          # large sums whose last bit matters
        a.fill_(127)
        w.fill_(127)
        w[:, -1] = torch.arange(n, device="cuda").remainder(255).sub(127).to(torch.int8)
        a[:, 0] = 1
    f = lambda s: torch.rand(s, generator=g, device="cuda") * 1e-2 + 1e-4  # noqa: E731
    return dict(a=a, w=w, sa=f(m), sw=f(n),
                bias=torch.randn(n, generator=g, device="cuda").to(dtype) if bias else None, dtype=dtype)


def check(d, **kw):
    t = d["dtype"]
    out = rq().matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"], out_dtype=t, **kw)
    # products of codes are whole numbers: sums below 2^53 are exact in fp64 in any order
    e = (d["a"].double() @ d["w"].double().t()) * d["sa"].double()[:, None] * d["sw"].double()[None, :]
    size = e.abs()
    if d["bias"] is not None:
        e = e + d["bias"].double()
        size = size + d["bias"].double().abs()
    h = torch.finfo(t).eps / 2
    low = 2.0 ** -25 if t == torch.float16 else 0.0
    off = (out.double() - e).abs()
    fits = e.abs() < torch.finfo(t).max
    assert bool((off <= h * e.abs() + 4 * U * size * (1 + h) + low)[fits].all()), float(off[fits].max())
    assert rq().rmsq_device_status() == 0
    return out


TOKENS = [1, 2, 3, 5, 8, 9, 16, 17, 31, 33, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300, 513]


@gpu
@pytest.mark.parametrize("m", TOKENS)
@pytest.mark.parametrize("n,k", [(256, 512), (1000, 1040), (129, 48)])
def test_token_counts(m, n, k):
    check(make(m, n, k, seed=m + n, dtype=DTYPES[m % 3], bias=m % 2 == 0))


@gpu
@pytest.mark.parametrize("m", [1, 7, 40, 200, 700])
@pytest.mark.parametrize("k", [16, 32, 64, 80, 128, 1008, 1024, 1040, 2032, 2048, 4096, 5120, 16384])
def test_lengths(m, k):
    check(make(m, 384, k, seed=k, dtype=torch.float32))


@gpu
@pytest.mark.parametrize("m", [1, 20, 260])
@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 127, 128, 130, 255, 257, 1001, 7168])
@pytest.mark.parametrize("dtype", DTYPES)
def test_channel_counts(m, n, dtype):
    check(make(m, n, 272, seed=n, dtype=dtype))


@gpu
@pytest.mark.parametrize("codes", ["lowest", "highest", "odd_ends"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 131056), (4, 130, 20000), (33, 200, 131056), (300, 260, 8192),
                                   (257, 513, 33008)])
def test_largest_sums_are_exact(codes, m, n, k):
    d = make(m, n, k, seed=1, dtype=torch.float32, bias=False, codes=codes)
    d["sa"].fill_(1.0)
    d["sw"].fill_(1.0)
    out = check(d)
    # with unit scales the output is the whole sum, rounded to fp32 once
    want = (d["a"].double() @ d["w"].double().t()).float()
    assert torch.equal(out, want)


@gpu
@pytest.mark.parametrize("m", [3, 48, 512])
def test_unit_scales_give_whole_numbers(m):
    d = make(m, 300, 1024, seed=m, dtype=torch.float32, bias=False)
    d["sa"].fill_(1.0)
    d["sw"].fill_(1.0)
    assert torch.equal(check(d), (d["a"].double() @ d["w"].double().t()).float())


@gpu
def test_large():
    check(make(2048, 4096, 8192, seed=4))
    check(make(4099, 5001, 1232, seed=5, dtype=torch.float16))


@gpu
@pytest.mark.parametrize("m", [1, 8, 11, 16])
@pytest.mark.parametrize("n", [1, 17, 7296, 7297, 12007])
def test_few_tokens_around_a_wave_of_narrow_ctas(m, n):
    check(make(m, n, 1104, seed=m + n))


@gpu
@pytest.mark.parametrize("m", [65, 100, 150, 200, 260, 500, 700, 1100])
@pytest.mark.parametrize("n,k", [(2100, 528), (5000, 1040), (11003, 272), (130, 2064)])
def test_each_kernel_for_many_tokens(m, n, k):
    # widths at which tiles of 128 (with and without a shared k) and pairs of 128 and 192 tokens are taken
    check(make(m, n, k, seed=m + n))


@gpu
@pytest.mark.parametrize("m", [1, 12, 24, 60, 100, 300])
def test_first_call_of_a_thread(m):
    # a thread with no CUDA call of its own before; every tensor made elsewhere
    d = make(m, 500, 192, seed=9)
    want = rq().matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"])
    out = torch.zeros_like(want)
    errors = []

    def call():
        try:
            rq().matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"], output=out)
        except Exception as e:
            errors.append(e)

    thread = threading.Thread(target=call)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not errors and torch.equal(out, want)


@gpu
@pytest.mark.parametrize("m,n", [(70000, 32768), (300, 8000000), (12, 3125000)])
def test_outputs_and_weights_past_32_bits(m, n):
    # outputs of over 2^31 elements (first two); rows and channels at the far end against a small call
    k = 64
    d = make(m, n, k, seed=6, bias=False)
    out = rq().matmul_int8(d["a"], d["sa"], d["w"], d["sw"])
    far = slice(n - 130, n)
    want = rq().matmul_int8(d["a"][-5:].contiguous(), d["sa"][-5:].clone(), d["w"][far].contiguous(), d["sw"][far].clone())
    assert torch.equal(out[-5:, far], want)


@gpu
@pytest.mark.parametrize("m", [1, 12, 100, 300])
def test_guard_bytes_and_leading_dimensions(m):
    d = make(m, 333, 208, seed=9)
    out, raw = guarded(m * 333, torch.bfloat16)
    check(d, output=out.view(m, 333))
    assert guards_intact([raw])
    whole = rq().matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"])
    split = rq().matmul_int8(d["a"].view(1, m, 208), d["sa"].view(1, m), d["w"], d["sw"], bias=d["bias"])
    assert split.shape == (1, m, 333) and torch.equal(split[0], whole)


@gpu
def test_rows_do_not_depend_on_their_batch():
    """A token's row is the same bits whatever batch it comes in: sums are exact and the rest is
    done per element, so a decode step repeats what the prompt gave."""
    d = make(600, 520, 2064, seed=3, dtype=torch.float32)
    whole = check(d)
    for m in (1, 2, 6, 16, 50, 130, 300):
        part = rq().matmul_int8(d["a"][:m], d["sa"][:m], d["w"], d["sw"], bias=d["bias"], out_dtype=torch.float32)
        assert torch.equal(part, whole[:m]), m


@gpu
def test_empty_calls_launch_nothing():
    d = make(4, 8, 32, seed=0)
    before = rq().rmsq_launch_count()
    assert rq().matmul_int8(d["a"][:0], d["sa"][:0], d["w"], d["sw"]).shape == (0, 8)
    assert rq().matmul_int8(d["a"], d["sa"], d["w"][:0], d["sw"][:0]).shape == (4, 0)
    assert rq().rmsq_launch_count() == before


@gpu
@pytest.mark.parametrize("m", [1, 24, 520])
@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_norm_then_product_eager_stream_and_graph(norm, m):
    """The projection behind a norm, as a served model runs it: residual add, norm, int8 rows,
    product with bias; on a side stream, and captured and replayed on new inputs. Two of them on two
    streams at once give what each gives alone."""
    k, n = 1536 + 16, 640
    q = rq()
    g = torch.Generator(device="cuda").manual_seed(m)
    x, r = (torch.randn((m, k), generator=g, device="cuda").bfloat16() for _ in range(2))
    gamma, beta = torch.ones(k, device="cuda").bfloat16(), torch.zeros(k, device="cuda").bfloat16()
    d = make(m, n, k, seed=m)

    def chain(x, stream=None):
        if norm == "layer":
            c, s, _ = q.layernorm_quant_int8(x, gamma, beta, residual=r, stream=stream)
        else:
            c, s, _ = q.rmsnorm_quant_int8(x, gamma, residual=r, stream=stream)
        return c, s, q.matmul_int8(c, s, d["w"], d["sw"], bias=d["bias"], stream=stream)

    want = chain(x)
    check(dict(d, a=want[0], sa=want[1]))
    other = chain(x * 2)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    x2 = x * 2
    torch.cuda.synchronize()
    for _ in range(20):
        a, b = chain(x, one), chain(x2, two)
    torch.cuda.synchronize()
    assert all(torch.equal(p, w) for p, w in zip(a, want)) and all(torch.equal(p, w) for p, w in zip(b, other))
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(buf)
    for f in (1.0, 2.0):
        buf.copy_(x * f)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, w) for p, w in zip(out, want if f == 1.0 else other))
    assert q.rmsq_device_status() == 0


def test_refusals_without_a_gpu():
    lib, A = rq().lib(), 1 << 20      # fake 16-byte aligned addresses: never dereferenced here

    def mm(a=A, sa=A, w=A, sw=A, b=None, m=4, n=8, k=32, out=A, dt=0):
        return lib.matmul_int8(a, sa, w, sw, b, m, n, k, out, dt, None)

    assert all(mm(**{x: None}) == 1 for x in ("a", "sa", "w", "sw", "out"))
    assert mm(k=0) == 2 and mm(k=24) == 2 and mm(k=131072) == 2 and mm(m=-1) == 2 and mm(n=-1) == 2
    assert mm(m=8388609) == 2 and mm(n=8388609) == 2
    assert all(mm(**{x: A + 4}) == 3 for x in ("a", "sa", "w", "sw", "b", "out"))
    assert mm(dt=3) == 4
    assert mm(m=0, a=None) == 0 and mm(n=0, w=None) == 0


@gpu
def test_python_refusals():
    d, mm = make(4, 8, 32, seed=0), rq().matmul_int8
    a, sa, w, sw = d["a"], d["sa"], d["w"], d["sw"]
    bad = [lambda: mm(a, sa, w[:, :16], sw), lambda: mm(a, sa[:3], w, sw), lambda: mm(a, sa, w, sw[:7]),
           lambda: mm(a, sa.double(), w, sw), lambda: mm(a, sa, w, sw, bias=sw),
           lambda: mm(a, sa, w.t().contiguous().t(), sw), lambda: mm(a.t().contiguous().t(), sa, w, sw),
           lambda: mm(a, sa, w, sw, output=torch.empty(4, 7, dtype=torch.bfloat16, device="cuda")),
           lambda: mm(a, sa, w, sw, output=torch.empty(4, 8, dtype=torch.float16, device="cuda"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mm(a.float(), sa, w, sw)
    with pytest.raises(TypeError):
        mm(a, sa, w, sw, out_dtype=torch.float64)
    with pytest.raises(rq().RmsqError):
        mm(a[:, :8].contiguous(), sa, w[:, :8].contiguous(), sw)
