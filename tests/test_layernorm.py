"""layernorm, layernorm_backward, layernorm_quant_int8 and rmsnorm_quant_int8 against their
formulas in 64 bits, at the widths where the row's owner changes (a warp to 1024 elements, a CTA to
16384, 8192 backward, then clusters), at widths that are no whole vectors, and at degenerate rows.

Tolerances. u = 2^-24 is half a step of fp32, h = finfo(t).eps / 2 half a step of the output type.
A sum over a row is at most 32 terms in a thread, then at most 14 levels of pairwise adds, so its
error is at most 46 u times the sum of magnitudes; the few products behind it keep it under K = 64.
 - y: an error of the mean (64 u mean|s|) and of rstd (64 u relative) reach y through rstd |w|, so
   |y - exact| <= h |exact| + K u (rstd |w| (mean|s| + |s - mean|) + |beta|) + one fp16 subnormal step.
 - ds: the same with |g| + mean|g| + |xhat| mean|g xhat| in place of the norm's terms; xhat is formed
   from fp32 statistics, which the 64-bit formula takes as they are.
 - dgamma, dbeta: `rows` terms in some order: (rows + K) u times the sum of magnitudes.
 - codes: |q - exact y / exact scale| <= 1/2 + (error of y) / scale + 127 * 4 u."""
import pytest
import torch

from gpu_common import guarded, guards_intact, rq

U = 2.0 ** -24
K = 64
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
gpu = pytest.mark.gpu


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return 2.0 ** -24 if t == torch.float16 else 0.0


def make(rows, hidden, dtype, seed, residual=False, beta=True, offset=0.0, centre=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return dict(x=(n(rows, hidden) + centre).to(dtype), gamma=(n(hidden) * 0.2 + 1.0 - offset).to(dtype),
                beta=(n(hidden) * 0.2).to(dtype) if beta else None,
                residual=n(rows, hidden).to(dtype) if residual else None)


def formula(s, gamma, beta, offset, eps, rms=False):
    """(y, mean, rstd, bound on the fp32 error of y) in 64 bits."""
    s, w = s.double(), gamma.double() + offset
    mean = torch.zeros_like(s[:, :1]) if rms else s.mean(1, keepdim=True)
    d = s - mean
    rstd = (d.square().mean(1, keepdim=True) + eps).rsqrt()
    b = beta.double() if beta is not None else torch.zeros_like(w)
    y = d * rstd * w + b
    err = K * U * (rstd * w.abs() * (s.abs().mean(1, keepdim=True) + d.abs()) + b.abs())
    return y, mean[:, 0], rstd[:, 0], err


def check_forward(d, offset=0.0, eps=1e-5):
    y, res, mean, rstd = rq().layernorm(d["x"], d["gamma"], d["beta"], residual=d["residual"],
                                        epsilon=eps, weight_offset=offset, stats=True)
    s = d["x"]
    if d["residual"] is not None:
        s = (d["x"].double() + d["residual"].double()).to(s.dtype)
        assert torch.equal(res, s)
    ey, em, er, err = formula(s, d["gamma"], d["beta"], offset, eps)
    t = s.dtype
    assert ((y.double() - ey).abs() <= half_step(t) * ey.abs() + err * (1 + half_step(t)) + tiny(t)).all()
    assert ((mean.double() - em).abs() <= K * U * s.double().abs().mean(1)).all()
    assert ((rstd.double() / er - 1).abs() <= K * U * (1 + em.square() * er.square())).all()


# widths: one element, inside a vector, both sides of every change of plan, odd, wide
WIDTHS = [1, 2, 7, 8, 31, 64, 250, 256, 257, 512, 520, 1000, 1024, 1025, 1032, 2051, 4096, 5120,
          8191, 8192, 8200, 16384]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", WIDTHS)
def test_forward_widths(dtype, hidden):
    rows = 37
    check_forward(make(rows, hidden, dtype, seed=hidden, residual=hidden % 2 == 0))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", [16385, 16400, 22761, 32768, 40008, 65536])
def test_forward_clusters(dtype, hidden):
    check_forward(make(5, hidden, dtype, seed=hidden, residual=True), offset=1.0)


@gpu
@pytest.mark.parametrize("hidden", [131072, 131071])
def test_forward_widest(hidden):
    check_forward(make(3, hidden, torch.bfloat16, seed=1))


@gpu
@pytest.mark.parametrize("rows", [1, 2, 8, 9, 1000, 70001])
@pytest.mark.parametrize("hidden", [96, 2048])
def test_forward_rows(rows, hidden):
    check_forward(make(rows, hidden, torch.bfloat16, seed=rows, beta=rows % 2 == 0), offset=1.0)


@gpu
@pytest.mark.parametrize("hidden", [8193, 9000, 12000, 16377, 16376, 16384, 32761, 32769, 32776, 65529, 65537, 65544])
def test_forward_around_each_plan(hidden):
    # where rows are packed, take a cluster of 4, of 8; with and without a residual
    check_forward(make(6, hidden, torch.bfloat16, seed=hidden))
    check_forward(make(6, hidden, torch.float16, seed=hidden, residual=True))


@gpu
@pytest.mark.parametrize("hidden", [16381, 16382, 32765, 32766, 32772, 65533, 65535])
def test_forward_around_each_plan_fp32(hidden):
    check_forward(make(6, hidden, torch.float32, seed=hidden))


@gpu
@pytest.mark.parametrize("hidden", [96, 1024, 4096, 12000, 16384, 20000, 65536])
@pytest.mark.parametrize("residual", [False, True])
def test_a_rows_bits_do_not_depend_on_the_other_rows(hidden, residual):
    d = make(700, hidden, torch.bfloat16, seed=hidden, residual=residual)
    cut = lambda t, n: None if t is None else t[:n].contiguous()  # noqa: E731
    for f in (rq().layernorm, rq().layernorm_quant_int8):
        many = f(d["x"], d["gamma"], d["beta"], residual=d["residual"])
        one = f(cut(d["x"], 3), d["gamma"], d["beta"], residual=cut(d["residual"], 3))
        assert all(torch.equal(a[:3], b) for a, b in zip(many, one) if a is not None)


@gpu
def test_forward_far_off_centre():
    # variance is formed about the mean: rows whose mean is 1000 times their spread keep it
    d = make(64, 4096, torch.float32, seed=5, centre=1000.0)
    check_forward(d)


@gpu
def test_offsets_past_32_bits():
    # 34000 x 65536 elements: the last rows start past 2^31 elements and 2^32 bytes
    rows, hidden = 34000, 65536
    x = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda")
    x[:-3].fill_(1.0)
    x[-3:].copy_(torch.randn(3, hidden, device="cuda"))
    gamma = (torch.randn(hidden, device="cuda") * 0.2 + 1.0).bfloat16()
    y, _, mean, rstd = rq().layernorm(x, gamma, stats=True)
    few = rq().layernorm(x[-3:].contiguous(), gamma, stats=True)
    assert torch.equal(y[-3:], few[0]) and torch.equal(mean[-3:], few[2]) and not y[:-3].any()
    q, scale, _ = rq().rmsnorm_quant_int8(x, gamma)
    fewq = rq().rmsnorm_quant_int8(x[-3:].contiguous(), gamma)
    assert torch.equal(q[-3:], fewq[0]) and torch.equal(scale[-3:], fewq[1])
    del q
    ds, dg, _ = rq().layernorm_backward(x, x, gamma, mean, rstd, grad_input=y, param_grad_dtype=torch.float32)
    fewb = rq().layernorm_backward(x[-3:].contiguous(), x[-3:].contiguous(), gamma, mean[-3:].clone(),
                                   rstd[-3:].clone(), param_grad_dtype=torch.float32)
    # the rows of ones have xhat = 0, so they add nothing to dgamma; other rows' sums differ in order
    assert torch.equal(ds[-3:], fewb[0])
    assert ((dg - fewb[1]).abs() <= 8 * U * (x[-3:].double().abs() * 8).sum(0)).all()


@gpu
@pytest.mark.parametrize("hidden", [96, 1003, 1024, 5121, 16384, 20000, 66001])
def test_int8_rows_that_are_not_finite_get_scale_nan(hidden):
    x = torch.randn(9, hidden, device="cuda").bfloat16()
    x[2, hidden - 1] = float("nan")
    x[4, hidden // 2] = float("inf")
    x[7, 0] = -float("inf")
    gamma = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    bad = torch.tensor([2, 4, 7], device="cuda")
    good = torch.tensor([0, 1, 3, 5, 6, 8], device="cuda")
    finite = x.clone()
    finite[bad] = 1.0
    for f in (rq().layernorm_quant_int8, rq().rmsnorm_quant_int8):
        q, scale, _ = f(x, gamma)
        assert scale[bad].isnan().all()
        # the same rows at the same places (their order of summing goes by the row's place at odd widths)
        want = f(finite, gamma)
        assert torch.equal(q[good], want[0][good]) and torch.equal(scale[good], want[1][good])


@gpu
def test_backward_far_off_centre():
    d = make(200, 2000, torch.float32, seed=3, centre=1000.0)
    d["dy"] = torch.randn_like(d["x"])
    d["dres"] = None
    x = d["x"].double()
    d["mean"] = x.mean(1).float()
    d["rstd"] = (x.var(1, correction=0) + 1e-5).rsqrt().float()
    check_backward(d)


@gpu
def test_constant_rows_give_beta():
    x = torch.full((5, 2048), 3.0, dtype=torch.float32, device="cuda")
    g = torch.full((2048,), 2.0, device="cuda")
    b = torch.linspace(-1, 1, 2048, device="cuda")
    y, _, mean, rstd = rq().layernorm(x, g, b, stats=True)
    # sums of 2048 threes are whole numbers below 2^24: the mean is exact
    assert torch.equal(y, b.expand(5, -1)) and bool((mean == 3.0).all())
    assert bool(((rstd - 1e-5 ** -0.5).abs() <= 4 * U * 1e-5 ** -0.5).all())
    q, scale, _ = rq().layernorm_quant_int8(x, g)
    assert not q.any() and not scale.any()


@gpu
def test_nan_stays_in_its_row():
    d = make(9, 1500, torch.bfloat16, seed=3)
    clean = rq().layernorm(d["x"], d["gamma"], d["beta"])[0]
    d["x"][4, 77] = float("nan")
    d["x"][6, 3] = float("inf")
    y = rq().layernorm(d["x"], d["gamma"], d["beta"])[0]
    assert y[4].isnan().all() and y[6].isnan().all()
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[keep], clean[keep])


@gpu
@pytest.mark.parametrize("hidden", [1000, 1003, 4096, 20000])
def test_in_place(hidden):
    d = make(33, hidden, torch.bfloat16, seed=8, residual=True)
    want = rq().layernorm(d["x"], d["gamma"], d["beta"], residual=d["residual"])
    rq().layernorm(d["x"], d["gamma"], d["beta"], residual=d["residual"], residual_output=d["residual"],
                   output=d["x"])
    assert torch.equal(d["x"], want[0]) and torch.equal(d["residual"], want[1])


@gpu
@pytest.mark.parametrize("hidden", [61, 1032, 5121, 17001])
def test_guard_bytes(hidden):
    rows = 13
    d = make(rows, hidden, torch.bfloat16, seed=2, residual=True)
    y, y_raw = guarded(rows * hidden, torch.bfloat16)
    ro, ro_raw = guarded(rows * hidden, torch.bfloat16)
    rq().layernorm(d["x"], d["gamma"], d["beta"], residual=d["residual"],
                   residual_output=ro.view(rows, hidden), output=y.view(rows, hidden))
    q, q_raw = guarded(rows * hidden, torch.int8)
    sc, sc_raw = guarded(rows, torch.float32)
    rq().layernorm_quant_int8(d["x"], d["gamma"], output=q.view(rows, hidden), scale_output=sc)
    ds, ds_raw = guarded(rows * hidden, torch.bfloat16)
    dg, dg_raw = guarded(hidden, torch.float32)
    db, db_raw = guarded(hidden, torch.float32)
    need = rq().layernorm_backward_workspace(rows, hidden)
    ws, ws_raw = guarded(need, torch.uint8)
    mean = torch.zeros(rows, device="cuda")
    rq().layernorm_backward(d["x"], d["x"], d["gamma"], mean, mean + 1, grad_residual=d["residual"],
                            grad_input=ds.view(rows, hidden), grad_gamma=dg, grad_beta=db,
                            param_grad_dtype=torch.float32, workspace=ws)
    torch.cuda.synchronize()
    assert guards_intact((y_raw, ro_raw, q_raw, sc_raw, ds_raw, dg_raw, db_raw, ws_raw))


# ------------------------------------------------------------------------------- int8 rows

def check_int8(d, rms, offset=0.0, eps=1e-5):
    m = rq()
    kw = dict(residual=d["residual"], epsilon=eps, weight_offset=offset)
    if rms:
        q, scale, res = m.rmsnorm_quant_int8(d["x"], d["gamma"], **kw)
    else:
        q, scale, res = m.layernorm_quant_int8(d["x"], d["gamma"], d["beta"], **kw)
    s = d["x"]
    if d["residual"] is not None:
        s = (d["x"].double() + d["residual"].double()).to(s.dtype)
        assert torch.equal(res, s)
    y, _, _, err = formula(s, d["gamma"], None if rms else d["beta"], offset, eps, rms)
    exact = y.abs().amax(1) / 127
    off = err.amax(1) / 127 + 2 * U * exact
    assert ((scale.double() - exact).abs() <= off).all()
    step = torch.where(exact > 0, exact, 1.0)[:, None]
    slack = 0.5 + (err + 127 * off[:, None]) / step + 127 * 4 * U
    assert ((q.double() - y / step).abs() <= slack).all()
    assert int(q.min()) >= -127
    assert bool((q.abs().amax(1) == 127)[exact > 0].all())


@gpu
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", [1, 8, 63, 256, 400, 1000, 1024, 1026, 4096, 5121, 8192, 12000, 16384, 20000, 33333,
                                    32761, 32776, 65535, 65536])
def test_int8_rows(rms, dtype, hidden):
    check_int8(make(19, hidden, dtype, seed=hidden + 1, residual=hidden % 2 == 0), rms, offset=1.0)


@gpu
def test_int8_tiny_rows():
    # amax / 127 is below the smallest normal number whose reciprocal is finite
    x = torch.randn(6, 512, device="cuda")
    gamma = torch.full((512,), 1e-37, device="cuda")
    q, scale, _ = rq().rmsnorm_quant_int8(x, gamma)
    y = formula(x, gamma, None, 0.0, 1e-6, rms=True)[0]
    step = y.abs().amax(1, keepdim=True) / 127
    # y near 1e-37 .. 4e-37 is kept to 2^-149 absolute, 1.4e-45 / 1e-39 = 2e-6 of a step
    assert ((q.double() - y / step).abs() <= 0.5 + 1e-4).all()
    assert q.abs().amax(1).eq(127).all()


# ------------------------------------------------------------------------------- backward

def make_backward(rows, hidden, dtype, seed, residual):
    d = make(rows, hidden, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    d["dy"] = torch.randn((rows, hidden), generator=g, device="cuda").to(dtype)
    d["dres"] = torch.randn((rows, hidden), generator=g, device="cuda").to(dtype) if residual else None
    x = d["x"].double()
    d["mean"] = x.mean(1).float()
    d["rstd"] = (x.var(1, correction=0) + 1e-5).rsqrt().float()
    return d


def check_backward(d, offset=0.0, pdt=None):
    t = d["x"].dtype
    ds, dg, db = rq().layernorm_backward(d["dy"], d["x"], d["gamma"], d["mean"], d["rstd"],
                                         grad_residual=d["dres"], weight_offset=offset,
                                         param_grad_dtype=pdt)
    rows = d["x"].shape[0]
    dy, w = d["dy"].double(), d["gamma"].double() + offset
    rstd = d["rstd"].double()[:, None]
    xh = (d["x"].double() - d["mean"].double()[:, None]) * rstd
    g = dy * w
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    e = rstd * (g - mean(g) - xh * mean(g * xh))
    size = rstd * (g.abs() + mean(g.abs()) + 2 * xh.abs() * mean((g * xh).abs()))
    if d["dres"] is not None:
        e = e + d["dres"].double()
        size = size + d["dres"].double().abs()
    h = half_step(t)
    assert ((ds.double() - e).abs() <= h * e.abs() + K * U * size * (1 + h) + tiny(t)).all()
    pdt = pdt or t
    h = half_step(pdt)
    for got, terms in ((dg, dy * xh), (db, dy)):
        assert got.dtype == pdt
        want, slack = terms.sum(0), (rows + K) * U * terms.abs().sum(0)
        assert ((got.double() - want).abs() <= h * want.abs() + slack * (1 + h) + tiny(pdt)).all()
    assert rq().rmsq_device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", [1, 3, 8, 9, 64, 250, 256, 264, 500, 512, 1024, 1030, 2048, 2051,
                                    4096, 5121, 8192])
def test_backward_widths(dtype, hidden):
    check_backward(make_backward(333, hidden, dtype, hidden, residual=hidden % 2 == 0), offset=1.0)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", [8200, 8193, 16384, 22761, 40008, 65536])
def test_backward_clusters(dtype, hidden):
    check_backward(make_backward(45, hidden, dtype, hidden, residual=hidden % 2 == 0))


@gpu
@pytest.mark.parametrize("hidden", [8191, 8193, 8200, 16383, 16393, 16401, 32767, 32793, 65543, 65544])
def test_backward_around_each_cluster(hidden):
    # enough rows that every CTA has several
    check_backward(make_backward(600, hidden, torch.bfloat16, hidden, residual=False))


@gpu
@pytest.mark.parametrize("hidden", [131072, 131071])
def test_backward_widest(hidden):
    check_backward(make_backward(11, hidden, torch.bfloat16, 4, residual=True))


@gpu
@pytest.mark.parametrize("rows", [1, 2, 151, 153, 700, 20011])
@pytest.mark.parametrize("hidden", [40, 1024, 2056])
def test_backward_rows(rows, hidden):
    check_backward(make_backward(rows, hidden, torch.float16, rows, residual=rows % 2 == 1),
                   pdt=torch.float32)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", [1000, 1003, 4096, 8192])
@pytest.mark.parametrize("residual", [False, True])
def test_backward_many_rows(dtype, hidden, residual):
    # every slot of the ring is refilled several times
    check_backward(make_backward(5003, hidden, dtype, hidden, residual=residual))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hidden", [1000, 1003, 4096, 8192, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_many_rows(dtype, hidden, residual):
    check_forward(make(20011 if hidden < 8000 else 5003, hidden, dtype, hidden, residual=residual))


@gpu
def test_backward_in_place_and_repeatable():
    for hidden in (1000, 1003, 4096, 9001):
        d = make_backward(400, hidden, torch.bfloat16, 6, residual=True)
        args = (d["x"], d["gamma"], d["mean"], d["rstd"])
        first = rq().layernorm_backward(d["dy"], *args, grad_residual=d["dres"])
        again = rq().layernorm_backward(d["dy"], *args, grad_residual=d["dres"])
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        place = rq().layernorm_backward(d["dy"], *args, grad_residual=d["dres"], grad_input=d["dres"])
        assert all(torch.equal(a, b) for a, b in zip(first, place))


@gpu
def test_backward_against_differences():
    # <ds, v> + <dgamma, vg> + <dbeta, vb> against central differences of the formula in 64 bits
    rows, hidden, eps = 29, 515, 1e-5
    d = make_backward(rows, hidden, torch.float32, 12, residual=False)
    ds, dg, db = rq().layernorm_backward(d["dy"], d["x"], d["gamma"], d["mean"], d["rstd"])
    g = torch.Generator(device="cuda").manual_seed(99)
    v, vg, vb = (torch.randn(s, generator=g, device="cuda", dtype=torch.float64)
                 for s in ((rows, hidden), (hidden,), (hidden,)))
    x, gamma, beta, dy = (d[k].double() for k in ("x", "gamma", "beta", "dy"))
    step = 1e-5

    def loss(a):
        return (formula(x + a * v, gamma + a * vg, beta + a * vb, 0.0, eps)[0] * dy).sum()

    slope = (loss(step) - loss(-step)) / (2 * step)
    parts = torch.cat([(ds.double() * v).flatten(), dg.double() * vg, db.double() * vb])
    # differences: step^2 times a third derivative and 2^-53 / step; gradients: K u of each term
    assert abs(float(slope - parts.sum())) <= 2 * K * U * float(parts.abs().sum()) + 1e-6 * float(parts.abs().sum())


@gpu
def test_backward_of_no_rows_writes_zeros():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    stat = torch.empty(0, device="cuda")
    gamma = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    dg = torch.full((256,), 7.0, dtype=torch.bfloat16, device="cuda")
    ds, dg, db = rq().layernorm_backward(x, x, gamma, stat, stat, grad_gamma=dg)
    assert ds.shape == (0, 256) and not dg.any() and not db.any()


@gpu
def test_forward_of_no_rows_launches_nothing():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    before = rq().rmsq_launch_count()
    y, _, mean, _ = rq().layernorm(x, torch.ones(256, dtype=torch.bfloat16, device="cuda"), stats=True)
    assert y.shape == (0, 256) and mean.shape == (0,) and rq().rmsq_launch_count() == before


# ------------------------------------------------------------------------------- a training step

@gpu
def test_training_chain_on_another_stream_and_in_a_graph():
    """Two layers of norm on one residual stream, forward and backward, as a training step runs
    them: eagerly on a side stream, and captured with shared buffers and replayed on new inputs."""
    m = rq()
    rows, hidden = 600, 2048
    d = make(rows, hidden, torch.bfloat16, seed=1, residual=True)
    e = make(rows, hidden, torch.bfloat16, seed=2)

    def step(stream=None):
        y1, s1, m1, r1 = m.layernorm(d["x"], d["gamma"], d["beta"], residual=d["residual"], stats=True,
                                     stream=stream)
        y2, s2, m2, r2 = m.layernorm(y1, e["gamma"], e["beta"], residual=s1, stats=True, stream=stream)
        b2 = m.layernorm_backward(e["x"], s2, e["gamma"], m2, r2, stream=stream)
        b1 = m.layernorm_backward(b2[0], s1, d["gamma"], m1, r1, grad_residual=b2[0], stream=stream)
        return y2, *b2, *b1

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (11, 12):
        fresh = make(rows, hidden, torch.bfloat16, seed=seed, residual=True)
        d["x"].copy_(fresh["x"])
        d["residual"].copy_(fresh["residual"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step(), out))


# ------------------------------------------------------------------------------- refusals (CPU)

def test_refusals_without_a_gpu():
    lib = rq().lib()
    A, nan = 1 << 20, float("nan")   # fake 16-byte aligned addresses: never dereferenced here

    def ln(x=A, r=None, ro=None, g=A, b=A, rows=4, h=60, dt=0, eps=1e-5, off=0.0, out=A, mean=A, rstd=A):
        return lib.layernorm(x, r, ro, g, b, rows, h, dt, eps, off, out, mean, rstd, None)

    assert ln(x=None) == 1 and ln(out=None) == 1 and ln(r=A) == 1 and ln(ro=A) == 1
    assert ln(h=0) == 2 and ln(h=131073) == 2 and ln(h=65537, dt=2) == 2 and ln(rows=-1) == 2
    assert ln(rows=1 << 40) == 2
    assert ln(x=A + 2) == 3 and ln(b=A + 8) == 3 and ln(mean=A + 4) == 3
    assert ln(dt=3) == 4 and ln(eps=-1.0) == 6 and ln(eps=nan) == 6 and ln(off=nan) == 6
    assert ln(rows=0, x=None) == 0

    def qt(fn, *beta, x=A, h=60, out=A, sc=A, rows=4):
        return getattr(lib, fn)(x, None, None, A, *beta, rows, h, 0, 1e-5, 0.0, out, sc, None)

    for fn, beta in (("layernorm_quant_int8", (A,)), ("rmsnorm_quant_int8", ())):
        assert qt(fn, *beta, sc=None) == 1 and qt(fn, *beta, sc=A + 4) == 3 and qt(fn, *beta, h=0) == 2
        assert qt(fn, *beta, rows=0, x=None) == 0

    def bw(dy=A, dres=None, s=A, g=A, rows=4, h=60, dt=0, dg=A, db=A, pdt=0, ws=A, nb=1 << 20, off=0.0):
        return lib.layernorm_backward(dy, dres, s, g, A, A, rows, h, dt, off, A, dg, db, pdt, ws, nb, None)

    assert bw(dy=None) == 1 and bw(dg=None) == 1 and bw(ws=None) == 1
    assert bw(h=0) == 2 and bw(rows=-1) == 2 and bw(nb=4 * 2 * 60 * 4 - 1) == 2
    assert bw(dres=A + 2) == 3 and bw(ws=A + 8) == 3 and bw(dt=7) == 4 and bw(pdt=1) == 4 and bw(off=nan) == 6
    assert lib.layernorm_backward_workspace(4, 60) == 4 * 2 * 60 * 4
    assert lib.layernorm_backward_workspace(10 ** 6, 60) == 152 * 2 * 60 * 4
    assert lib.layernorm_backward_workspace(0, 60) == 0


@gpu
def test_python_refusals():
    m = rq()
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(4, device="cuda")
    bad = [lambda: m.layernorm(x.t(), g[:4]), lambda: m.layernorm(x, g[:63]),
           lambda: m.layernorm(x, g.float()), lambda: m.layernorm(x, g, g[:63]),
           lambda: m.layernorm(x, g, output=x[:2]), lambda: m.layernorm(x, g, output=x.float()),
           lambda: m.layernorm(x, g, residual=x, residual_output=x.float()),
           lambda: m.layernorm_quant_int8(x, g, output=x), lambda: m.rmsnorm_quant_int8(x, g, scale_output=st[:3]),
           lambda: m.layernorm_backward(x[:2], x, g, st, st), lambda: m.layernorm_backward(x, x, g, st[:2], st),
           lambda: m.layernorm_backward(x, x, g, st.double(), st),
           lambda: m.layernorm_backward(x, x, g, st, st, grad_residual=x.half())]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        m.layernorm_backward(x, x, g, st, st, param_grad_dtype=torch.float16)
    with pytest.raises(m.RmsqError):
        m.layernorm_backward(x, x, g, st, st, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(m.RmsqError):
        m.layernorm(x.reshape(-1)[1:129].view(2, 64), g)
