"""rmsnorm_rope and rmsnorm_rope_backward against their formulas in 64 bits (the gradient by automatic differentiation of
the forward formula there, and against differences of the kernel itself).

Tolerances, u = 2^-24, h half a step of the output's type. The sum of squares of at most 512 positive terms is added in
chains of 16 and 5 (off by 21 u), the mean, epsilon, root and reciprocal add 4 u: rstd is off by (21 + 2) / 2 + 2 < 14 u.
Forward: with three products and the rotation's two roundings an element is off by 20 u of |z_a c| + |z_b s|. Backward: u_i
carries the rotation (2 u) and gamma (2 u), xhat 15 u, their dot product 21 u more; dx = rstd (u - xhat dot) is
off by 60 u of rstd (|u| + |xhat| <|u xhat|>). The gammas' gradients add n terms of 20 u each in chains of at most n:
(20 + n) u of the sum of magnitudes, n = tokens * heads. A rounded gradient adds h."""
import pytest
import torch

from gpu_common import rq

U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
gpu = pytest.mark.gpu


def table(places, half, base=10000.0):
    angle = torch.arange(places, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
        base, -torch.arange(half, device="cuda", dtype=torch.float64) / half)
    return angle.cos().float(), angle.sin().float()


def make(tokens, heads, kv, dim, dtype, seed, rotated=None, sections=None, inter=False, layout="plain", bits=64, offset=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rotated = dim if rotated is None else rotated
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731

    def pair():
        if layout == "packed":
            both = (r(tokens, (heads + 2 * kv) * dim) + 0.1).to(dtype)
            return both[:, :heads * dim].unflatten(1, (heads, dim)), both[:, heads * dim:(heads + kv) * dim].unflatten(1, (kv, dim))
        if layout == "heads_first":
            return tuple(r(n, tokens, dim).to(dtype).transpose(0, 1) for n in (heads, kv))
        if layout == "odd":           # rows that start anywhere
            return tuple(r(tokens, n, dim + 3).to(dtype)[:, :, 1:dim + 1] for n in (heads, kv))
        return tuple(r(tokens, n, dim).to(dtype) for n in (heads, kv))

    q, k = pair()
    dq, dk = pair()
    cos, sin = table(500, rotated // 2)
    shape = (tokens,) if sections is None else (len(sections), tokens)
    pos = torch.randint(0, 500, shape, generator=g, device="cuda", dtype=torch.int64 if bits == 64 else torch.int32)
    gq, gk = ((r(dim) * 0.2 + 1 - offset).to(dtype) for _ in range(2))
    return dict(q=q, k=k, dq=dq, dk=dk, gq=gq, gk=gk, cos=cos, sin=sin, pos=pos, sections=sections, inter=inter, offset=offset)


def opts(d):
    return dict(sections=d["sections"], interleaved=d["inter"], weight_offset=d["offset"])


def forward(d, **kw):
    return rq().rmsnorm_rope(d["q"], d["k"], d["gq"], d["gk"], d["cos"], d["sin"], d["pos"], **opts(d), **kw)


def backward(d, **kw):
    return rq().rmsnorm_rope_backward(d["dq"], d["dk"], d["q"], d["k"], d["gq"], d["gk"], d["cos"], d["sin"], d["pos"],
                                      **opts(d), **kw)


def angles(d):
    half = d["cos"].shape[1]
    if d["sections"] is None:
        at = d["pos"][:, None].expand(-1, half)
    else:
        axis = torch.repeat_interleave(torch.arange(len(d["sections"]), device="cuda"),
                                       torch.tensor(d["sections"], device="cuda"))
        at = d["pos"].t()[:, axis]
    i = torch.arange(half, device="cuda")
    return d["cos"].double()[at.long(), i][:, None], d["sin"].double()[at.long(), i][:, None]


def turned(z, c, s, inter):
    half = c.shape[-1]
    head, rest = z[..., :2 * half], z[..., 2 * half:]
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, rest), -1)


def formula(x, gamma, c, s, d, eps=1e-6):
    z = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * (gamma + d["offset"])
    return turned(z, c, s, d["inter"]), z


def check_forward(d, **kw):
    out = forward(d, **kw)
    c, s = angles(d)
    for x, g, y in ((d["q"], d["gq"], out[0]), (d["k"], d["gk"], out[1])):
        e, z = formula(x.double(), g.double(), c, s, d)
        size = turned(z.abs(), c.abs(), -s.abs(), d["inter"])          # |z_a c| + |z_b s| in the first halves
        size = torch.maximum(size, turned(z.abs(), c.abs(), s.abs(), d["inter"]))
        h, low = torch.finfo(x.dtype).eps / 2, 2.0 ** -25 if x.dtype == torch.float16 else 0.0
        off = (y.double() - e).abs()
        assert y.shape == x.shape and y.dtype == x.dtype
        assert bool((off <= h * e.abs() + 20 * U * size * (1 + h) + low).all()), float(off.max())
    return out


def check_backward(d, **kw):
    got = backward(d, **kw)
    c, s = angles(d)
    for i, (x, g, dy) in enumerate(((d["q"], d["gq"], d["dq"]), (d["k"], d["gk"], d["dk"]))):
        xd, gd = x.double().requires_grad_(), g.double().requires_grad_()
        ex, eg = torch.autograd.grad(formula(xd, gd, c, s, d)[0], (xd, gd), dy.double())
        with torch.no_grad():
            back = turned(dy.double(), c, -s, d["inter"])
            wide = torch.maximum(turned(dy.double().abs(), c.abs(), s.abs(), d["inter"]),
                                 turned(dy.double().abs(), c.abs(), -s.abs(), d["inter"]))
            r = torch.rsqrt(xd.square().mean(-1, keepdim=True) + 1e-6)
            u, xhat = (wide * (gd + d["offset"])).abs(), (xd * r).abs()
            size = r * (u + xhat * (u * xhat).mean(-1, keepdim=True))
            gsize = (wide * xhat).sum((0, 1))
            h, low = torch.finfo(x.dtype).eps / 2, 2.0 ** -25 if x.dtype == torch.float16 else 0.0
            off = (got[i].double() - ex).abs()
            assert bool((off <= h * ex.abs() + 60 * U * size * (1 + h) + low).all()), float(off.max())
            n = x.shape[0] * x.shape[1]
            hg = torch.finfo(got[2 + i].dtype).eps / 2
            off = (got[2 + i].double() - eg).abs()
            assert bool((off <= hg * eg.abs() + (20 + n) * U * gsize * (1 + hg) + low).all()), float(off.max())
            del back
    assert rq().rmsq_device_status() == 0
    return got


def both(d):
    check_forward(d)
    check_backward(d)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim", [2, 4, 6, 10, 16, 32, 40, 64, 72, 80, 96, 112, 120, 128, 130, 160, 192, 250, 256, 320, 384, 510, 512])
def test_head_sizes(dtype, inter, dim):
    both(make(19, 6, 2, dim, dtype, dim, inter=inter))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rotated", [(128, 64), (128, 2), (128, 126), (80, 32), (80, 60), (192, 64), (96, 90), (256, 64), (12, 4)])
def test_part_of_a_head(dtype, inter, dim, rotated):
    both(make(11, 5, 3, dim, dtype, rotated, rotated=rotated, inter=inter, offset=1.0))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sections", [(64,), (16, 24, 24), (1, 63), (0, 40, 24), (10, 20, 30, 4), (24, 20, 20, 0)])
def test_axes(dtype, inter, sections):
    both(make(23, 4, 2, 128, dtype, 3, sections=sections, inter=inter, bits=32 if len(sections) == 3 else 64))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [1, 2, 7, 64, 300])
@pytest.mark.parametrize("heads,kv", [(1, 1), (32, 8), (7, 7), (33, 3), (129, 1)])
def test_tokens_and_heads(dtype, tokens, heads, kv):
    both(make(tokens, heads, kv, 64, dtype, tokens + heads, bits=32 if tokens % 2 else 64))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("layout", ["packed", "heads_first", "odd"])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_layouts(dtype, inter, layout, dim):
    d = make(37, 8, 2, dim, dtype, 5, inter=inter, layout=layout)
    both(d)
    if layout == "packed":         # outputs inside another tensor, which stays as it is elsewhere
        whole = torch.full((37, 12, dim), 3.0, dtype=dtype, device="cuda")
        y = check_forward(d, query_output=whole[:, 1:9], key_output=whole[:, 9:11])
        assert y[0].data_ptr() == whole[:, 1:9].data_ptr()
        assert bool((whole[:, 0] == 3).all()) and bool((whole[:, 11] == 3).all())


@gpu
@pytest.mark.parametrize("inter", [False, True])
def test_slices_of_tables_gammas_and_broadcast_inputs(inter):
    d = make(9, 4, 2, 80, torch.bfloat16, 1, rotated=30, inter=inter)
    want = check_forward(d)
    grads = check_backward(d)
    e = dict(d)
    for name in ("cos", "sin"):
        e[name] = torch.cat((d[name][:1], d[name]))[1:]                        # rows of 60 bytes
    for name in ("gq", "gk"):
        e[name] = torch.cat((d[name][:1], d[name]))[1:]
    assert all(torch.equal(a, b) for a, b in zip(check_forward(e), want))
    assert all(torch.equal(a, b) for a, b in zip(check_backward(e)[:2], grads[:2]))
    e = dict(d, q=d["q"][:1].expand(9, 4, 80), dq=d["dq"][:, :1].expand(9, 4, 80), k=d["k"][:, 1:].expand(9, 2, 80))
    both(e)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 33, 1000])
@pytest.mark.parametrize("heads,kv,dim,sections", [(12, 2, 80, (10, 10, 20)), (28, 4, 128, None), (9, 3, 64, None), (1, 1, 256, (64, 64))])
def test_turns_of_two_tokens(dtype, tokens, heads, kv, dim, sections):
    """Heads in an odd number of the groups that a warp takes at a time: groups of two tokens, with places of their own, lie together."""
    both(make(tokens, heads, kv, dim, dtype, seed=tokens + dim, sections=sections, inter=sections is not None, layout="packed"))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
def test_in_place(dtype, inter):
    d = make(50, 8, 2, 96, dtype, 2, inter=inter, layout="packed")
    want, grads = forward(d), backward(d)
    e = {n: v.clone() if torch.is_tensor(v) else v for n, v in d.items()}
    got = forward(e, query_output=e["q"], key_output=e["k"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    e = {n: v.clone() if torch.is_tensor(v) else v for n, v in d.items()}
    got = backward(e, query_grad=e["dq"], key_grad=e["dk"])
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    e = {n: v.clone() if torch.is_tensor(v) else v for n, v in d.items()}
    got = backward(e, query_grad=e["q"], key_grad=e["k"])
    assert all(torch.equal(a, b) for a, b in zip(got, grads))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sections", [None, (8, 8, 8)])
def test_places_outside_the_table(dtype, inter, sections):
    d = make(12, 3, 2, 64, dtype, 4, rotated=48, inter=inter, sections=sections)
    want = forward(d)
    bad = {2: -1, 5: 500, 9: 2 ** 40, 10: -2 ** 62}
    for t, at in bad.items():
        d["pos"][..., t] = at
    rows = torch.tensor(list(bad), device="cuda")
    keep = torch.ones(12, dtype=torch.bool, device="cuda")
    keep[rows] = False
    for y, w in zip(forward(d), want):
        assert torch.isnan(y[rows][..., :48]).all()
        assert torch.equal(y[rows][..., 48:], w[rows][..., 48:]) and torch.equal(y[keep], w[keep])
    g = backward(d)
    assert torch.isnan(g[0][rows]).all() and torch.isfinite(g[0][keep]).all() and torch.isnan(g[2][:48]).all()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
def test_a_head_that_is_not_finite(dtype, inter):
    d = make(9, 6, 3, 80, dtype, 6, rotated=40, inter=inter)
    want = forward(d)
    d["q"][3, 2, 7], d["k"][8, 0, 70] = float("nan"), float("inf")
    q, k = forward(d)
    assert torch.isnan(q[3, 2]).all() and torch.isnan(k[8, 0, 70])
    assert bool((k[8, 0, 40:70] == 0).all())
    for y, w, t, h in ((q, want[0], 3, 2), (k, want[1], 8, 0)):
        y[t, h] = w[t, h]
        assert torch.equal(y, w)
    zero = make(3, 2, 1, 64, dtype, 6, inter=inter)
    zero["q"].zero_()
    y, g = forward(zero), backward(zero)
    assert bool((y[0] == 0).all()) and torch.isfinite(g[0]).all()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_training_batch(dtype):
    both(make(700, 16, 4, 128, dtype, 8, layout="packed"))
    check_backward(make(700, 4, 4, 80, dtype, 8), param_grad_dtype=torch.float32)


@gpu
@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(inter):
    """Central differences of the kernel's own forward pass in 32 bits along random directions: with a step of 2^-6 the
    third derivative's part is about 4e-5 of the norms and the outputs' rounding 2^-24 * 2^6 = 4e-6, so 1e-3 of the
    product of the norms is wide of both."""
    d = make(6, 3, 2, 64, torch.float32, 11, inter=inter)
    dq, dk, dgq, dgk = check_backward(d)
    loss = lambda e: sum((y.double() * w.double()).sum() for y, w in zip(forward(e), (d["dq"], d["dk"])))  # noqa: E731
    step = 2.0 ** -6
    for name, grad in (("q", dq), ("k", dk), ("gq", dgq), ("gk", dgk)):
        v = torch.randn(d[name].shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
        diff = (loss(dict(d, **{name: d[name] + step * v})) - loss(dict(d, **{name: d[name] - step * v}))) / (2 * step)
        along = (grad.double() * v.double()).sum()
        assert abs(float(diff - along)) <= 1e-3 * float(grad.double().norm() * v.double().norm())


@gpu
def test_past_32_bits():
    # queries of over 2^31 elements, in a packed projection's output of over 2^32
    t, h, dim = 300000, 64, 128
    both_ = torch.zeros((t, (h + 48) * dim), dtype=torch.bfloat16, device="cuda")
    d = make(3, h, 16, dim, torch.bfloat16, 3)
    q, k = both_[:, :h * dim].unflatten(1, (h, dim)), both_[:, h * dim:(h + 16) * dim].unflatten(1, (16, dim))
    q[-3:], k[-3:] = d["q"], d["k"]
    pos = torch.zeros(t, dtype=torch.int64, device="cuda")
    pos[-3:] = d["pos"]
    want = forward(d)
    got = rq().rmsnorm_rope(q, k, d["gq"], d["gk"], d["cos"], d["sin"], pos, query_output=q, key_output=k)
    assert torch.equal(got[0][-3:], want[0]) and torch.equal(got[1][-3:], want[1])
    assert bool((both_[-3:, (h + 16) * dim:] == 0).all())
    # in the backward pass, with gradients that are zero but for the same tokens
    q[-3:], k[-3:] = d["q"], d["k"]
    dq, dk = torch.zeros_like(q), torch.zeros_like(k)
    dq[-3:], dk[-3:] = d["dq"], d["dk"]
    want = backward(d, param_grad_dtype=torch.float32)
    got = rq().rmsnorm_rope_backward(dq, dk, q, k, d["gq"], d["gk"], d["cos"], d["sin"], pos, param_grad_dtype=torch.float32)
    assert torch.equal(got[0][-3:], want[0]) and torch.equal(got[1][-3:], want[1])
    assert bool((got[0][:-3] == 0).all())
    for a, b in zip(got[2:], want[2:]):
        assert bool(((a - b).abs() <= 4 * 192 * U * b.abs().max()).all())      # the same terms in another order


@gpu
def test_leading_dimensions():
    d = make(24, 4, 2, 64, torch.bfloat16, 4)
    want, grads = forward(d), backward(d)
    e = dict(d, **{n: d[n].view(2, 12, *d[n].shape[1:]) for n in ("q", "k", "dq", "dk")}, pos=d["pos"].view(2, 12))
    got = forward(e)
    assert got[0].shape == (2, 12, 4, 64) and all(torch.equal(a.flatten(0, 1), b) for a, b in zip(got, want))
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(backward(e), grads))


@gpu
@pytest.mark.parametrize("inter", [False, True])
def test_streams_graph_and_equal_bits(inter):
    d = make(400, 16, 4, 128, torch.bfloat16, 9, inter=inter)
    other = dict(d, q=d["q"] * 2 + 1, dk=d["dk"] * 2)
    run = lambda e, stream=None: (*forward(e, stream=stream), *backward(e, stream=stream))  # noqa: E731
    want, want2 = run(d), run(other)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a, b = run(d, one), run(other, two)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, want)) and all(torch.equal(x, y) for x, y in zip(b, want2))
    buf = {n: v.clone() if torch.is_tensor(v) else v for n, v in d.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(buf)
    for src, w in ((other, want2), (d, want)):
        buf["q"].copy_(src["q"])
        buf["dk"].copy_(src["dk"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, w))


@gpu
def test_empty_calls():
    d = make(0, 4, 2, 64, torch.bfloat16, 1)
    before = rq().rmsq_launch_count()
    q, k = forward(d)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64) and rq().rmsq_launch_count() == before
    fill = torch.full((64,), 7.0, dtype=torch.bfloat16, device="cuda")
    g = backward(d, query_gamma_grad=fill, key_gamma_grad=fill.clone())
    assert bool((g[2] == 0).all()) and bool((g[3] == 0).all())


def test_refusals_without_a_gpu():
    import rmsnorm_precision_activation_gb300 as m
    lib, A = rq().lib(), 1 << 20      # fake addresses: never dereferenced here

    def call(q=(A, 512, 64, 8), k=(A, 128, 64, 2), gq=A, gk=A, rot=(A, A, A, 100, 64, 64, 0, 1), sections=(), tokens=4, dim=64,
             dt=0, eps=1e-6, off=0.0, oq=(A, 512, 64, 8), ok=(A, 128, 64, 2), back=None):
        parts = tuple(sections) + (0,) * (4 - len(sections))
        r = None if rot is None else m.ROTATION.pack(*(p or 0 for p in rot[:3]), *rot[3:], *parts)
        h = lambda t: None if t is None else m.HEADS.pack(t[0] or 0, *t[1:])  # noqa: E731
        if back is None:
            return lib.rmsnorm_rope(h(q), h(k), gq, gk, r, tokens, dim, dt, eps, off, h(oq), h(ok), None)
        b = dict(dq=(A, 512, 64, 8), dk=(A, 128, 64, 2), pq=A, pk=A, pdt=dt, ws=A, size=1 << 30)
        b.update(back)
        return lib.rmsnorm_rope_backward(h(b["dq"]), h(b["dk"]), h(q), h(k), gq, gk, r, tokens, dim, dt, eps, off, h(oq), h(ok),
                                         b["pq"], b["pk"], b["pdt"], b["ws"], b["size"], None)

    for back in (None, {}):
        f = lambda **kw: call(back=back, **kw)  # noqa: E731
        assert all(f(**{x: None}) == 1 for x in ("q", "k", "gq", "gk", "rot", "oq", "ok"))
        assert f(q=(None, 512, 64, 8)) == 1 and f(rot=(A, None, A, 100, 64, 64, 0, 1)) == 1 and f(rot=(A, A, None, 100, 64, 64, 0, 1)) == 1
        assert all(f(dim=n) == 2 for n in (0, 1, 63, 514)) and f(tokens=-1) == 2 and f(tokens=2 ** 27) == 2
        assert f(q=(A, 512, 64, 0), oq=(A, 512, 64, 0)) == 2 and f(q=(A, -1, 64, 8)) == 2 and f(q=(A, 512, 2 ** 31, 8)) == 2
        assert f(oq=(A, 512, 64, 7)) == 2                                               # heads differ
        assert f(oq=(A, 512, 32, 8)) == 2 and f(oq=(A, 256, 64, 8)) == 2 and f(ok=(A, 0, 64, 2)) == 2   # outputs that overlap
        assert f(q=(A + 1, 512, 64, 8)) == 3 and f(rot=(A, A, A + 4, 100, 64, 64, 0, 1)) == 3 and f(gq=A + 1) == 3
        assert f(rot=(A, A, A, 100, 16, 64, 0, 1)) == 4 and f(dt=3) == 4
        for rotated in (0, 63, 66, -2):
            assert f(rot=(A, A, A, 100, 64, rotated, 0, 1)) == 2
        assert f(rot=(A, A, A, 0, 64, 64, 0, 1)) == 2 and f(rot=(A, A, A, 100, 64, 64, 0, 5)) == 2
        assert f(rot=(A, A, A, 100, 64, 64, 0, 3), sections=(10, 10, 11)) == 2
        assert f(rot=(A, A, A, 100, 64, 64, 0, 3), sections=(-1, 16, 17)) == 2
        assert f(eps=float("nan")) == 6 and f(eps=-1.0) == 6 and f(off=float("inf")) == 6
    assert call(tokens=0) == 0
    assert call(back=dict(pq=None)) == 1 and call(back=dict(ws=None)) == 1 and call(back=dict(dq=None)) == 1
    assert call(back=dict(size=lib.rmsnorm_rope_backward_workspace(4, 64) - 1)) == 2 and call(back=dict(ws=A + 4)) == 3
    assert call(back=dict(pdt=1)) == 4 and call(back=dict(dk=(A, 128, 64, 3))) == 2
    assert lib.rmsnorm_rope_backward_workspace(0, 64) == 0 and lib.rmsnorm_rope_backward_workspace(5, 1024) == 0


@gpu
def test_python_refusals():
    d, q = make(4, 4, 2, 64, torch.bfloat16, 0), rq()
    e = lambda **kw: lambda: forward(dict(d, **kw))  # noqa: E731
    bad = [e(k=d["k"][:3]), e(k=d["k"][:, :, :32]), e(k=d["k"].half()), e(q=d["q"].transpose(1, 2)), e(gq=d["gq"][:32]),
           e(gk=d["gk"].float()), e(cos=d["cos"][:, :16]), e(sin=d["sin"].double()), e(pos=d["pos"][:3]), e(sections=(16, 15)),
           e(sections=(16, 16)), e(pos=d["pos"].cpu()), e(q=d["q"].cpu()),
           lambda: forward(d, query_output=torch.empty(4, 4, 32, dtype=torch.bfloat16, device="cuda")),
           lambda: backward(d, query_gamma_grad=torch.empty(64, device="cuda")),
           lambda: forward(dict(d, q=d["q"].view(2, 2, 4, 64).transpose(0, 1), k=d["k"].view(2, 2, 2, 64), pos=d["pos"].view(2, 2)))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print(i)
    for call in (e(pos=d["pos"].float()), lambda: backward(d, param_grad_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(q.RmsqError):
        forward(d, query_output=torch.empty(4, 1, 64, dtype=torch.bfloat16, device="cuda").expand(4, 4, 64))
    with pytest.raises(q.RmsqError):
        backward(d, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
