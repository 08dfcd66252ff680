"""The heads' norm with rotation where a warp takes many turns: ring slots and angle slots taken again, the stride from turn to
turn, and the gammas' gradients over all of them, in both kinds of kernel. (A turn is two groups of heads; where
the groups of queries and of keys are both even in number and vectors hold 4 elements or more, no turn has rows of two tokens,
and kernels of their own serve that.)

Tolerances, u = 2^-24: outputs and their gradients as in test_rmsnorm_rope.py. A term g xhat of a gamma's gradient is off by 20 u
of its magnitude. They are added by a lane over its two rows of every turn, then over the warp's groups of rows (5 steps at
most), the CTA's 6 warps, then the CTAs' sums by 32 warps and those 32 sums: the gradient is off by
(20 + 2 turns + 5 + 6 + CTAs / 32 + 32) u of the sum of magnitudes, and a thousandth of that for products of errors."""
import math

import pytest
import torch

from gpu_common import rq
from test_rmsnorm_rope import DTYPES, U, angles, backward, check_forward, forward, make, turned

gpu = pytest.mark.gpu


def plan(tokens, heads, kv, dim, dtype, inter, back, rotated=None):
    """(whether no turn has two tokens, turns of a warp of the queries' and of the keys' at most, at least, CTAs of each), for tensors
    whose rows start on 16-byte boundaries."""
    half = (rotated or dim) // 2
    vec = 16 // dtype.itemsize
    fits = lambda v: dim % v == 0 and 2 * half % v == 0 if inter else half % v == 0 and (dim // 2 - half) % v == 0  # noqa: E731
    while vec > 1 and not fits(vec):
        vec //= 2
    step = max(vec // 2, 1) if inter else vec
    units = -(-(dim // 2 // step) // (8 // step))
    lanes = 1
    while lanes < units:
        lanes *= 2
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    warps, most = (6, min(2 * sms, 304)) if back else (4, 4 * sms)
    groups = [-(-h // (32 // lanes)) for h in (heads, kv)]
    turns = [-(-tokens * n // 2) for n in groups]
    ctas = [-(-t // warps) for t in turns]
    if sum(ctas) > most:
        q = min(max((most * turns[0] + sum(turns) // 2) // sum(turns), 1), most - 1)
        q = max(min(q, ctas[0]), most - ctas[1])
        ctas = [q, most - q]
    return (vec >= 4 and groups[0] % 2 == 0 and groups[1] % 2 == 0, [-(-t // (c * warps)) for t, c in zip(turns, ctas)],
            [t // (c * warps) for t, c in zip(turns, ctas)], ctas)


def check_backward(d, turns, ctas, **kw):
    """As in test_rmsnorm_rope.py, but with the gammas' gradients in 32 bits held to the sums that the kernels form."""
    got = backward(d, param_grad_dtype=torch.float32, **kw)
    c, s = angles(d)
    for i, (x, g, dy) in enumerate(((d["q"], d["gq"], d["dq"]), (d["k"], d["gk"], d["dk"]))):
        xd, gd, dyd = x.double(), g.double() + d["offset"], dy.double()
        r = torch.rsqrt(xd.square().mean(-1, keepdim=True) + 1e-6)
        xhat, back = xd * r, turned(dyd, c, -s, d["inter"])
        wide = torch.maximum(turned(dyd.abs(), c.abs(), s.abs(), d["inter"]), turned(dyd.abs(), c.abs(), -s.abs(), d["inter"]))
        u = back * gd
        ex = r * (u - xhat * (u * xhat).mean(-1, keepdim=True))
        uw, xa = (wide * gd).abs(), xhat.abs()
        size = r * (uw + xa * (uw * xa).mean(-1, keepdim=True))
        h, low = torch.finfo(x.dtype).eps / 2, 2.0 ** -25 if x.dtype == torch.float16 else 0.0
        off = (got[i].double() - ex).abs()
        assert bool((off <= h * ex.abs() + 60 * U * size * (1 + h) + low).all()), float(off.max())
        chain = 20 + 2 * turns[i] + 5 + 6 + math.ceil(ctas[i] / 32) + 32
        most = chain * U * 1.001 * (wide * xa).sum((0, 1)) + U * (back * xhat).sum((0, 1)).abs()
        off = (got[2 + i].double() - (back * xhat).sum((0, 1))).abs()
        assert got[2 + i].dtype == torch.float32 and bool((off <= most).all()), (float((off / most).max()), chain)
    assert rq().rmsq_device_status() == 0
    return got


# (tokens, heads, key heads, elements, rotated, whether no turn has two tokens)
SHAPES = [(3001, 32, 8, 128, 128, True), (4801, 64, 16, 64, 64, True), (4001, 8, 4, 256, 256, True), (4803, 16, 8, 96, 96, True),
          (3001, 8, 8, 192, 64, True), (5001, 16, 8, 80, 32, True), (1501, 12, 4, 512, 512, True), (3001, 28, 4, 128, 128, False),
          (5001, 12, 2, 80, 32, False), (7001, 9, 3, 64, 64, False)]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("layout", ["plain", "packed"])
@pytest.mark.parametrize("tokens,heads,kv,dim,rotated,whole", SHAPES)
def test_many_turns(dtype, inter, layout, tokens, heads, kv, dim, rotated, whole):
    for back in (False, True):
        one, turns, least, ctas = plan(tokens, heads, kv, dim, dtype, inter, back, rotated)
        assert one == whole and min(least) >= 4
    d = make(tokens, heads, kv, dim, dtype, heads + dim, rotated=rotated, inter=inter, layout=layout)
    check_forward(d)
    check_backward(d, turns, ctas)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads,kv,dim", [(32, 8, 128), (64, 16, 64), (28, 4, 128)])
def test_many_turns_in_place(dtype, inter, heads, kv, dim):
    d = make(3001, heads, kv, dim, dtype, 5, inter=inter, layout="packed")
    want, grads = forward(d), backward(d)

    def joined(a, b):            # both in one tensor, as they come from a projection
        whole = torch.cat((d[a].flatten(1), d[b].flatten(1)), 1)
        return {a: whole[:, :heads * dim].unflatten(1, (heads, dim)), b: whole[:, heads * dim:].unflatten(1, (kv, dim))}

    e = dict(d, **joined("q", "k"))
    assert all(torch.equal(a, b) for a, b in zip(forward(e, query_output=e["q"], key_output=e["k"]), want))
    e = dict(d, **joined("dq", "dk"))
    assert all(torch.equal(a, b) for a, b in zip(backward(e, query_grad=e["dq"], key_grad=e["dk"]), grads))
    e = dict(d, **joined("q", "k"))
    assert all(torch.equal(a, b) for a, b in zip(backward(e, query_grad=e["q"], key_grad=e["k"]), grads))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads,kv,dim", [(32, 8, 128), (64, 16, 64), (28, 4, 128), (12, 2, 80), (1, 1, 256)])
def test_every_row_counts_once_in_the_gammas_gradients(dtype, inter, heads, kv, dim):
    """Elements of 1 and -1, epsilon 0 and no rotation: xhat is x but for a mean of squares and a reciprocal root of 1 (off by 6 u at
    most), so a gradient is a sum of whole numbers, and one row's left out or added twice is off by 1 at least. One row in 16 has
    a gradient, so that all rounding together stays below 1 / 4."""
    tokens = 9001 if heads == 1 else 4801 if dim < 128 else 3001
    _, turns, _, ctas = plan(tokens, heads, kv, dim, dtype, inter, True)
    g = torch.Generator(device="cuda").manual_seed(heads)
    sign = lambda n: (2.0 * torch.randint(0, 2, (tokens, n, dim), generator=g, device="cuda") - 1).to(dtype)  # noqa: E731
    some = lambda n: (torch.rand((tokens, n, 1), generator=g, device="cuda") < 1 / 16).to(dtype)  # noqa: E731
    q, k = sign(heads), sign(kv)
    dq, dk = sign(heads) * some(heads), sign(kv) * some(kv)
    one, none = torch.ones((8, dim // 2), device="cuda"), torch.zeros((8, dim // 2), device="cuda")
    pos = torch.randint(0, 8, (tokens,), generator=g, device="cuda")
    gamma = torch.ones(dim, dtype=dtype, device="cuda")
    got = rq().rmsnorm_rope_backward(dq, dk, q, k, gamma, gamma, one, none, pos, interleaved=inter, epsilon=0.0,
                                     param_grad_dtype=torch.float32)[2:]
    for i, (x, dy) in enumerate(((q, dq), (k, dk))):
        want, size = (dy.double() * x.double()).sum((0, 1)), dy.double().abs().sum((0, 1))
        most = (6 + 2 * turns[i] + 5 + 6 + math.ceil(ctas[i] / 32) + 32) * U * 1.001 * size
        assert float(most.max()) < 0.25 and float(size.min()) > 8
        assert bool(((got[i].double() - want).abs() <= most).all()), float((got[i].double() - want).abs().max())
