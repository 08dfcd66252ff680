"""The gradients of the heads' norm with rotation where some tokens are padding: with places outside the table, and as the header says
to mark them."""
import pytest
import torch

from test_rmsnorm_rope import DTYPES, U, backward, make

gpu = pytest.mark.gpu
PAD = [0, 3, 4, 17, 29]


def padded(dtype, inter):
    d = make(30, 6, 2, 64, dtype, 12, rotated=48, inter=inter)
    keep = torch.ones(30, dtype=torch.bool, device="cuda")
    keep[PAD] = False
    return d, keep


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
def test_places_outside_the_table_reach_the_gammas_gradients(dtype, inter):
    d, keep = padded(dtype, inter)
    want = backward(d, param_grad_dtype=torch.float32)
    d["pos"][PAD] = -1
    got = backward(d, param_grad_dtype=torch.float32)
    for g, w in zip(got[:2], want[:2]):
        assert torch.isnan(g[~keep]).all() and torch.equal(g[keep], w[keep])
    for g, w in zip(got[2:], want[2:]):
        assert torch.isnan(g[:48]).all() and torch.equal(g[48:], w[48:])


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
def test_padding_with_gradients_of_zero_adds_nothing(dtype, inter):
    """Against the other tokens alone: the same terms in another order, each sum off by (20 + n) u of its magnitudes at most
    (test_rmsnorm_rope.py), which are at most twice |dy| |xhat| each."""
    d, keep = padded(dtype, inter)
    d["pos"][PAD] = 0
    d["dq"][PAD], d["dk"][PAD] = 0, 0
    got = backward(d, param_grad_dtype=torch.float32)
    e = dict(d, **{n: d[n][keep] for n in ("q", "k", "dq", "dk", "pos")})
    want = backward(e, param_grad_dtype=torch.float32)
    for i, (x, dy) in enumerate(((e["q"], e["dq"]), (e["k"], e["dk"]))):
        assert bool((got[i][~keep] == 0).all()) and torch.equal(got[i][keep], want[i])
        most = 2 * float(dy.double().abs().max()) * float((x.double() * torch.rsqrt(x.double().square().mean(-1, keepdim=True))).abs().max())
        n = x.shape[0] * x.shape[1]
        assert bool(((got[2 + i] - want[2 + i]).abs() <= 2 * (20 + n) * U * n * most).all())
