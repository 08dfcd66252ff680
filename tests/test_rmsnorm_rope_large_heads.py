"""Heads whose elements are finite and whose squares leave float's range, beside ordinary ones."""
import pytest
import torch

from test_rmsnorm_rope import backward, check_backward, check_forward, forward, make

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim", [64, 66, 128])
def test_a_head_whose_squares_leave_the_range(dtype, inter, dim):
    d = make(13, 8, 2, dim, dtype, 21, inter=inter)
    want, grads = forward(d), backward(d)
    e = dict(d, q=d["q"].clone())
    e["q"][5, 3] = 2.0 ** 70
    got, back = forward(e), backward(e)
    assert bool((got[0][5, 3] == 0).all()) and bool((back[0][5, 3] == 0).all())
    for a, b in ((got[0], want[0]), (back[0], grads[0])):
        a[5, 3] = b[5, 3]
        assert torch.equal(a, b)
    assert torch.equal(got[1], want[1]) and torch.equal(back[1], grads[1]) and torch.isfinite(back[2]).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_heads_within_the_range(dtype):
    # 128 squares of at most 2^120: 2^127
    d = make(13, 8, 2, 128, dtype, 22)
    for n in ("q", "k"):
        d[n] = (d[n].double().clamp(-4, 4) * 2.0 ** 58).to(dtype)
    check_forward(d)
    check_backward(d)
