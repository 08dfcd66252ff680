"""The aliases that layernorm and layernorm_backward allow, at whole-vector, odd and clustered widths: the
bits of the call with separate outputs. (output = input together with residual_output = residual, and
grad_input = grad_residual, are tested beside the operators.)"""
import pytest
import torch

from gpu_common import rq
from test_layernorm import make, make_backward

gpu = pytest.mark.gpu
WIDTHS = [1, 61, 1000, 1003, 4096, 5121, 9001, 12000, 20000, 40001, 65544, 66001]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)


@gpu
@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward(hidden, dtype):
    if hidden > 65536 and dtype == torch.float32:
        hidden = 65533
    d = make(50, hidden, dtype, seed=hidden, residual=True)
    want = rq().layernorm(d["x"], d["gamma"], d["beta"], residual=d["residual"], stats=True)
    # residual_output = input
    x = d["x"].clone()
    got = rq().layernorm(x, d["gamma"], d["beta"], residual=d["residual"], residual_output=x, stats=True)
    assert same(want, got) and torch.equal(x, want[1])
    # residual_output = residual
    r = d["residual"].clone()
    got = rq().layernorm(d["x"], d["gamma"], d["beta"], residual=r, residual_output=r, stats=True)
    assert same(want, got) and torch.equal(r, want[1])
    # output = input, with a residual and without one
    x = d["x"].clone()
    got = rq().layernorm(x, d["gamma"], d["beta"], residual=d["residual"], output=x, stats=True)
    assert same(want, got) and torch.equal(x, want[0])
    want, x = rq().layernorm(d["x"], d["gamma"], d["beta"], stats=True), d["x"].clone()
    got = rq().layernorm(x, d["gamma"], d["beta"], output=x, stats=True)
    assert same(want, got) and torch.equal(x, want[0])


@gpu
@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("rms", [False, True])
def test_int8_with_the_residual_in_place(hidden, rms):
    d = make(50, hidden, torch.float16, seed=hidden, residual=True)
    call = rq().rmsnorm_quant_int8 if rms else rq().layernorm_quant_int8
    want = call(d["x"], d["gamma"], residual=d["residual"])
    for key in ("x", "residual"):
        e = {k: v.clone() for k, v in d.items()}
        got = call(e["x"], e["gamma"], residual=e["residual"], residual_output=e[key])
        assert same(want, got) and torch.equal(e[key], want[2])


@gpu
@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_backward(hidden, dtype, residual):
    if hidden > 65536 and dtype == torch.float32:
        hidden = 65533
    d = make_backward(300, hidden, dtype, hidden, residual)
    stats = (d["gamma"], d["mean"], d["rstd"])
    want = rq().layernorm_backward(d["dy"], d["x"], *stats, grad_residual=d["dres"])
    for key in ("dy", "x", "dres"):
        if d[key] is None:
            continue
        e = {k: d[k] if d[k] is None else d[k].clone() for k in ("dy", "x", "dres")}
        got = rq().layernorm_backward(e["dy"], e["x"], *stats, grad_residual=e["dres"], grad_input=e[key])
        assert same(want, got) and torch.equal(e[key], want[0]), key
    assert rq().rmsq_device_status() == 0
