"""Calls on some of the tokens or channels of larger tensors: scales, bias and row statistics that are
slices off 16-byte boundaries give the bits that whole calls give, eagerly, on a side stream and in a
captured graph that is replayed on new values."""
import pytest
import torch

from gpu_common import rq
from test_layernorm import make as make_norm, make_backward
from test_matmul_int8 import make

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("first,last", [(1, 3), (2, 40), (3, 131), (5, 6), (129, 260)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matmul_on_some_tokens(first, last, dtype):
    d = make(260, 520, 208, seed=first, dtype=dtype)
    whole = rq().matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"], out_dtype=dtype)
    some = slice(first, last)
    args = (d["a"][some], d["sa"][some], d["w"], d["sw"])
    assert torch.equal(rq().matmul_int8(*args, bias=d["bias"], out_dtype=dtype), whole[some])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = rq().matmul_int8(*args, bias=d["bias"], out_dtype=dtype, stream=side)
    side.synchronize()
    assert torch.equal(out, whole[some])


@gpu
@pytest.mark.parametrize("first,last", [(1, 90), (3, 520), (7, 8), (130, 401)])
@pytest.mark.parametrize("m", [1, 30, 260])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_matmul_on_some_channels(first, last, m, dtype):
    d = make(m, 520, 208, seed=last, dtype=dtype)
    whole = rq().matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"], out_dtype=dtype)
    some = slice(first, last)
    out = rq().matmul_int8(d["a"], d["sa"], d["w"][some], d["sw"][some], bias=d["bias"][some], out_dtype=dtype)
    assert torch.equal(out, whole[:, some])


@gpu
def test_captured_with_slices():
    d = make(50, 300, 208, seed=3)
    some = slice(1, 30)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rq().matmul_int8(d["a"][some], d["sa"][some], d["w"], d["sw"], bias=d["bias"])
    for f in (1.0, 3.0):
        d["sa"].mul_(f)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, rq().matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"])[some])


@gpu
@pytest.mark.parametrize("hidden", [64, 2048, 20000])
def test_backward_on_some_rows(hidden):
    d = make_backward(40, hidden, torch.bfloat16, hidden, residual=True)
    whole = rq().layernorm_backward(d["dy"], d["x"], d["gamma"], d["mean"], d["rstd"], grad_residual=d["dres"])
    for some in (slice(1, 3), slice(7, 40)):
        args = [d[k][some] for k in ("dy", "x")]
        # (rows of whole vectors: a row's gradient does not depend on where it stands)
        got = rq().layernorm_backward(*args, d["gamma"], d["mean"][some], d["rstd"][some], grad_residual=d["dres"][some])
        want = rq().layernorm_backward(*args, d["gamma"], d["mean"][some].clone(), d["rstd"][some].clone(),
                                       grad_residual=d["dres"][some])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(got[0], whole[0][some])
    assert rq().rmsq_device_status() == 0


@gpu
@pytest.mark.parametrize("name", ["layernorm_quant_int8", "rmsnorm_quant_int8"])
@pytest.mark.parametrize("hidden", [64, 2048])
def test_int8_rows_written_in_pieces(name, hidden):
    call = getattr(rq(), name)
    d = make_norm(50, hidden, torch.bfloat16, seed=hidden)
    want = call(d["x"], d["gamma"])
    q = torch.zeros(50, hidden, dtype=torch.int8, device="cuda")
    scale = torch.full((52,), 7.0, device="cuda")
    ends = [0, 1, 3, 4, 9, 30, 50]
    for a, b in zip(ends, ends[1:]):
        call(d["x"][a:b], d["gamma"], output=q[a:b], scale_output=scale[a:b])
    assert torch.equal(q, want[0]) and torch.equal(scale[:50], want[1]) and bool((scale[50:] == 7.0).all())
    # on a side stream, and captured and replayed on new inputs
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(d["x"][1:30], d["gamma"], output=q[1:30], scale_output=scale[1:30], stream=side)
    side.synchronize()
    assert torch.equal(got[1], want[1][1:30]) and got[1].data_ptr() == scale[1:30].data_ptr()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(d["x"][1:30], d["gamma"], output=q[1:30], scale_output=scale[1:30])
    for f in (2.0, 0.5):
        d["x"].mul_(f)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(scale[1:30], call(d["x"], d["gamma"])[1][1:30])
