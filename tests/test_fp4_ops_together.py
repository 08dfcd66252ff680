"""The 4-bit quantisation and products and the per-head norm with rotation as a model runs them: from a residual stream to
queries, keys and values, from an attention's output through its projection, and the queries' and keys' gradients. Each
step against its formula in 64 bits; kernels that overlap, several threads, graphs and bounds of waits against the
same calls one at a time, bit for bit."""
import os
import re
import subprocess
import sys
import threading
import types

import pytest
import torch

import fp4_common as F
import test_matmul_fp4 as M
import test_rmsnorm_rope as R
from gpu_common import rq

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADS, KV, DIM = 8, 2, 64
WIDTH = (HEADS + 2 * KV) * DIM


def make(tokens, hidden, fmt, seed):
    """A layer's weights, inputs, and buffers that every pass overwrites."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    new = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    d = dict(fmt=fmt, tokens=tokens, x=n(tokens, hidden), r=n(tokens, hidden), gamma=n(hidden), gq=n(DIM), gk=n(DIM),
             gs=torch.full((1,), 200.0, device="cuda"), res=new(tokens, hidden), qkv=new(tokens, WIDTH), out=new(tokens, hidden))
    for name, rows, k in (("wqkv", WIDTH, hidden), ("wo", hidden, HEADS * DIM)):
        w = torch.randn((rows, k), generator=g, device="cuda") * 0.05
        if fmt == "nvfp4":
            d[name + "_g"] = rq().nvfp4_global_scale(w)
            d[name], d[name + "_s"] = rq().quant_nvfp4(w, global_scale=d[name + "_g"], swizzled=True)
        else:
            d[name], d[name + "_s"] = rq().quant_mxfp4(w, swizzled=True)
    d["cos"], d["sin"] = R.table(300, DIM // 2)
    d["pos"] = torch.randint(0, 300, (tokens,), generator=g, device="cuda")
    d["dq"], d["dk"] = n(tokens, HEADS, DIM), n(tokens, KV, DIM)
    return d


def heads(qkv):
    return (qkv[:, :HEADS * DIM].unflatten(1, (HEADS, DIM)), qkv[:, HEADS * DIM:(HEADS + KV) * DIM].unflatten(1, (KV, DIM)),
            qkv[:, (HEADS + KV) * DIM:])


def layer(d, x, pause=False, stream=None):
    """One pass; every output, copied where a buffer holds it."""
    q, nv, out = rq(), d["fmt"] == "nvfp4", []
    kw = dict(stream=stream)

    def step(*t):
        if pause:
            torch.cuda.synchronize()
        return t

    if nv:
        c, s, _ = step(*q.rmsnorm_quant_nvfp4(x, d["gamma"], global_scale=d["gs"], residual=d["r"], residual_output=d["res"],
                                              swizzled=True, **kw))
        step(q.matmul_nvfp4(c, s, d["wqkv"], d["wqkv_s"], input_global_scale=d["gs"], weight_global_scale=d["wqkv_g"],
                            output=d["qkv"], **kw))
    else:
        c, s, _ = step(*q.rmsnorm_quant_mxfp4(x, d["gamma"], residual=d["r"], residual_output=d["res"], swizzled=True, **kw))
        step(q.matmul_mxfp4(c, s, d["wqkv"], d["wqkv_s"], output=d["qkv"], **kw))
    hq, hk, _ = heads(d["qkv"])
    rope = (d["gq"], d["gk"], d["cos"], d["sin"], d["pos"])
    grads = step(*q.rmsnorm_rope_backward(d["dq"], d["dk"], hq, hk, *rope, **kw))
    y = step(*q.rmsnorm_rope(hq, hk, *rope, **kw))
    attended = y[0].view(d["tokens"], HEADS * DIM)
    if nv:
        gs = step(q.nvfp4_global_scale(attended, **kw))[0]
        oc, os_ = step(*q.quant_nvfp4(attended, global_scale=gs, swizzled=True, **kw))
        step(q.matmul_nvfp4(oc, os_, d["wo"], d["wo_s"], input_global_scale=gs, weight_global_scale=d["wo_g"], output=d["out"], **kw))
    else:
        gs = None
        oc, os_ = step(*q.quant_mxfp4(attended, swizzled=True, **kw))
        step(q.matmul_mxfp4(oc, os_, d["wo"], d["wo_s"], output=d["out"], **kw))
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
        out = [d["res"].clone(), d["qkv"].clone(), *y, *grads, d["out"].clone(), c, oc]
    return out, (c, s, oc, os_, gs)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens,hidden", [(1, 512), (20, 1024), (70, 544), (300, 2048)])
def test_each_step_of_a_layer(fmt, tokens, hidden):
    d = make(tokens, hidden, fmt, tokens)
    out, (c, s, oc, os_, gs) = layer(d, d["x"])
    nv = fmt == "nvfp4"

    def product(codes, scale, k, w, g, got):
        rows = lambda t, n: F.untiled(t.view(torch.uint8), n, k // F.BLOCK[fmt])[0]  # noqa: E731
        m = dict(a=codes, sa=rows(scale, tokens), ta=scale, w=d[w], sw=rows(d[w + "_s"], d[w].shape[0]), tw=d[w + "_s"], fmt=fmt,
                 dtype=torch.bfloat16, ga=g if nv else None, gw=d[w + "_g"] if nv else None, bias=None)
        assert torch.equal(M.check(m), got)

    product(c, s, hidden, "wqkv", d["gs"], out[1])
    product(oc, os_, HEADS * DIM, "wo", gs, out[8])
    hq, hk, _ = heads(out[1])
    e = dict(q=hq, k=hk, dq=d["dq"], dk=d["dk"], gq=d["gq"], gk=d["gk"], cos=d["cos"], sin=d["sin"], pos=d["pos"], sections=None,
             inter=False, offset=0.0)
    assert same(R.check_forward(e), out[2:4]) and same(R.check_backward(e), out[4:8])


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens,hidden", [(1, 1024), (24, 2048), (60, 1024), (120, 1024), (600, 2048)])
def test_kernels_that_overlap_give_the_same_bits(fmt, tokens, hidden):
    d = make(tokens, hidden, fmt, 3)
    inputs = [d["x"] * (1.0 + 0.25 * i) for i in range(4)]
    rq().lib().rmsq_set_pdl(0)
    try:
        want = [layer(d, x, pause=True)[0] for x in inputs]
    finally:
        rq().lib().rmsq_set_pdl(1)
    torch.cuda.synchronize()
    for _ in range(5):
        got = [layer(d, x)[0] for x in inputs]
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
    assert rq().rmsq_device_status() == 0


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_threads_with_streams_of_their_own(fmt):
    data = [make(t, 1024, fmt, t) for t in (2, 90, 400)]
    want = [layer(d, d["x"])[0] for d in data]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(8):
                got = layer(data[i], data[i]["x"])[0]
                stream.synchronize()
                if not same(got, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and rq().rmsq_device_status() == 0


@gpu
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_two_graphs_at_once(fmt):
    data = [make(t, 1024, fmt, t) for t in (30, 300)]
    bufs, graphs, outs = [], [], []
    for d in data:
        layer(d, d["x"])
        buf = d["x"].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(d, buf)[0]
        bufs.append(buf)
        graphs.append(graph)
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in data]
    for f in (2.0, 0.5):
        for d, buf in zip(data, bufs):
            buf.copy_(d["x"] * f)
        torch.cuda.synchronize()
        for _ in range(6):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in out] for out in outs]
        for d, g in zip(data, got):
            assert same(g, layer(d, d["x"] * f)[0])


@gpu
@pytest.mark.parametrize("ns", [10 ** 6, 5 * 10 ** 9, 2 ** 40, 2 ** 62])
def test_results_under_each_bound(ns):
    d = [M.make(m, 300, 1056, "nvfp4", seed=m) for m in (1, 24, 60, 100, 600)]
    want = [M.call(e) for e in d]
    rq().lib().rmsq_set_wait_timeout_ns(ns)
    try:
        got = [M.call(e) for e in d]
        assert rq().rmsq_device_status() == 0
    finally:
        rq().lib().rmsq_set_wait_timeout_ns(2 * 10 ** 9)
    assert same(got, want)


PROGRAM = """
import sys
sys.path.insert(0, "tests")
import torch
import rmsnorm_precision_activation_gb300 as rq
g = torch.Generator(device="cuda").manual_seed(1)
n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
codes = {m: torch.randint(0, 256, (m, 544), device="cuda", dtype=torch.uint8) for m in (1, 24, 60, 100, 600)}
weight = torch.randint(0, 256, (300, 544), device="cuda", dtype=torch.uint8)
scale = lambda rows, block: torch.full((rq.swizzled_scale_numel(rows, 1088, block),), 0x38 if block == 16 else 120, device="cuda", dtype=torch.uint8)
sa = {b: {m: scale(m, b) for m in codes} for b in (16, 32)}
sw = {b: scale(300, b) for b in (16, 32)}
x = {h: n(100, h) for h in (64, 1024, 4096)}
heads = [(n(9, 4, d), n(9, 2, d), n(d), n(d), torch.rand(50, d // 2, device="cuda"), torch.rand(50, d // 2, device="cuda")) for d in (64, 72, 130)]
pos = torch.arange(9, device="cuda")

def calls():
    out = []
    for h in x.values():
        gs = rq.nvfp4_global_scale(h)
        out += [gs, *rq.quant_nvfp4(h, global_scale=gs), *rq.quant_mxfp4(h)]
    for m in codes:
        out.append(rq.matmul_nvfp4(codes[m], sa[16][m], weight, sw[16]))
        out.append(rq.matmul_mxfp4(codes[m], sa[32][m], weight, sw[32]))
    for q, k, gq, gk, c, s in heads:
        for inter in (False, True):
            out += rq.rmsnorm_rope(q, k, gq, gk, c, s, pos, interleaved=inter)
            out += rq.rmsnorm_rope_backward(q, k, q, k, gq, gk, c, s, pos, interleaved=inter)
    return [t.view(torch.uint8) for t in out]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, calls()))
assert rq.rmsq_device_status() == 0
print("same")
"""


@gpu
def test_first_call_in_a_capture():
    # function attributes, the tensor-map encoder and lazily loaded kernels are all set up inside the capture
    run = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip().endswith("same"), run.stderr[-2000:]


CALLS = {
    "nvfp4_global_scale": lambda x, s: rq().nvfp4_global_scale(x, stream=s),
    "quant_nvfp4": lambda x, s: rq().quant_nvfp4(x, stream=s),
    "quant_mxfp4": lambda x, s: rq().quant_mxfp4(x, stream=s),
    "matmul_nvfp4": lambda x, s: rq().matmul_nvfp4(x, None, None, None, stream=s),
    "matmul_mxfp4": lambda x, s: rq().matmul_mxfp4(x, None, None, None, stream=s),
    "rmsnorm_rope": lambda x, s: rq().rmsnorm_rope(x, *[None] * 6, stream=s),
    "rmsnorm_rope_backward": lambda x, s: rq().rmsnorm_rope_backward(None, None, x, *[None] * 6, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(name):
    # stand-ins for a tensor of device 0 and a stream of device 1
    x = types.SimpleNamespace(is_cuda=True, get_device=lambda: 0)
    with pytest.raises(ValueError, match="stream of the input's device"):
        CALLS[name](x, types.SimpleNamespace(device_index=1))


@pytest.mark.parametrize("name", ["rmsq_fp4.cuh", "rmsq_fp4_pair.cuh"])
def test_tmem_is_allocated_before_dependents_may_come(name):
    # (a CTA of the next kernel could take an SM's columns and then wait for this kernel; not for a GPU to show)
    with open(os.path.join(ROOT, "rmsnorm_precision_activation_gb300", "csrc", name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel = text[text.index("__global__"):]
    alloc = kernel.index("tcgen05.alloc")
    assert "pdl_wait()" not in kernel[:alloc] and "launch_dependents" not in kernel[:alloc]
    after = kernel[alloc:]
    assert after.index("__syncthreads()") < after.index("pdl_wait()")
