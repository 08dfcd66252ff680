"""The layer-norm and int8 calls as the first CUDA work of a process that captures them: function
attributes, the tensor-map encoder and lazily loaded kernels are all set up inside the capture.
Run in a process of its own, which compares the replayed graph with eager calls made afterwards."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
import rmsnorm_precision_activation_gb300 as rq
g = torch.Generator(device="cuda").manual_seed(1)
n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
x = {h: n(40, h) for h in (96, 1003, 4096, 20000)}
w = {h: n(h) for h in x}
stat = torch.rand(40, device="cuda") + 0.5
q = {m: torch.randint(-128, 128, (m, 1040), device="cuda", dtype=torch.int8) for m in (1, 12, 24, 60, 100, 400)}
weight = torch.randint(-128, 128, (300, 1040), device="cuda", dtype=torch.int8)
sw = torch.rand(300, device="cuda")
sa = {m: torch.rand(m, device="cuda") for m in q}

def calls():
    out = []
    for h in x:
        out += rq.layernorm(x[h], w[h], w[h], stats=True)
        out += rq.layernorm_backward(x[h], x[h], w[h], stat, stat)
        out += rq.layernorm_quant_int8(x[h], w[h])
        out += rq.rmsnorm_quant_int8(x[h], w[h])
    for m in q:
        out.append(rq.matmul_int8(q[m], sa[m], weight, sw))
    return [t for t in out if t is not None]

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


@pytest.mark.gpu
def test_first_call_in_a_capture():
    run = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip().endswith("same"), run.stderr[-2000:]
