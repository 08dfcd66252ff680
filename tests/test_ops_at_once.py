"""The layer-norm and int8 calls from several threads at once, each on a stream of its own, and without
programmatic dependent launch: the same bits as one call after another."""
import threading

import pytest
import torch

from gpu_common import rq

gpu = pytest.mark.gpu


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    c = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    return dict(x={h: n(200, h) for h in (512, 4096, 5001, 20000, 65536)},
                w={h: n(h) for h in (512, 4096, 5001, 20000, 65536)},
                q={m: c(m, 2064) for m in (1, 16, 30, 60, 100, 300, 700)}, weight=c(1030, 2064),
                sa=torch.rand(700, device="cuda", generator=g), sw=torch.rand(1030, device="cuda", generator=g))


def calls(d):
    out = []
    for h, x in d["x"].items():
        y, _, mean, rstd = rq().layernorm(x, d["w"][h], d["w"][h], stats=True)
        out += [y, mean, rstd, *rq().layernorm_backward(y, x, d["w"][h], mean, rstd)]
        out += [*rq().layernorm_quant_int8(x, d["w"][h])[:2], *rq().rmsnorm_quant_int8(x, d["w"][h])[:2]]
    for m, q in d["q"].items():
        out.append(rq().matmul_int8(q, d["sa"][:m], d["weight"], d["sw"]))
    return out


@gpu
def test_threads_with_streams_of_their_own():
    data = [inputs(s) for s in range(3)]
    want = [calls(d) for d in data]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(8):
                got = calls(data[i])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and rq().rmsq_device_status() == 0


@gpu
def test_without_dependent_launch():
    d = inputs(7)
    want = calls(d)
    rq().lib().rmsq_set_pdl(0)
    try:
        got = calls(d)
    finally:
        rq().lib().rmsq_set_pdl(1)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
