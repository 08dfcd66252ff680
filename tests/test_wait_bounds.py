"""The bounds of device-side waits that layernorm_backward and matmul_int8 get from
rmsq_set_wait_timeout_ns: what is asked for, up to the stated most, and four times it (a second at
least) for what a stopping CTA has in flight, without wrapping around."""
import pytest
import torch

import host_program
from gpu_common import rq

SECOND = 10 ** 9
SETTINGS = [1, 1023, 1024, 10 ** 6, 2 * SECOND, 4 * SECOND, 5 * SECOND, 60 * SECOND, 2 ** 39, 2 ** 40, 2 ** 41, 2 ** 61,
            2 ** 62, 2 ** 64 - 1]


def test_units(tmp_path):
    out = host_program.run("""
#include <cstdio>
#include <initializer_list>
#include "rmsq_ops_plan.h"
int main()
{
    for (uint64_t ns : {%s})
        std::printf("%%llu %%u %%u\\n", (unsigned long long)ns, rmsq::wait_units(ns), rmsq::drain_units(ns));
}
""" % ", ".join("%dull" % s for s in SETTINGS), tmp_path)
    rows = [tuple(int(v) for v in line.split()) for line in out.splitlines()]
    assert [r[0] for r in rows] == SETTINGS
    for ns, wait, drain in rows:
        # a unit is 1024 ns; a wait lasts what is asked, a unit more at most
        assert ns <= 2 ** 40 and ns < wait * 1024 <= ns + 1024 or ns >= 2 ** 40 and wait == 2 ** 30
        assert drain == max(4 * wait, SECOND // 1024) if wait <= 2 ** 29 else drain == 2 ** 31


@pytest.mark.gpu
@pytest.mark.parametrize("ns", SETTINGS[4:])
def test_results_under_each_bound(ns):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((300, 20000), generator=g, device="cuda").bfloat16()
    w = torch.ones(20000, device="cuda").bfloat16()
    stat = torch.ones(300, device="cuda")
    q = torch.randint(-128, 128, (300, 1040), generator=g, device="cuda", dtype=torch.int8)
    one = torch.ones(300, device="cuda")

    def calls():
        return (*rq().layernorm_backward(x, x, w, stat, stat), rq().matmul_int8(q, one, q, one),
                rq().matmul_int8(q[:40], one[:40], q, one))

    want = calls()
    rq().lib().rmsq_set_wait_timeout_ns(ns)
    try:
        got = calls()
        assert rq().rmsq_device_status() == 0
    finally:
        rq().lib().rmsq_set_wait_timeout_ns(2 * SECOND)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
