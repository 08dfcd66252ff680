"""How layer norm's backward pass deals rows out to clusters: every row to one group, a CTA's rows at one
place against a 16-byte boundary, no more partial rows than the workspace has, and a plan for every valid
call, however few clusters the device runs at a time."""
import collections

import pytest
import torch

import host_program
from gpu_common import rq
from test_layernorm import check_backward, make_backward

ROWS = [1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 15, 16, 17, 40, 151, 152, 153, 160, 305, 1000]


@pytest.mark.parametrize("period", [1, 2, 4, 8])
def test_every_row_has_a_group_of_its_place(period, tmp_path):
    out = host_program.run("""
#include <cstdio>
#include <initializer_list>
#include "rmsq_ops_plan.h"
int main()
{
    for (int rows : {%s})
        for (int groups : {1, 2, 3, 7, 15})
            for (int resident : {1, 2, 3, 5, 6, 7, 8, 9, 15, 16, 19, 37, 75, 152})
                std::printf("%%d %%d %%d %%lld\\n", rows, groups, resident,
                            (long long)rmsq::bwd_clusters(rows, groups, %d, resident, rows < 152 ? rows : 152));
}
""" % (", ".join(map(str, ROWS)), period), tmp_path)
    for line in out.splitlines():
        rows, groups, resident, clusters = map(int, line.split())
        if groups > 1 and rows < 100:          # a device has more SMs than that, and a CTA no second group
            continue
        assert 1 <= clusters <= min(rows, 152), line
        # more than run at a time only for the sake of the period
        assert clusters <= max(resident, period), line
        taken = collections.Counter()
        for c in range(clusters):
            mine = [r for g in range(groups) for r in range(g * clusters + c, rows, clusters * groups)]
            taken.update(mine)
            assert len({r % period for r in mine}) <= 1, line
        assert taken == collections.Counter(range(rows)), line


@pytest.mark.gpu
@pytest.mark.parametrize("rows", range(1, 10))
@pytest.mark.parametrize("hidden,dtype", [(131071, torch.bfloat16), (131070, torch.float16), (65535, torch.float32),
                                          (40001, torch.bfloat16)])
def test_few_wide_rows_off_16_byte_boundaries(rows, hidden, dtype):
    check_backward(make_backward(rows, hidden, dtype, rows, residual=rows % 2 == 0))
    assert rq().rmsq_device_status() == 0
