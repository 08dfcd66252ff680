"""The quantising RMS norms and the layer-norm and int8 operators one after another on shared buffers, as
a model that mixes them runs: kernels that start while the one before them ends give the bits that kernels
run one at a time give. And rows that are not finite stay to themselves where vectors span two rows."""
import pytest
import torch

from gpu_common import rq
from test_layernorm import make_backward

gpu = pytest.mark.gpu


class Chain:
    """Buffers that every pass overwrites, so that a kernel that starts early meets the last one's."""

    def __init__(self, rows, hidden, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        c = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
        new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.x, self.r, self.w, self.b = n(rows, hidden), n(rows, hidden), n(hidden), n(hidden)
        self.weight, self.scale = c(hidden, hidden), torch.rand(hidden, generator=g, device="cuda") * 1e-3
        self.s, self.y, self.ds = (new(rows, hidden) for _ in range(3))
        self.fp8 = new(rows, hidden, dtype=torch.float8_e4m3fn)
        self.q, self.q_scale = new(rows, hidden, dtype=torch.int8), new(rows, dtype=torch.float32)
        self.dg, self.db = new(hidden, dtype=torch.float32), new(hidden, dtype=torch.float32)
        self.work = new(rq().layernorm_backward_workspace(rows, hidden), dtype=torch.uint8)

    def run(self, x, pause):
        m, out = rq(), []

        def step(*t):
            if pause:
                torch.cuda.synchronize()
            return t

        step(m.rmsnorm_quant_fp8(x, self.w, residual=self.r, residual_output=self.s, output=self.fp8))
        _, _, mean, rstd = m.layernorm(self.s, self.w, self.b, output=self.y, stats=True)
        step(m.rmsnorm_quant_int8(self.y, self.w, residual=self.s, residual_output=self.s, output=self.q,
                                  scale_output=self.q_scale))
        step(m.matmul_int8(self.q, self.q_scale, self.weight, self.scale, output=self.y))
        nv = m.rmsnorm_quant_nvfp4(self.y, self.w, global_scale=m.rmsnorm_nvfp4_global_scale(self.y, self.w))
        step()
        step(m.layernorm_quant_int8(self.y, self.w, self.b, output=self.q, scale_output=self.q_scale))
        step(m.matmul_int8(self.q, self.q_scale, self.weight, self.scale, output=self.y))
        step(m.layernorm_backward(self.y, self.s, self.w, mean, rstd, grad_input=self.ds, grad_gamma=self.dg,
                                  grad_beta=self.db, param_grad_dtype=torch.float32, workspace=self.work))
        step(m.layernorm(self.ds, self.w, residual=self.s, residual_output=self.s, output=self.ds))
        out += [t.clone() for t in (self.s, self.y, self.ds, self.dg, self.db, self.q, self.q_scale)]
        return out + [self.fp8.view(torch.uint8).clone(), nv[0].clone(), nv[1].view(torch.uint8).clone()]


@gpu
@pytest.mark.parametrize("rows,hidden", [(1, 1024), (16, 4096), (30, 1024), (100, 4096), (300, 2048), (700, 9216)])
def test_kernels_that_overlap_give_the_same_bits(rows, hidden):
    chain = Chain(rows, hidden, seed=rows)
    inputs = [chain.x * (1.0 + 0.25 * i) for i in range(4)]
    rq().lib().rmsq_set_pdl(0)
    try:
        want = [chain.run(x, pause=True) for x in inputs]
    finally:
        rq().lib().rmsq_set_pdl(1)
    for _ in range(5):
        got = [chain.run(x, pause=False) for x in inputs]
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert rq().rmsq_device_status() == 0


@gpu
@pytest.mark.parametrize("hidden", [5, 61, 1003, 5121, 9001, 20001, 66001])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_not_finite_stay_to_themselves(hidden, bad):
    # rows share 16-byte vectors with their neighbours at these widths
    d = make_backward(20, hidden, torch.bfloat16, hidden, residual=True)
    keep = [i for i in range(20) if i not in (3, 11)]

    def calls():
        y, s, mean, rstd = rq().layernorm(d["x"], d["gamma"], d["beta"], residual=d["dres"], stats=True)
        ds, dg, db = rq().layernorm_backward(d["dy"], d["x"], d["gamma"], d["mean"], d["rstd"], grad_residual=d["dres"])
        return (y, s, mean, rstd, ds), (dg, db)

    for key in ("x", "dy", "dres"):
        d[key][3], d[key][11] = 0.5, 0.5
    clean, sums = calls()
    d["x"][3, 0] = d["x"][11, hidden - 1] = bad
    rows, _ = calls()
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(rows, clean))
    assert rows[0][[3, 11]].isnan().all()
    d["x"][3, 0] = d["x"][11, hidden - 1] = 0.5
    # a gradient that is not finite reaches its own row and its own column of the sums alone
    d["dy"][3, 0] = d["dy"][11, hidden - 1] = bad
    rows, (dg, db) = calls()
    assert torch.equal(rows[4][keep], clean[4][keep]) and not rows[4][[3, 11]].isfinite().any()
    inner = slice(1, hidden - 1)
    assert torch.equal(dg[inner], sums[0][inner]) and torch.equal(db[inner], sums[1][inner])
    assert not db[0].isfinite() and not db[-1].isfinite()
    assert rq().rmsq_device_status() == 0
