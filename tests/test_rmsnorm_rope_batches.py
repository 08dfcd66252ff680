"""Batches of heads that lie before their tokens, as attention code holds them: one sequence as it is, several one at a time."""
import pytest
import torch

from gpu_common import rq
from test_rmsnorm_rope import DTYPES, forward, make

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_heads_before_tokens(dtype):
    d = make(2 * 11, 6, 2, 64, dtype, 7)
    want = [y.unflatten(0, (2, 11)) for y in forward(d)]
    q, k = (d[n].unflatten(0, (2, 11)).transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k"))      # [2, 11, heads, 64]
    pos = d["pos"].view(2, 11)
    with pytest.raises(ValueError, match="leading dimensions"):
        forward(dict(d, q=q, k=k, pos=pos))
    outs = [torch.empty_strided(t.shape, t.stride(), dtype=dtype, device="cuda") for t in (q, k)]
    for b in range(2):
        forward(dict(d, q=q[b], k=k[b], pos=pos[b]), query_output=outs[0][b], key_output=outs[1][b])
        one = forward(dict(d, q=q[b:b + 1], k=k[b:b + 1], pos=pos[b:b + 1]))       # a batch of one
        assert all(torch.equal(y[0], w[b]) for y, w in zip(one, want))
    assert all(torch.equal(y, w) for y, w in zip(outs, want)) and rq().rmsq_device_status() == 0
