"""A stream of another device than the input's is refused, by every layer-norm and int8 call, before
anything is made current or launched."""
import types

import pytest

from gpu_common import rq

CALLS = {
    "layernorm": lambda x, s: rq().layernorm(x, None, stream=s),
    "layernorm_backward": lambda x, s: rq().layernorm_backward(None, x, None, None, None, stream=s),
    "layernorm_quant_int8": lambda x, s: rq().layernorm_quant_int8(x, None, stream=s),
    "rmsnorm_quant_int8": lambda x, s: rq().rmsnorm_quant_int8(x, None, stream=s),
    "matmul_int8": lambda x, s: rq().matmul_int8(x, None, None, None, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(name):
    # stand-ins for a tensor of device 0 and a stream of device 1
    x = types.SimpleNamespace(is_cuda=True, get_device=lambda: 0)
    with pytest.raises(ValueError, match="stream of the input's device"):
        CALLS[name](x, types.SimpleNamespace(device_index=1))
