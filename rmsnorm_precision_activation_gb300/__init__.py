"""GB300 (sm_103a) fused residual-add + RMSNorm + dynamic FP8 / NVFP4 / MXFP4 quantisation.

Python binding of librmsq.so (C ABI in include/rmsq.h). The functions here only marshal
arguments: they check shapes and dtypes, allocate outputs the caller did not pass, and call the
C entry point of the same name on the current CUDA stream. Every step of the computation runs in
the library's CUDA kernels; there is no fallback. If librmsq.so has not been built, every call
raises.

    out, scale, res_out = rmsnorm_quant_fp8(x, gamma, residual=r, scale_ub=1200.0)
    q, block_scale, res_out = rmsnorm_quant_nvfp4(x, gamma, global_scale=gs)
    q, block_scale, res_out = rmsnorm_quant_mxfp4(x, gamma, residual=r)

    gs = nvfp4_global_scale(w)
    w4, w_scale = quant_nvfp4(w, global_scale=gs, swizzled=True)
    out = matmul_nvfp4(q, block_scale, w4, w_scale, weight_global_scale=gs)      # (q with swizzled=True)
    query, key = rmsnorm_rope(query, key, query_gamma, key_gamma, cos, sin, positions)
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librmsq.so")

RMSQ_BF16, RMSQ_FP16, RMSQ_F32 = 0, 1, 2
SCALE_ROW_MAJOR, SCALE_SWIZZLED_128x4 = 0, 1
SCHED_AUTO, SCHED_PIPE, SCHED_REG, SCHED_WARP, SCHED_CLUSTER = 0, 1, 2, 3, 4
# Widest row accepted, in elements (fp32 input: half). Rows wider than ONE_CTA_HIDDEN (fp32:
# half) run on a thread-block cluster and must be a multiple of 256 elements.
MAX_HIDDEN, ONE_CTA_HIDDEN = 131072, 32768

STATUS = {0: "RMSQ_OK", 1: "RMSQ_ERR_NULL", 2: "RMSQ_ERR_SHAPE", 3: "RMSQ_ERR_ALIGN",
          4: "RMSQ_ERR_DTYPE", 5: "RMSQ_ERR_LAUNCH", 6: "RMSQ_ERR_VALUE", 7: "RMSQ_ERR_DEVICE",
          8: "RMSQ_ERR_TIMEOUT"}

_DT = {torch.bfloat16: RMSQ_BF16, torch.float16: RMSQ_FP16, torch.float32: RMSQ_F32}

# Exported C symbols and their ctypes signatures.
_P, _I64, _I, _F, _U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_uint64
SIGNATURES = {
    "rmsnorm_quant_fp8": ([_P, _P, _P, _P, _I64, _I64, _I, _F, _F, _F, _P, _P, _I, _P], _I),
    "rmsnorm_quant_fp8_static_scratch": ([_P, _P, _P, _P, _I64, _I64, _I, _F, _F, _F, _P, _P, _I, _P], _I),
    "rmsnorm_quant_nvfp4": ([_P, _P, _P, _P, _I64, _I64, _I, _F, _F, _P, _P, _P, _I, _P], _I),
    "rmsnorm_quant_mxfp4": ([_P, _P, _P, _P, _I64, _I64, _I, _F, _F, _P, _P, _I, _P], _I),
    "rmsnorm_nvfp4_global_scale": ([_P, _P, _P, _I64, _I64, _I, _F, _F, _P, _P], _I),
    "layernorm": ([_P, _P, _P, _P, _P, _I64, _I64, _I, _F, _F, _P, _P, _P, _P], _I),
    "layernorm_backward_workspace": ([_I64, _I64], _I64),
    "layernorm_backward": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I, _F, _P, _P, _P, _I, _P, _I64, _P], _I),
    "layernorm_quant_int8": ([_P, _P, _P, _P, _P, _I64, _I64, _I, _F, _F, _P, _P, _P], _I),
    "rmsnorm_quant_int8": ([_P, _P, _P, _P, _I64, _I64, _I, _F, _F, _P, _P, _P], _I),
    "matmul_int8": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I, _P], _I),
    "quant_nvfp4": ([_P, _I64, _I64, _I, _P, _P, _P, _I, _P], _I),
    "quant_mxfp4": ([_P, _I64, _I64, _I, _P, _P, _I, _P], _I),
    "nvfp4_global_scale_workspace": ([_I64], _I64),
    "nvfp4_global_scale": ([_P, _I64, _I, _P, _P, _I64, _P], _I),
    "matmul_nvfp4": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I, _P], _I),
    "matmul_mxfp4": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I, _P], _I),
    "rmsnorm_rope": ([_P, _P, _P, _P, _P, _I64, _I64, _I, _F, _F, _P, _P, _P], _I),
    "rmsnorm_rope_backward_workspace": ([_I64, _I64], _I64),
    "rmsnorm_rope_backward": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I, _F, _F, _P, _P, _P, _P, _I, _P, _I64, _P], _I),
    "rmsq_status_string": ([_I], ctypes.c_char_p),
    "rmsq_device_status": ([], _I),
    "rmsq_set_schedule": ([_I], _I),
    "rmsq_set_tuning": ([_I, _I, _I], _I),
    "rmsq_set_row_warps": ([_I], _I),
    "rmsq_set_cluster_size": ([_I], _I),
    "rmsq_set_dynamic_rows": ([_I], _I),
    "rmsq_set_pdl": ([_I], _I),
    "rmsq_set_wait_timeout_ns": ([_U64], None),
    "rmsq_selftest_wait_timeout": ([_U64, _P], _I),
    "rmsq_debug_convert": ([_I, _P, _P, _I64, _P], _I),
    "rmsq_launch_count": ([], _U64),
    "rmsq_plan": ([_I, _I, _I, _F, _I64, _I, _I, _I, _P], _I),
}

# rmsq_plan's modes, and GB300's shared-memory limits in bytes (opt-in per CTA, per SM, reserved
# per CTA), which let it plan without a GPU.
MODES = {"fp8": 0, "nvfp4": 1, "mxfp4": 2, "global_scale": 3}
GB300_SMEM = (232448, 233472, 1024)


class PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("schedule", "vectors_per_thread", "threads", "stages",
                                            "cluster", "smem_bytes", "ctas_per_sm", "w16")]


# rmsq_heads (data, token_stride, head_stride, heads) and rmsq_rotation (cos, sin, positions, places, position_bits,
# rotated, neighbours, axes, sections[4]) as bytes: packing takes a third of what filling a ctypes structure does.
HEADS, ROTATION = struct.Struct("Pqqq"), struct.Struct("PPPq8i")


_lib = None


class RmsqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, STATUS.get(status, "status %d" % status)))


def lib() -> ctypes.CDLL:
    """The loaded librmsq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("librmsq.so is not built (%s); run "
                               "rmsnorm_precision_activation_gb300.build.build()" % LIB_PATH)
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise RmsqError(status, where)


def _stream(device, stream):
    return _raw_stream(device.index) if stream is None else stream.cuda_stream


def _on(device):
    """Makes the device current; nothing to do, and to undo, where it is (a context costs 3 us a call)."""
    return _NOTHING if device.index == torch.cuda.current_device() else torch.cuda.device(device)


_NOTHING = contextlib.nullcontext()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _flat(t, H):
    return t.reshape(-1, H) if t.dim() != 2 else t


def _prepare(input, gamma, residual, residual_output):
    if not input.is_cuda:
        raise ValueError("input must be a CUDA tensor")
    dtype, shape, index = input.dtype, input.shape, input.get_device()
    if dtype not in _DT:
        raise TypeError("input dtype must be bfloat16, float16 or float32")
    H = shape[-1]
    x = input if len(shape) == 2 else input.reshape(-1, H)
    for name, t in (("input", x), ("gamma", gamma), ("residual", residual)):
        if t is not None and (not t.is_contiguous() or t.dtype is not dtype or t.get_device() != index):
            raise ValueError("%s must be a contiguous %s tensor on %s" % (name, dtype, input.device))
    if gamma.shape != (H,):
        raise ValueError("gamma must have shape (%d,)" % H)
    r = None
    if residual is not None:
        r = residual if residual.dim() == 2 else residual.reshape(-1, H)
        if r.shape != x.shape:
            raise ValueError("residual must have the input's shape")
        if residual_output is None:
            residual_output = torch.empty_like(input)
        if residual_output.shape != shape or not residual_output.is_contiguous():
            raise ValueError("residual_output must be a contiguous tensor of the input's shape")
    elif residual_output is not None:
        raise ValueError("residual_output given without residual")
    ro = None if residual_output is None else _flat(residual_output, H)
    return x, r, ro, residual_output, H


def rmsnorm_quant_fp8(input, gamma, *, residual=None, residual_output=None, epsilon=1e-6,
                      weight_offset=0.0, scale_ub=1200.0, output=None, scale_output=None,
                      scale_dtype=torch.float32, stream=None):
    """Residual add + RMSNorm + FP8 E4M3 with a per-row dynamic scale.

    Returns (output float8_e4m3fn [..., H], scale_output [...] of scale_dtype, residual_output)."""
    x, r, ro, residual_output, H = _prepare(input, gamma, residual, residual_output)
    lead = input.shape[:-1]
    if output is None:
        output = torch.empty(input.shape, dtype=torch.float8_e4m3fn, device=input.device)
    if scale_output is None:
        scale_output = torch.empty(lead, dtype=scale_dtype, device=input.device)
    with _on(input.device):
        st = lib().rmsnorm_quant_fp8(_ptr(x), _ptr(r), _ptr(ro), _ptr(gamma), x.shape[0], H,
                                     _DT[input.dtype], float(epsilon), float(weight_offset),
                                     float(scale_ub), _ptr(output), _ptr(scale_output),
                                     _DT[scale_output.dtype], _stream(input.device, stream))
    _check(st, "rmsnorm_quant_fp8")
    return output, scale_output, residual_output


def swizzled_scale_numel(rows: int, hidden: int, block: int) -> int:
    """Bytes of a swizzled 128x4 block-scale tensor (whole 128 x 4 tiles of 512 bytes)."""
    return ((rows + 127) // 128) * ((hidden // block + 3) // 4) * 512


def _fp4_outputs(input, H, block, output, block_scale, swizzled, scale_torch_dtype):
    rows = input.numel() // H
    if output is None:
        output = torch.empty(tuple(input.shape[:-1]) + (H // 2,), dtype=torch.uint8, device=input.device)
    if block_scale is None:
        if swizzled:
            block_scale = torch.empty(swizzled_scale_numel(rows, H, block), dtype=scale_torch_dtype,
                                      device=input.device)
        else:
            block_scale = torch.empty(tuple(input.shape[:-1]) + (H // block,), dtype=scale_torch_dtype,
                                      device=input.device)
    return output, block_scale


def rmsnorm_quant_nvfp4(input, gamma, *, global_scale=None, residual=None, residual_output=None,
                        epsilon=1e-6, weight_offset=0.0, output=None, block_scale=None,
                        swizzled=False, stream=None):
    """Residual add + RMSNorm + NVFP4 (packed E2M1, E4M3 scale per 16 elements, fp32 global
    scale read on the device). global_scale: a CUDA float32 tensor of one element (default 1.0).

    Returns (output uint8 [..., H/2], block_scale float8_e4m3fn, residual_output)."""
    x, r, ro, residual_output, H = _prepare(input, gamma, residual, residual_output)
    if global_scale is None:
        global_scale = torch.ones(1, dtype=torch.float32, device=input.device)
    if global_scale.dtype != torch.float32 or global_scale.numel() != 1 or not global_scale.is_cuda:
        raise ValueError("global_scale must be a CUDA float32 tensor with one element")
    output, block_scale = _fp4_outputs(input, H, 16, output, block_scale, swizzled, torch.float8_e4m3fn)
    with _on(input.device):
        st = lib().rmsnorm_quant_nvfp4(_ptr(x), _ptr(r), _ptr(ro), _ptr(gamma), x.shape[0], H,
                                       _DT[input.dtype], float(epsilon), float(weight_offset),
                                       _ptr(global_scale), _ptr(output), _ptr(block_scale),
                                       SCALE_SWIZZLED_128x4 if swizzled else SCALE_ROW_MAJOR,
                                       _stream(input.device, stream))
    _check(st, "rmsnorm_quant_nvfp4")
    return output, block_scale, residual_output


def rmsnorm_quant_mxfp4(input, gamma, *, residual=None, residual_output=None, epsilon=1e-6,
                        weight_offset=0.0, output=None, block_scale=None, swizzled=False,
                        stream=None):
    """Residual add + RMSNorm + MXFP4 (packed E2M1, UE8M0 scale per 32 elements).

    Returns (output uint8 [..., H/2], block_scale uint8 (UE8M0 codes), residual_output)."""
    x, r, ro, residual_output, H = _prepare(input, gamma, residual, residual_output)
    output, block_scale = _fp4_outputs(input, H, 32, output, block_scale, swizzled, torch.uint8)
    with _on(input.device):
        st = lib().rmsnorm_quant_mxfp4(_ptr(x), _ptr(r), _ptr(ro), _ptr(gamma), x.shape[0], H,
                                       _DT[input.dtype], float(epsilon), float(weight_offset),
                                       _ptr(output), _ptr(block_scale),
                                       SCALE_SWIZZLED_128x4 if swizzled else SCALE_ROW_MAJOR,
                                       _stream(input.device, stream))
    _check(st, "rmsnorm_quant_mxfp4")
    return output, block_scale, residual_output


def rmsnorm_nvfp4_global_scale(input, gamma, *, residual=None, epsilon=1e-6, weight_offset=0.0,
                               out=None, stream=None):
    """gs = 448 * 6 / max |y| over the whole tensor, computed on the device (one extra read of
    input and residual). Returns a CUDA float32 tensor of one element."""
    H = input.shape[-1]
    x = _flat(input, H)
    r = None if residual is None else _flat(residual, H)
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=input.device)
    with _on(input.device):
        st = lib().rmsnorm_nvfp4_global_scale(_ptr(x), _ptr(r), _ptr(gamma), x.shape[0], H,
                                              _DT[input.dtype], float(epsilon),
                                              float(weight_offset), _ptr(out),
                                              _stream(input.device, stream))
    _check(st, "rmsnorm_nvfp4_global_scale")
    return out


# The calls below are short enough on the device that the binding's own time shows, so it checks with
# the cheapest attributes, reads the stream's handle directly and enters a device or stream context
# only where the call names another one (measured on one 8192-wide row: layernorm takes 12 us of host
# time a call this way, 22 us with a context manager and torch.device comparisons).

def _elsewhere(input, stream):
    """Whether the call needs another device or stream to be current (_queue)."""
    if not input.is_cuda:
        raise ValueError("input must be a CUDA tensor")
    if stream is not None:
        # (making a stream current makes its device current, where the call would look for another stream)
        if stream.device_index != input.get_device():
            raise ValueError("stream must be a stream of the input's device")
        return True
    return input.get_device() != torch.cuda.current_device()


@contextlib.contextmanager
def _queue(input, stream):
    """Makes the input's device and the stream current; tensors made inside belong to the stream."""
    with torch.cuda.device(input.device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _same(name, t, shape, dtype, index):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError("%s must be a contiguous %s tensor of shape %s on the input's device"
                         % (name, dtype, tuple(shape)))
    return t.data_ptr()


def _count(name, t, n, dtype, index):
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != index:
        raise ValueError("%s must be a contiguous %s tensor of %d elements on the input's device"
                         % (name, dtype, n))
    return t.data_ptr()


def _vector(name, t, n, dtype, index):
    """_count for a vector that is only read, one element at a time: (what is read, its pointer). A slice
    off 16-byte boundaries, as a program makes that splits its tokens or channels, is read from a copy."""
    p = _count(name, t, n, dtype, index)
    if p & 15:
        t = t.clone()
        p = t.data_ptr()
    return t, p


def _norm_inputs(input, gamma, beta, residual, residual_output):
    """Checks a norm's inputs; (device index, shape, rows, H, the C call's first pointers,
    residual_output)."""
    dtype, shape, index = input.dtype, input.shape, input.get_device()
    if dtype not in _DT:
        raise TypeError("input dtype must be bfloat16, float16 or float32")
    if not shape or not input.is_contiguous():
        raise ValueError("input must be a contiguous tensor of at least one dimension")
    H = shape[-1]
    rows = input.numel() // H if H else 0
    g = _count("gamma", gamma, H, dtype, index)
    b = None if beta is None else _count("beta", beta, H, dtype, index)
    r = ro = None
    if residual is not None:
        r = _same("residual", residual, shape, dtype, index)
        if residual_output is None:
            residual_output = torch.empty_like(residual)
            ro = residual_output.data_ptr()
        else:
            ro = _same("residual_output", residual_output, shape, dtype, index)
    elif residual_output is not None:
        raise ValueError("residual_output given without residual")
    return index, shape, rows, H, (input.data_ptr(), r, ro, g, b), residual_output


def layernorm(input, gamma, beta=None, *, residual=None, residual_output=None, epsilon=1e-5,
              weight_offset=0.0, output=None, stats=False, stream=None):
    """Residual add + layer norm, in the input's type; any hidden size up to MAX_HIDDEN.

    Returns (output [..., H], residual_output, mean [...], rstd [...]); mean and rstd are the fp32
    statistics layernorm_backward reads, None unless stats is true."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return layernorm(input, gamma, beta, residual=residual, residual_output=residual_output,
                             epsilon=epsilon, weight_offset=weight_offset, output=output, stats=stats)
    index, shape, rows, H, head, residual_output = _norm_inputs(input, gamma, beta, residual,
                                                                residual_output)
    if output is None:
        output = torch.empty_like(input)
        out = output.data_ptr()
    else:
        out = _same("output", output, shape, input.dtype, index)
    mean = rstd = mp = rp = None
    if stats:
        mean = torch.empty(shape[:-1], dtype=torch.float32, device=input.device)
        rstd = torch.empty_like(mean)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    _check((_lib or lib()).layernorm(*head, rows, H, _DT[input.dtype], float(epsilon),
                                     float(weight_offset), out, mp, rp, _raw_stream(index)), "layernorm")
    return output, residual_output, mean, rstd


def layernorm_backward_workspace(rows: int, hidden: int) -> int:
    """Bytes of workspace layernorm_backward needs."""
    return lib().layernorm_backward_workspace(int(rows), int(hidden))


def layernorm_backward(grad_output, input, gamma, mean, rstd, *, grad_residual=None,
                       weight_offset=0.0, grad_input=None, grad_gamma=None, grad_beta=None,
                       param_grad_dtype=None, workspace=None, stream=None):
    """The gradients of layernorm. input: what was normalised (layernorm's residual_output where it
    had a residual); grad_residual: the gradient that reaches residual_output from elsewhere.
    param_grad_dtype: type of grad_gamma and grad_beta, the input's (default) or torch.float32.
    workspace: a CUDA uint8 tensor of layernorm_backward_workspace(rows, H) bytes, allocated when
    not passed. mean and rstd may be slices off 16-byte boundaries (they are copied then); every other
    tensor starts on one.

    Returns (grad_input [..., H], grad_gamma [H], grad_beta [H])."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return layernorm_backward(grad_output, input, gamma, mean, rstd, grad_residual=grad_residual,
                                      weight_offset=weight_offset, grad_input=grad_input,
                                      grad_gamma=grad_gamma, grad_beta=grad_beta,
                                      param_grad_dtype=param_grad_dtype, workspace=workspace)
    index, shape, rows, H, (x, _, _, g, _), _ = _norm_inputs(input, gamma, None, None, None)
    dtype = input.dtype
    dy = _same("grad_output", grad_output, shape, dtype, index)
    dr = None if grad_residual is None else _same("grad_residual", grad_residual, shape, dtype, index)
    mean, mp = _vector("mean", mean, rows, torch.float32, index)
    rstd, rp = _vector("rstd", rstd, rows, torch.float32, index)
    pdt = dtype if param_grad_dtype is None else param_grad_dtype
    if pdt is not dtype and pdt is not torch.float32:
        raise TypeError("param_grad_dtype must be the input's dtype or float32")
    if grad_input is None:
        grad_input = torch.empty_like(input)
        dx = grad_input.data_ptr()
    else:
        dx = _same("grad_input", grad_input, shape, dtype, index)
    if grad_gamma is None:
        grad_gamma = torch.empty((H,), dtype=pdt, device=input.device)
        dg = grad_gamma.data_ptr()
    else:
        dg = _count("grad_gamma", grad_gamma, H, pdt, index)
    if grad_beta is None:
        grad_beta = torch.empty((H,), dtype=pdt, device=input.device)
        db = grad_beta.data_ptr()
    else:
        db = _count("grad_beta", grad_beta, H, pdt, index)
    if workspace is None:
        size = layernorm_backward_workspace(rows, H)
        workspace = torch.empty((size,), dtype=torch.uint8, device=input.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the input's device")
    else:
        size = workspace.numel() * workspace.element_size()
    _check((_lib or lib()).layernorm_backward(dy, dr, x, g, mp, rp, rows, H, _DT[dtype], float(weight_offset), dx,
                                              dg, db, _DT[pdt], workspace.data_ptr(), size,
                                              _raw_stream(index)), "layernorm_backward")
    return grad_input, grad_gamma, grad_beta


def _int8_outputs(input, index, shape, rows, output, scale_output):
    """(output, scale_output, their pointers, staged): staged is what the scales are written to, to be
    copied to scale_output after the call, where that is a slice off 16-byte boundaries; else None."""
    staged = None
    if output is None:
        output = torch.empty(shape, dtype=torch.int8, device=input.device)
        out = output.data_ptr()
    else:
        out = _same("output", output, shape, torch.int8, index)
    if scale_output is None:
        scale_output = torch.empty(shape[:-1], dtype=torch.float32, device=input.device)
        scale = scale_output.data_ptr()
    else:
        scale = _count("scale_output", scale_output, rows, torch.float32, index)
        if scale & 15:
            staged = torch.empty_like(scale_output)
            scale = staged.data_ptr()
    return output, scale_output, out, scale, staged


def layernorm_quant_int8(input, gamma, beta=None, *, residual=None, residual_output=None,
                         epsilon=1e-5, weight_offset=0.0, output=None, scale_output=None, stream=None):
    """Residual add + layer norm + int8 codes with one fp32 scale per row (max |y| / 127). scale_output may be
    a slice off 16-byte boundaries (it is copied to then); every other tensor starts on one.

    Returns (output int8 [..., H], scale_output float32 [...], residual_output)."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return layernorm_quant_int8(input, gamma, beta, residual=residual,
                                        residual_output=residual_output, epsilon=epsilon,
                                        weight_offset=weight_offset, output=output,
                                        scale_output=scale_output)
    index, shape, rows, H, head, residual_output = _norm_inputs(input, gamma, beta, residual,
                                                                residual_output)
    output, scale_output, out, scale, staged = _int8_outputs(input, index, shape, rows, output, scale_output)
    _check((_lib or lib()).layernorm_quant_int8(*head, rows, H, _DT[input.dtype], float(epsilon),
                                                float(weight_offset), out, scale, _raw_stream(index)),
           "layernorm_quant_int8")
    if staged is not None:
        scale_output.copy_(staged)
    return output, scale_output, residual_output


def rmsnorm_quant_int8(input, gamma, *, residual=None, residual_output=None, epsilon=1e-6,
                       weight_offset=0.0, output=None, scale_output=None, stream=None):
    """Residual add + RMSNorm + int8 codes with one fp32 scale per row (max |y| / 127). scale_output may be a
    slice off 16-byte boundaries (it is copied to then); every other tensor starts on one.

    Returns (output int8 [..., H], scale_output float32 [...], residual_output)."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return rmsnorm_quant_int8(input, gamma, residual=residual, residual_output=residual_output,
                                      epsilon=epsilon, weight_offset=weight_offset, output=output,
                                      scale_output=scale_output)
    index, shape, rows, H, head, residual_output = _norm_inputs(input, gamma, None, residual,
                                                                residual_output)
    output, scale_output, out, scale, staged = _int8_outputs(input, index, shape, rows, output, scale_output)
    _check((_lib or lib()).rmsnorm_quant_int8(*head[:4], rows, H, _DT[input.dtype], float(epsilon),
                                              float(weight_offset), out, scale, _raw_stream(index)),
           "rmsnorm_quant_int8")
    if staged is not None:
        scale_output.copy_(staged)
    return output, scale_output, residual_output


def matmul_int8(input, input_scale, weight, weight_scale, *, bias=None, out_dtype=torch.bfloat16,
                output=None, stream=None):
    """(input @ weight.T) * input_scale * weight_scale + bias on int8 codes, integer sums exact.

    input int8 [..., K] with one fp32 scale per row, weight int8 [N, K] with one fp32 scale per
    output channel, bias [N] of out_dtype. K must be a multiple of 16. The codes and the output start on
    16-byte boundaries; scales and bias may be slices that do not (they are copied then).

    Returns output [..., N] of out_dtype."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return matmul_int8(input, input_scale, weight, weight_scale, bias=bias, out_dtype=out_dtype,
                               output=output)
    if input.dtype is not torch.int8 or weight.dtype is not torch.int8:
        raise TypeError("input and weight must be int8")
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be bfloat16, float16 or float32")
    index, shape = input.get_device(), input.shape
    if not shape or not input.is_contiguous():
        raise ValueError("input must be a contiguous tensor of at least one dimension")
    K = shape[-1]
    M = input.numel() // K if K else 0
    if weight.dim() != 2:
        raise ValueError("weight must have shape (N, %d)" % K)
    N = weight.shape[0]
    w = _same("weight", weight, (N, K), torch.int8, index)
    input_scale, sa = _vector("input_scale", input_scale, M, torch.float32, index)
    weight_scale, sw = _vector("weight_scale", weight_scale, N, torch.float32, index)
    bias, b = (None, None) if bias is None else _vector("bias", bias, N, out_dtype, index)
    oshape = shape[:-1] + (N,)
    if output is None:
        output = torch.empty(oshape, dtype=out_dtype, device=input.device)
        out = output.data_ptr()
    else:
        out = _same("output", output, oshape, out_dtype, index)
    _check((_lib or lib()).matmul_int8(input.data_ptr(), sa, w, sw, b, M, N, K, out, _DT[out_dtype],
                                       _raw_stream(index)), "matmul_int8")
    return output


def _one(name, t, index):
    """Pointer to a device scalar, None for none."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.numel() != 1 or t.get_device() != index:
        raise ValueError("%s must be a float32 tensor of one element on the input's device" % name)
    return t.data_ptr()


def nvfp4_global_scale(input, *, out=None, workspace=None, stream=None):
    """gs = 448 * 6 / max |input|, computed on the device (quant_nvfp4's global_scale). workspace: a CUDA uint8
    tensor of nvfp4_global_scale_workspace(input.numel()) bytes, allocated when not passed.

    Returns a CUDA float32 tensor of one element: 1 for zeros, NaN where the input has a NaN, 0 (no scale to quantise by)
    where it has an infinity."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return nvfp4_global_scale(input, out=out, workspace=workspace)
    if input.dtype not in _DT:
        raise TypeError("input dtype must be bfloat16, float16 or float32")
    if not input.is_contiguous():
        raise ValueError("input must be a contiguous tensor")
    index, count = input.get_device(), input.numel()
    if out is None:
        out = torch.empty((1,), dtype=torch.float32, device=input.device)
        o = out.data_ptr()
    else:
        o = _one("out", out, index)
    ws = None
    if workspace is None:
        size = (_lib or lib()).nvfp4_global_scale_workspace(count)
        if size:
            workspace = torch.empty((size,), dtype=torch.uint8, device=input.device)
            ws = workspace.data_ptr()
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the input's device")
    else:
        size, ws = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    _check((_lib or lib()).nvfp4_global_scale(input.data_ptr(), count, _DT[input.dtype], o, ws, size, _raw_stream(index)),
           "nvfp4_global_scale")
    return out


def nvfp4_global_scale_workspace(count: int) -> int:
    """Bytes of workspace nvfp4_global_scale needs."""
    return lib().nvfp4_global_scale_workspace(int(count))


_BYTES = {torch.uint8, torch.int8, torch.float8_e4m3fn, getattr(torch, "float8_e8m0fnu", torch.uint8)}


def _bytes(name, t, n, index):
    if t.dtype not in _BYTES or t.numel() != n or not t.is_contiguous() or t.get_device() != index:
        raise ValueError("%s must be a contiguous tensor of %d bytes on the input's device" % (name, n))
    return t.data_ptr()


def _quant_fp4(input, block, scale_dtype, output, block_scale, swizzled):
    """Checks a 4-bit quantisation's tensors; (device index, rows, H, output, block_scale, their pointers)."""
    if input.dtype not in _DT:
        raise TypeError("input dtype must be bfloat16, float16 or float32")
    shape, index = input.shape, input.get_device()
    if not shape or not input.is_contiguous():
        raise ValueError("input must be a contiguous tensor of at least one dimension")
    H = shape[-1]
    if H == 0 or H % block:
        raise ValueError("the last dimension must be a multiple of %d" % block)
    rows = input.numel() // H
    if output is None:
        output = torch.empty(shape[:-1] + (H // 2,), dtype=torch.uint8, device=input.device)
        out = output.data_ptr()
    else:
        out = _same("output", output, shape[:-1] + (H // 2,), torch.uint8, index)
    if block_scale is None:
        sshape = (swizzled_scale_numel(rows, H, block),) if swizzled else shape[:-1] + (H // block,)
        block_scale = torch.empty(sshape, dtype=scale_dtype, device=input.device)
        scale = block_scale.data_ptr()
    else:
        scale = _bytes("block_scale", block_scale, swizzled_scale_numel(rows, H, block) if swizzled else rows * (H // block),
                       index)
    return index, rows, H, output, block_scale, out, scale


def quant_nvfp4(input, *, global_scale=None, output=None, block_scale=None, swizzled=False, stream=None):
    """NVFP4 (packed E2M1, E4M3 scale per 16 elements) of a tensor that comes from no norm. global_scale: a CUDA
    float32 tensor of one element, read on the device (nvfp4_global_scale's; default 1.0).

    Returns (output uint8 [..., H/2], block_scale float8_e4m3fn)."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return quant_nvfp4(input, global_scale=global_scale, output=output, block_scale=block_scale, swizzled=swizzled)
    index, rows, H, output, block_scale, out, scale = _quant_fp4(input, 16, torch.float8_e4m3fn, output, block_scale, swizzled)
    gs = _one("global_scale", global_scale, index)
    _check((_lib or lib()).quant_nvfp4(input.data_ptr(), rows, H, _DT[input.dtype], gs, out, scale,
                                       SCALE_SWIZZLED_128x4 if swizzled else SCALE_ROW_MAJOR, _raw_stream(index)),
           "quant_nvfp4")
    return output, block_scale


def quant_mxfp4(input, *, output=None, block_scale=None, swizzled=False, stream=None):
    """MXFP4 (packed E2M1, UE8M0 scale per 32 elements) of a tensor that comes from no norm. Blocks whose elements are at most
    6 * 2^-127 become zeros.

    Returns (output uint8 [..., H/2], block_scale uint8 (UE8M0 codes))."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return quant_mxfp4(input, output=output, block_scale=block_scale, swizzled=swizzled)
    index, rows, H, output, block_scale, out, scale = _quant_fp4(input, 32, torch.uint8, output, block_scale, swizzled)
    _check((_lib or lib()).quant_mxfp4(input.data_ptr(), rows, H, _DT[input.dtype], out, scale,
                                       SCALE_SWIZZLED_128x4 if swizzled else SCALE_ROW_MAJOR, _raw_stream(index)),
           "quant_mxfp4")
    return output, block_scale


def _matmul_fp4(input, input_scale, weight, weight_scale, block, bias, out_dtype, output):
    """Checks a 4-bit product's tensors; (device index, M, N, K, pointers of the four operands, the bias that is read,
    its pointer, output, its pointer)."""
    u8 = torch.uint8
    if input.dtype is not u8 or weight.dtype is not u8:
        raise TypeError("input and weight must be uint8 (two codes per byte)")
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be bfloat16, float16 or float32")
    index, shape, wshape = input.get_device(), input.shape, weight.shape
    if not shape or not input.is_contiguous():
        raise ValueError("input must be a contiguous tensor of at least one dimension")
    half = shape[-1]
    if len(wshape) != 2 or wshape[1] != half or not weight.is_contiguous() or weight.get_device() != index:
        raise ValueError("weight must be a contiguous uint8 tensor of shape (N, %d) on the input's device" % half)
    N, K = wshape[0], 2 * half
    if len(shape) == 2:
        M = shape[0]
        oshape = (M, N)
    else:
        M = input.numel() // half if half else 0
        oshape = shape[:-1] + (N,)
    row = (K // block + 3) // 4 * 512                     # bytes of 128 rows' scales
    sa = _bytes("input_scale", input_scale, (M + 127) // 128 * row, index)
    sw = _bytes("weight_scale", weight_scale, (N + 127) // 128 * row, index)
    b = None
    if bias is not None:
        bias, b = _vector("bias", bias, N, out_dtype, index)
    if output is None:
        output = torch.empty(oshape, dtype=out_dtype, device=input.device)
        out = output.data_ptr()
    else:
        out = _same("output", output, oshape, out_dtype, index)
    return index, M, N, K, (input.data_ptr(), sa, weight.data_ptr(), sw), bias, b, output, out


def matmul_nvfp4(input, input_scale, weight, weight_scale, *, input_global_scale=None, weight_global_scale=None, bias=None,
                 out_dtype=torch.bfloat16, output=None, stream=None):
    """input @ weight.T / (input_global_scale * weight_global_scale) + bias on NVFP4 codes.

    input uint8 [..., K/2] and weight uint8 [N, K/2] as rmsnorm_quant_nvfp4 and quant_nvfp4 give them with
    swizzled=True, with their block scales; the global scales they were formed with (CUDA float32 tensors of one
    element, read on the device; default 1.0); bias [N] of out_dtype. K must be a multiple of 32. Tensors start on
    16-byte boundaries; bias may be a slice that does not (it is copied then).

    Returns output [..., N] of out_dtype."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return matmul_nvfp4(input, input_scale, weight, weight_scale, input_global_scale=input_global_scale,
                                weight_global_scale=weight_global_scale, bias=bias, out_dtype=out_dtype, output=output)
    index, M, N, K, (a, sa, w, sw), bias, b, output, out = _matmul_fp4(input, input_scale, weight, weight_scale, 16, bias,
                                                                       out_dtype, output)
    ga = _one("input_global_scale", input_global_scale, index)
    gw = _one("weight_global_scale", weight_global_scale, index)
    _check((_lib or lib()).matmul_nvfp4(a, sa, ga, w, sw, gw, b, M, N, K, out, _DT[out_dtype], _raw_stream(index)),
           "matmul_nvfp4")
    return output


def matmul_mxfp4(input, input_scale, weight, weight_scale, *, bias=None, out_dtype=torch.bfloat16, output=None, stream=None):
    """input @ weight.T + bias on MXFP4 codes.

    input uint8 [..., K/2] and weight uint8 [N, K/2] as rmsnorm_quant_mxfp4 and quant_mxfp4 give them with
    swizzled=True, with their block scales; bias [N] of out_dtype. K must be a multiple of 32. Tensors start on 16-byte
    boundaries; bias may be a slice that does not (it is copied then).

    Returns output [..., N] of out_dtype."""
    if _elsewhere(input, stream):
        with _queue(input, stream):
            return matmul_mxfp4(input, input_scale, weight, weight_scale, bias=bias, out_dtype=out_dtype, output=output)
    index, M, N, K, (a, sa, w, sw), bias, b, output, out = _matmul_fp4(input, input_scale, weight, weight_scale, 32, bias,
                                                                       out_dtype, output)
    _check((_lib or lib()).matmul_mxfp4(a, sa, w, sw, b, M, N, K, out, _DT[out_dtype], _raw_stream(index)), "matmul_mxfp4")
    return output


def _heads(name, t, shape, dtype, index):
    """The C view of [..., heads, D], whose leading dimensions count as tokens."""
    stride = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or stride[-1] != 1:
        raise ValueError("%s must be a %s tensor of shape %s on the input's device, its last dimension contiguous"
                         % (name, dtype, tuple(shape)))
    if len(shape) != 3:
        try:
            t = t.view((-1 if t.numel() else 0,) + tuple(shape[-2:]))
        except RuntimeError:
            raise ValueError("%s: its leading dimensions must lie behind each other" % name) from None
        shape, stride = t.shape, t.stride()
    tokens, heads, _ = shape
    return HEADS.pack(t.data_ptr(), stride[0] if tokens > 1 else 0, stride[1] if heads > 1 else 0, heads)


def _rope(query, key, query_gamma, key_gamma, cos, sin, positions, sections, interleaved):
    """Checks the inputs of rmsnorm_rope; (device index, dtype, tokens, D, query, key, gammas, rotation)."""
    dtype, index, shape, kshape = query.dtype, query.get_device(), query.shape, key.shape
    if dtype not in _DT:
        raise TypeError("query dtype must be bfloat16, float16 or float32")
    lead, D = shape[:-2], shape[-1] if shape else 0
    if len(shape) < 3 or len(kshape) != len(shape) or kshape[:-2] != lead or kshape[-1] != D:
        raise ValueError("query and key must have shapes [..., heads, D] with the same tokens and D")
    q = _heads("query", query, shape, dtype, index)
    k = _heads("key", key, kshape, dtype, index)
    gq = _count("query_gamma", query_gamma, D, dtype, index)
    gk = _count("key_gamma", key_gamma, D, dtype, index)
    table = cos.shape
    if len(table) != 2:
        raise ValueError("cos must have shape (positions, rotated / 2)")
    c = _same("cos", cos, table, torch.float32, index)
    s = _same("sin", sin, table, torch.float32, index)
    if sections is None:
        axes, parts, want = 1, (0, 0, 0, 0), lead
    else:
        axes, want = len(sections), (len(sections),) + tuple(lead)
        if not 1 <= axes <= 4:
            raise ValueError("sections must have 1 to 4 entries")
        if sum(sections) != table[1] or min(sections) < 0:
            raise ValueError("sections must not be negative, and add up to rotated / 2")
        parts = tuple(sections) + (0,) * (4 - axes)
    pdtype = positions.dtype
    if pdtype is not torch.int64 and pdtype is not torch.int32:
        raise TypeError("positions must be int32 or int64")
    at = _same("positions", positions, want, pdtype, index)
    r = ROTATION.pack(c, s, at, table[0], 64 if pdtype is torch.int64 else 32, 2 * table[1], 1 if interleaved else 0, axes, *parts)
    return index, dtype, lead.numel(), D, q, k, gq, gk, r


def _like(name, t, of, dtype, index):
    """(tensor, its C view) of an output like `of`; a contiguous one where none is given."""
    if t is not None:
        return t, _heads(name, t, of.shape, dtype, index)
    shape = of.shape
    t = torch.empty(shape, dtype=dtype, device=of.device)
    heads, D = shape[-2:]
    return t, HEADS.pack(t.data_ptr(), heads * D, D, heads)


def rmsnorm_rope(query, key, query_gamma, key_gamma, cos, sin, positions, *, sections=None, interleaved=False, epsilon=1e-6,
                 weight_offset=0.0, query_output=None, key_output=None, stream=None):
    """RMS norm of every head's query and key, then the rotation by the token's position.

    query [..., heads, D] and key [..., kv_heads, D], the last dimension contiguous, the heads and the tokens with any stride
    each (slices of a projection's output; [heads, tokens, D] transposed); several leading dimensions must lie behind each other
    as one does, which a transposed batch of [batch, heads, tokens, D] does not: ValueError. gammas [D]; cos and sin float32 [places, R / 2], R <= D elements of a head being rotated;
    positions int32 or int64 [...], or [axes, ...] with sections, which says how many of the R / 2 frequencies go by
    each axis. interleaved: neighbours are rotated together, instead of the halves of the R elements. A position outside
    the table gives NaN. query_output and key_output may be query and key themselves.

    Returns (query_output [..., heads, D], key_output [..., kv_heads, D])."""
    if _elsewhere(query, stream):
        with _queue(query, stream):
            return rmsnorm_rope(query, key, query_gamma, key_gamma, cos, sin, positions, sections=sections,
                                interleaved=interleaved, epsilon=epsilon, weight_offset=weight_offset,
                                query_output=query_output, key_output=key_output)
    index, dtype, tokens, D, q, k, gq, gk, r = _rope(query, key, query_gamma, key_gamma, cos, sin, positions, sections,
                                                     interleaved)
    query_output, qo = _like("query_output", query_output, query, dtype, index)
    key_output, ko = _like("key_output", key_output, key, dtype, index)
    _check((_lib or lib()).rmsnorm_rope(q, k, gq, gk, r, tokens, D, _DT[dtype], float(epsilon), float(weight_offset),
                                        qo, ko, _raw_stream(index)), "rmsnorm_rope")
    return query_output, key_output


def rmsnorm_rope_backward_workspace(tokens: int, dim: int) -> int:
    """Bytes of workspace rmsnorm_rope_backward needs."""
    return lib().rmsnorm_rope_backward_workspace(int(tokens), int(dim))


def rmsnorm_rope_backward(grad_query, grad_key, query, key, query_gamma, key_gamma, cos, sin, positions, *, sections=None,
                          interleaved=False, epsilon=1e-6, weight_offset=0.0, query_grad=None, key_grad=None,
                          query_gamma_grad=None, key_gamma_grad=None, param_grad_dtype=None, workspace=None, stream=None):
    """The gradients of rmsnorm_rope. grad_query, grad_key: the gradients of its outputs; query, key and the rest: its
    inputs. param_grad_dtype: type of the gammas' gradients, the input's (default) or torch.float32. query_grad and
    key_grad may be grad_query and grad_key themselves. A position outside the table gives NaN in its token's gradients and
    in the gammas' rotated elements (for padding: a place in the table, and gradients of 0). workspace: a CUDA uint8 tensor of
    rmsnorm_rope_backward_workspace(tokens, D) bytes, allocated when not passed.

    Returns (query_grad [..., heads, D], key_grad [..., kv_heads, D], query_gamma_grad [D], key_gamma_grad [D])."""
    if _elsewhere(query, stream):
        with _queue(query, stream):
            return rmsnorm_rope_backward(grad_query, grad_key, query, key, query_gamma, key_gamma, cos, sin, positions,
                                         sections=sections, interleaved=interleaved, epsilon=epsilon,
                                         weight_offset=weight_offset, query_grad=query_grad, key_grad=key_grad,
                                         query_gamma_grad=query_gamma_grad, key_gamma_grad=key_gamma_grad,
                                         param_grad_dtype=param_grad_dtype, workspace=workspace)
    index, dtype, tokens, D, q, k, gq, gk, r = _rope(query, key, query_gamma, key_gamma, cos, sin, positions, sections,
                                                     interleaved)
    dq = _heads("grad_query", grad_query, query.shape, dtype, index)
    dk = _heads("grad_key", grad_key, key.shape, dtype, index)
    pdt = dtype if param_grad_dtype is None else param_grad_dtype
    if pdt is not dtype and pdt is not torch.float32:
        raise TypeError("param_grad_dtype must be the input's dtype or float32")
    query_grad, qo = _like("query_grad", query_grad, query, dtype, index)
    key_grad, ko = _like("key_grad", key_grad, key, dtype, index)
    if query_gamma_grad is None:
        query_gamma_grad = torch.empty((D,), dtype=pdt, device=query.device)
        pq = query_gamma_grad.data_ptr()
    else:
        pq = _count("query_gamma_grad", query_gamma_grad, D, pdt, index)
    if key_gamma_grad is None:
        key_gamma_grad = torch.empty((D,), dtype=pdt, device=query.device)
        pk = key_gamma_grad.data_ptr()
    else:
        pk = _count("key_gamma_grad", key_gamma_grad, D, pdt, index)
    if workspace is None:
        size = rmsnorm_rope_backward_workspace(tokens, D)
        workspace = torch.empty((size,), dtype=torch.uint8, device=query.device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the input's device")
    else:
        size = workspace.numel() * workspace.element_size()
    _check((_lib or lib()).rmsnorm_rope_backward(dq, dk, q, k, gq, gk, r, tokens, D, _DT[dtype], float(epsilon),
                                                 float(weight_offset), qo, ko, pq, pk, _DT[pdt], workspace.data_ptr(), size, _raw_stream(index)),
           "rmsnorm_rope_backward")
    return query_grad, key_grad, query_gamma_grad, key_gamma_grad


def rmsq_device_status() -> int:
    return lib().rmsq_device_status()


def rmsq_set_schedule(schedule: int) -> int:
    return lib().rmsq_set_schedule(int(schedule))


def rmsq_set_tuning(stages: int = 0, ctas_per_sm: int = 0, vectors_per_thread: int = 0):
    _check(lib().rmsq_set_tuning(stages, ctas_per_sm, vectors_per_thread), "rmsq_set_tuning")


def rmsq_set_cluster_size(ctas_per_cluster: int = 0):
    _check(lib().rmsq_set_cluster_size(int(ctas_per_cluster)), "rmsq_set_cluster_size")


def rmsq_set_row_warps(warps_per_cta: int = 0):
    _check(lib().rmsq_set_row_warps(int(warps_per_cta)), "rmsq_set_row_warps")


def rmsq_set_dynamic_rows(enable: bool) -> bool:
    return bool(lib().rmsq_set_dynamic_rows(int(bool(enable))))


def rmsq_set_pdl(enable: bool) -> bool:
    return bool(lib().rmsq_set_pdl(int(bool(enable))))


def rmsq_set_wait_timeout_ns(ns: int):
    lib().rmsq_set_wait_timeout_ns(int(ns))


def rmsq_selftest_wait_timeout(timeout_ns: int, stream=None):
    dev = torch.device("cuda", torch.cuda.current_device())
    _check(lib().rmsq_selftest_wait_timeout(int(timeout_ns), _stream(dev, stream)),
           "rmsq_selftest_wait_timeout")


def rmsq_debug_convert(fmt: int, values: torch.Tensor, stream=None) -> torch.Tensor:
    """Convert fp32 values on the device with the kernels' conversion instructions.
    fmt 0: E4M3 codes; fmt 1: E2M1 codes (low nibble). Returns uint8 codes."""
    out = torch.empty(values.shape, dtype=torch.uint8, device=values.device)
    with torch.cuda.device(values.device):
        _check(lib().rmsq_debug_convert(int(fmt), _ptr(values), _ptr(out), values.numel(),
                                        _stream(values.device, stream)), "rmsq_debug_convert")
    return out


def rmsq_launch_count() -> int:
    return lib().rmsq_launch_count()


def rmsq_plan(mode: str, dtype, hidden: int, residual: bool = False, weight_offset: float = 0.0,
              smem=GB300_SMEM) -> dict:
    """The launch plan the entry point of `mode` ("fp8", "nvfp4", "mxfp4", "global_scale") would
    choose now for rows of `hidden` elements, tuning settings included (rmsq_plan in
    include/rmsq.h). smem: the (opt-in per CTA, per SM, reserved per CTA) shared-memory limits in
    bytes, GB300's by default; None takes the current device's."""
    dt = _DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    optin, per_sm, reserved = smem if smem is not None else (0, 0, 0)
    info = PlanInfo()
    _check(lib().rmsq_plan(MODES[mode], dt, int(bool(residual)), float(weight_offset), int(hidden),
                           optin, per_sm, reserved, ctypes.byref(info)), "rmsq_plan")
    return {n: getattr(info, n) for n, _ in PlanInfo._fields_}
