"""The 4-bit products and the per-head norm with rotation as a user's program calls them, with plain forms.

matmul                matmul_nvfp4 or matmul_mxfp4: out = (a * a_scale) @ (w * w_scale)^T + bias, a and w
                      E2M1 codes with one scale per 16 (E4M3 under a global scale) or 32 (UE8M0) elements
quant_matmul          a projection whose input comes from no norm: quant_nvfp4 (its global scale from
                      nvfp4_global_scale) or quant_mxfp4, then the product
rmsnorm_rope          RMS norm of every head's query and key, then the rotation by its position
rmsnorm_rope_backward the gradients of the queries, the keys and both gammas
qkv                   rmsnorm_quant_nvfp4, matmul_nvfp4 and rmsnorm_rope: from a residual stream to the
                      queries, keys and values of an attention

Where `own` is false, run() computes these with elementary torch operations in 32 bits (in 64 what is
about to be rounded to 4 or 8 bits); where it is true, with the package's calls. Both take what prepare()
gives.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = {"nvfp4": 16, "mxfp4": 32}
EPS = 1e-6
TABLE = 65536                    # positions of the rotation's table

# Ranges that draw() covers: no drawn case costs more than the largest listed one of its operator.
MOST_PRODUCTS = 8192 ** 3
MOST_QUANTISED = 16384 * 8192
MOST_ROTATED = 16384 * 40 * 128


def listed():
    return [
        # one decoded token through a projection
        {"name": "mm_token", "op": "matmul", "format": "nvfp4", "m": 1, "n": 7168, "k": 8192, "out": "bf16",
         "bias": False},
        # a decode batch of ragged size; neither width is a whole number of tiles
        {"name": "mm_batch", "op": "matmul", "format": "mxfp4", "m": 100, "n": 5001, "k": 5152, "out": "fp16",
         "bias": True},
        # a long prompt through a square projection
        {"name": "mm_prompt", "op": "matmul", "format": "nvfp4", "m": 8192, "n": 8192, "k": 8192, "out": "bf16",
         "bias": False},
        # a decode batch's attention output, quantised and projected
        {"name": "quant_mm_batch", "op": "quant_matmul", "format": "mxfp4", "m": 48, "n": 4096, "k": 4096,
         "dtype": "fp16", "bias": False},
        # a large batch of prompts into a narrow projection, most of whose time goes to the quantisation
        {"name": "quant_mm_narrow", "op": "quant_matmul", "format": "nvfp4", "m": 16384, "n": 512, "k": 8192,
         "dtype": "bf16", "bias": True},
        # one decoded token's queries and keys
        {"name": "rope_token", "op": "rmsnorm_rope", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotated": 128, "axes": 1, "interleaved": False, "dtype": "bf16", "packed": True},
        # the queries and keys of a batch of prompts, inside the projection's output
        {"name": "rope_prompt", "op": "rmsnorm_rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotated": 128, "axes": 1, "interleaved": False, "dtype": "bf16", "packed": True},
        # images and text in 32 bits: time, height and width, neighbours rotated together, part of an odd head
        {"name": "rope_axes", "op": "rmsnorm_rope", "tokens": 4099, "heads": 12, "kv_heads": 2, "dim": 80,
         "rotated": 60, "axes": 3, "interleaved": True, "dtype": "fp32", "packed": False},
        # a fine-tuning step on one short sequence
        {"name": "rope_grad_short", "op": "rmsnorm_rope_backward", "tokens": 70, "heads": 16, "kv_heads": 16,
         "dim": 64, "rotated": 64, "axes": 1, "interleaved": True, "dtype": "fp16", "packed": False},
        # a training step on a full batch
        {"name": "rope_grad_step", "op": "rmsnorm_rope_backward", "tokens": 16384, "heads": 32, "kv_heads": 8,
         "dim": 128, "rotated": 128, "axes": 1, "interleaved": False, "dtype": "bf16", "packed": True},
        # a decode batch from its residual stream to queries, keys and values
        {"name": "qkv_batch", "op": "qkv", "tokens": 16, "hidden": 4096, "heads": 32, "kv_heads": 8, "dim": 128,
         "dtype": "bf16"},
        # the same for a prompt
        {"name": "qkv_prompt", "op": "qkv", "tokens": 4096, "hidden": 8192, "heads": 64, "kv_heads": 8,
         "dim": 128, "dtype": "bf16"},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["matmul", "quant_matmul", "rmsnorm_rope", "rmsnorm_rope_backward", "qkv"])
    if op in ("matmul", "quant_matmul"):
        k = 32 * _log(rng, 4, 512)
        n = _log(rng, 64, 16384)
        m = _log(rng, 1, min(8192, MOST_PRODUCTS // (n * k)))
        case = {"op": op, "format": rng.choice(["nvfp4", "mxfp4"]), "m": m, "n": n, "k": k,
                "bias": rng.random() < 0.5}
        case["out" if op == "matmul" else "dtype"] = rng.choice(["bf16", "fp16", "fp32"])
        return case
    if op == "qkv":
        kv = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 4096), "hidden": 128 * _log(rng, 4, 64),
                "heads": kv * rng.choice([1, 4, 8]), "kv_heads": kv, "dim": rng.choice([64, 128, 256]),
                "dtype": rng.choice(["bf16", "fp16"])}
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    dim = rng.choice([64, 80, 96, 128, 192, 256, 2 * _log(rng, 8, 128)])
    rotated = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
    kv = rng.choice([1, 2, 3, 4, 8, 16])
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    cost = MOST_ROTATED // ((heads + kv) * dim * (2 if dtype == "fp32" else 1))
    return {"op": op, "tokens": _log(rng, 1, min(65536, cost)), "heads": heads, "kv_heads": kv, "dim": dim,
            "rotated": rotated, "axes": min(rng.choice([1, 1, 3]), rotated // 2), "interleaved": rng.random() < 0.5,
            "dtype": dtype, "packed": rng.random() < 0.5}


# -- 4-bit formats: codes two to a byte (element 2k in the low nibble), scales in tiles of 128 rows x 4 ------

_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e2m1(t):
    """Nearest E2M1 code of each value, ties to the even code: steps of 1/2 below 2, of 1 below 4, of 2 above."""
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    value = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.where(value < 2, 2 * value, torch.where(value < 4, value + 2, value / 2 + 4))
    return code.to(torch.uint8) + 8 * torch.signbit(t).to(torch.uint8)


def _pack(code):
    pair = code.reshape(code.shape[0], -1, 2)
    return pair[:, :, 0] + 16 * pair[:, :, 1]


def _e2m1_values(packed):
    table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=packed.device)
    code = torch.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1)
    return table[code.int()]


def _tiled(scale):
    """Scale bytes [rows, blocks] in tiles of 128 rows x 4 scales."""
    rows, blocks = scale.shape
    full = torch.zeros(((rows + 127) // 128 * 128, (blocks + 3) // 4 * 4), dtype=torch.uint8, device=scale.device)
    full[:rows, :blocks] = scale
    return full.reshape(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untiled(tiles, rows, blocks):
    wide = (blocks + 3) // 4
    full = tiles.reshape(-1, wide, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * wide)
    return full[:rows, :blocks]


def _scale_values(byte, fmt):
    if fmt == "nvfp4":
        return byte.contiguous().view(torch.float8_e4m3fn).float()
    return torch.exp2(byte.float() - 127.0)


def _global_scale(x):
    return (448.0 * 6.0 / x.abs().amax().float()).reshape(1)


def _quantise(x, fmt, gs):
    """Codes and scale bytes (row-major) of x; what is rounded to few bits is formed in 64."""
    rows, block = x.shape[0], BLOCK[fmt]
    amax = x.float().reshape(rows, -1, block).abs().amax(-1)
    if fmt == "nvfp4":
        scale = (amax.double() * gs.double() / 6.0).clamp(max=448.0).float().to(torch.float8_e4m3fn)
        byte, each = scale.view(torch.uint8), scale.double()
        factor = torch.where(each > 0, gs.double() / each, 0.0)
    else:
        mantissa, exponent = torch.frexp(amax)
        e = exponent - 3 + (mantissa > 0.75) + 127
        byte = torch.where(amax > 0, e, 0).clamp(0, 255).to(torch.uint8)
        factor = torch.where(byte > 0, torch.exp2(127.0 - byte.double()), 0.0)
    t = x.reshape(rows, -1, block).double() * factor[:, :, None]
    return _pack(_e2m1(t.reshape(rows, -1))), byte


def _dequantise(packed, tiles, fmt):
    rows, k, block = packed.shape[0], packed.shape[1] * 2, BLOCK[fmt]
    scale = _scale_values(_untiled(tiles.view(torch.uint8), rows, k // block), fmt)
    return (_e2m1_values(packed).reshape(rows, -1, block) * scale[:, :, None]).reshape(rows, k)


# -- inputs ----------------------------------------------------------------------------------------------

def _normal(g, shape, mean, std, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _activations(g, m, k, dtype):
    """Rows of differing size with a few channels that stand out."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x *= 0.5 + torch.rand((m, 1), generator=g, device="cuda")
    return (x * torch.where(torch.rand((1, k), generator=g, device="cuda") < 0.005, 8.0, 1.0)).to(dtype)


def _operand(s, name, x, fmt):
    """x as codes, tiled scales and (NVFP4) a global scale."""
    gs = _global_scale(x) if fmt == "nvfp4" else None
    s[name], byte = _quantise(x, fmt, gs)
    tiles = _tiled(byte)
    s[name + "_scale"] = tiles.view(torch.float8_e4m3fn) if fmt == "nvfp4" else tiles
    s[name + "_global"] = gs


def _sections(axes, half):
    """How many of the rotation's frequencies go by each axis; None for one axis."""
    if axes == 1:
        return None
    first = max(1, half // 4)
    rest = (half - first) // (axes - 1)
    return (first,) + (rest,) * (axes - 2) + (half - first - rest * (axes - 2),)


def _rotation(s, g, tokens, half, axes):
    """Tables of cosines and sines by position, and the positions of tokens of packed sequences."""
    angle = torch.arange(TABLE, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
        500000.0, -torch.arange(half, device="cuda", dtype=torch.float64) / half)
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    start = torch.randint(0, TABLE - tokens % TABLE, (axes, 1), generator=g, device="cuda")
    place = (start + torch.arange(tokens, device="cuda")) % TABLE
    if axes > 1:                                     # height and width run within an image
        place[1:] = torch.randint(0, 64, (axes - 1, tokens), generator=g, device="cuda")
    s["positions"] = place if axes > 1 else place[0]
    s["sections"] = _sections(axes, half)


def _heads(s, case, g, name, dtype):
    """Queries and keys of every token, behind each other in a projection's output or by themselves."""
    t, h, kv, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    if case["packed"]:
        both = _normal(g, (t, (h + 2 * kv) * d), 0.1, 1.0, dtype)
        s[name + "q"], s[name + "k"] = _split(both, h, kv, d)[:2]
    else:
        s[name + "q"] = _normal(g, (t, h, d), 0.1, 1.0, dtype)
        s[name + "k"] = _normal(g, (t, kv, d), 0.1, 1.0, dtype)


def _split(qkv, h, kv, d):
    return (qkv[:, :h * d].unflatten(1, (h, d)), qkv[:, h * d:(h + kv) * d].unflatten(1, (kv, d)),
            qkv[:, (h + kv) * d:].unflatten(1, (kv, d)))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op in ("matmul", "quant_matmul"):
        m, n, k, fmt = case["m"], case["n"], case["k"], case["format"]
        _operand(s, "w", _normal(g, (n, k), 0.0, 0.02), fmt)
        if op == "matmul":
            _operand(s, "a", _activations(g, m, k, torch.bfloat16), fmt)
        else:
            s["x"] = _activations(g, m, k, DTYPES[case["dtype"]])
        s["bias"] = _normal(g, (n,), 0.0, 0.1, DTYPES[case["out" if op == "matmul" else "dtype"]]) if case["bias"] else None
        return s
    t, dt, dim = case["tokens"], DTYPES[case["dtype"]], case["dim"]
    s["gq"], s["gk"] = _normal(g, (dim,), 1.0, 0.1, dt), _normal(g, (dim,), 1.0, 0.1, dt)
    if op == "qkv":
        hidden, width = case["hidden"], (case["heads"] + 2 * case["kv_heads"]) * dim
        s["x"], s["residual"] = _normal(g, (t, hidden), 0.0, 1.0, dt), _normal(g, (t, hidden), 0.0, 2.0, dt)
        s["gamma"] = _normal(g, (hidden,), 1.0, 0.1, dt)
        _operand(s, "w", _normal(g, (width, hidden), 0.0, 0.02), "nvfp4")
        s["x_global"] = torch.full((1,), 448.0 * 6.0 / 8.0, device="cuda")       # calibrated once
        _rotation(s, g, t, dim // 2, 1)
        return s
    _rotation(s, g, t, case["rotated"] // 2, case["axes"])
    _heads(s, case, g, "", dt)
    if op == "rmsnorm_rope_backward":
        s["dq"] = _normal(g, s["q"].shape, 0.0, 1.0, dt)
        s["dk"] = _normal(g, s["k"].shape, 0.0, 1.0, dt)
    return s


# -- plain forms -----------------------------------------------------------------------------------------

def _plain_matmul(a, w, a_global, w_global, bias, dtype):
    out = a @ w.t()
    if a_global is not None:
        out = out / a_global / w_global
    return (out if bias is None else out + bias.float()).to(dtype)


def _angles(state, half):
    """Cosine and sine of every token's frequencies, [tokens, 1, half]."""
    cos, sin, place, sections = state["cos"], state["sin"], state["positions"], state["sections"]
    if sections is None:
        return cos[place][:, None], sin[place][:, None]
    axis = torch.repeat_interleave(torch.arange(len(sections), device=cos.device),
                                   torch.tensor(sections, device=cos.device), output_size=half)
    at, i = place.t()[:, axis], torch.arange(half, device=cos.device)
    return cos[at, i][:, None], sin[at, i][:, None]


def _turn(x, cos, sin, interleaved):
    """x with its first 2 * half elements rotated."""
    half = cos.shape[-1]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _plain_norm(x):
    f = x.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)
    return f * rstd, rstd


def _plain_rope(x, gamma, cos, sin, interleaved):
    return _turn(_plain_norm(x)[0] * gamma.float(), cos, sin, interleaved).to(x.dtype)


def _plain_rope_backward(dy, x, gamma, cos, sin, interleaved):
    xhat, rstd = _plain_norm(x)
    g = _turn(dy.float(), cos, -sin, interleaved)
    u = g * gamma.float()
    dx = (u - xhat * (u * xhat).mean(-1, keepdim=True)) * rstd
    return dx.to(x.dtype), (g * xhat).sum((0, 1)).to(gamma.dtype)


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op in ("matmul", "quant_matmul"):
        fmt = case["format"]
        w = _dequantise(state["w"], state["w_scale"], fmt)
        if op == "matmul":
            return {"out": _plain_matmul(_dequantise(state["a"], state["a_scale"], fmt), w, state["a_global"],
                                         state["w_global"], state["bias"], DTYPES[case["out"]])}
        gs = _global_scale(state["x"]) if fmt == "nvfp4" else None
        packed, byte = _quantise(state["x"], fmt, gs)
        a = _dequantise(packed, _tiled(byte), fmt)
        return {"out": _plain_matmul(a, w, gs, state["w_global"], state["bias"], DTYPES[case["dtype"]])}
    if op == "qkv":
        s = (state["x"].float() + state["residual"].float()).to(state["x"].dtype)
        y = _plain_norm(s)[0] * state["gamma"].float()
        packed, byte = _quantise(y, "nvfp4", state["x_global"])
        qkv = _plain_matmul(_dequantise(packed, _tiled(byte), "nvfp4"), _dequantise(state["w"], state["w_scale"], "nvfp4"),
                            state["x_global"], state["w_global"], None, s.dtype)
        q, k, v = _split(qkv, case["heads"], case["kv_heads"], case["dim"])
        cos, sin = _angles(state, case["dim"] // 2)
        return {"q": _plain_rope(q, state["gq"], cos, sin, False), "k": _plain_rope(k, state["gk"], cos, sin, False),
                "v": v, "residual": s}
    cos, sin = _angles(state, case["rotated"] // 2)
    turn = case["interleaved"]
    if op == "rmsnorm_rope":
        return {"q": _plain_rope(state["q"], state["gq"], cos, sin, turn),
                "k": _plain_rope(state["k"], state["gk"], cos, sin, turn)}
    dq, dgq = _plain_rope_backward(state["dq"], state["q"], state["gq"], cos, sin, turn)
    dk, dgk = _plain_rope_backward(state["dk"], state["k"], state["gk"], cos, sin, turn)
    return {"dq": dq, "dk": dk, "dgq": dgq, "dgk": dgk}


def run(state):
    if not own:
        return _plain(state)
    import rmsnorm_precision_activation_gb300 as rq
    case = state["case"]
    op = case["op"]
    if op in ("matmul", "quant_matmul"):
        nv = case["format"] == "nvfp4"
        if op == "matmul":
            a, scale, gs, dtype = state["a"], state["a_scale"], state["a_global"], DTYPES[case["out"]]
        elif nv:
            gs, dtype = rq.nvfp4_global_scale(state["x"]), DTYPES[case["dtype"]]
            a, scale = rq.quant_nvfp4(state["x"], global_scale=gs, swizzled=True)
        else:
            dtype = DTYPES[case["dtype"]]
            a, scale = rq.quant_mxfp4(state["x"], swizzled=True)
        if nv:
            return {"out": rq.matmul_nvfp4(a, scale, state["w"], state["w_scale"], input_global_scale=gs,
                                           weight_global_scale=state["w_global"], bias=state["bias"], out_dtype=dtype)}
        return {"out": rq.matmul_mxfp4(a, scale, state["w"], state["w_scale"], bias=state["bias"], out_dtype=dtype)}
    if op == "qkv":
        codes, scale, res = rq.rmsnorm_quant_nvfp4(state["x"], state["gamma"], global_scale=state["x_global"],
                                                   residual=state["residual"], epsilon=EPS, swizzled=True)
        qkv = rq.matmul_nvfp4(codes, scale, state["w"], state["w_scale"], input_global_scale=state["x_global"],
                              weight_global_scale=state["w_global"], out_dtype=state["x"].dtype)
        q, k, v = _split(qkv, case["heads"], case["kv_heads"], case["dim"])
        q, k = rq.rmsnorm_rope(q, k, state["gq"], state["gk"], state["cos"], state["sin"], state["positions"],
                               epsilon=EPS)
        return {"q": q, "k": k, "v": v, "residual": res}
    if op == "rmsnorm_rope":
        q, k = rq.rmsnorm_rope(state["q"], state["k"], state["gq"], state["gk"], state["cos"], state["sin"],
                               state["positions"], sections=state["sections"], interleaved=case["interleaved"],
                               epsilon=EPS)
        return {"q": q, "k": k}
    dq, dk, dgq, dgk = rq.rmsnorm_rope_backward(
        state["dq"], state["dk"], state["q"], state["k"], state["gq"], state["gk"], state["cos"], state["sin"],
        state["positions"], sections=state["sections"], interleaved=case["interleaved"], epsilon=EPS)
    return {"dq": dq, "dk": dk, "dgq": dgq, "dgk": dgk}


def _codes_bytes(rows, k, fmt):
    return rows * k // 2 + rows * k // BLOCK[fmt]


def work(case):
    op = case["op"]
    if op in ("matmul", "quant_matmul"):
        m, n, k, fmt = case["m"], case["n"], case["k"], case["format"]
        e = SIZE[case["out" if op == "matmul" else "dtype"]]
        moved = _codes_bytes(n, k, fmt) + m * n * e + (n * e if case["bias"] else 0)
        if op == "matmul":
            return {"bytes": moved + _codes_bytes(m, k, fmt), "flops": 2 * m * n * k}
        # x; the codes stay on the chip
        return {"bytes": moved + m * k * e, "flops": 2 * m * n * k + 4 * m * k}
    t, h, kv, d, e = case["tokens"], case["heads"], case["kv_heads"], case["dim"], SIZE[case["dtype"]]
    if op == "qkv":
        width, hidden = (h + 2 * kv) * d, case["hidden"]
        # x, the residual and the sum; the weight; the outputs; table rows, positions and gammas
        return {"bytes": 3 * t * hidden * e + _codes_bytes(width, hidden, "nvfp4") + t * width * e
                + min(t, TABLE) * d * 4 + 8 * t + (hidden + 2 * d) * e,
                "flops": 2 * t * width * hidden + 10 * t * hidden + 10 * t * (h + kv) * d}
    n, around = t * (h + kv) * d, 8 * t * case["axes"] + min(t, TABLE) * case["rotated"] * 4
    if op == "rmsnorm_rope":
        return {"bytes": 2 * n * e + around + 2 * d * e, "flops": 8 * n}
    # the gradients that come, the heads and their gradients; gammas and their gradients
    return {"bytes": 3 * n * e + around + 4 * d * e, "flops": 18 * n}


# -- the same in 64 bits ---------------------------------------------------------------------------------

def _exact_codes(packed):
    """Values of packed E2M1 codes, from their bits: sign, two of exponent, one of mantissa."""
    nibble = torch.empty((packed.shape[0], packed.shape[1] * 2), dtype=torch.uint8, device=packed.device)
    nibble[:, 0::2] = packed & 15
    nibble[:, 1::2] = packed >> 4
    exponent, mantissa = ((nibble >> 1) & 3).double(), (nibble & 1).double()
    value = torch.where(exponent > 0, torch.exp2(exponent - 1) * (1 + mantissa / 2), mantissa / 2)
    return torch.where(nibble > 7, -value, value)


def _exact_operand(packed, tiles, fmt):
    rows, k = packed.shape[0], 2 * packed.shape[1]
    r = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(k // BLOCK[fmt], device="cuda")[None]
    wide = (k // BLOCK[fmt] + 3) // 4
    byte = tiles.view(torch.uint8)[((r // 128 * wide + b // 4) * 32 + r % 32) * 16 + r % 128 // 32 * 4 + b % 4]
    scale = byte.view(torch.float8_e4m3fn).double() if fmt == "nvfp4" else torch.pow(2.0, byte.double() - 127)
    return _exact_codes(packed) * scale.repeat_interleave(BLOCK[fmt], dim=1)


def _exact_rounded(t):
    """The nearest of E2M1's values: one is passed at each midpoint, at it only where the next code is even."""
    a, value = t.abs(), torch.zeros_like(t)
    for i, (low, high) in enumerate(zip(_VALUES, _VALUES[1:])):
        mid = (low + high) / 2
        value += (high - low) * ((a >= mid) if i % 2 else (a > mid))
    return torch.copysign(value, t)


def _exact_quantised(x, fmt, gs):
    """x after quantisation, divided by nothing: codes times block scales."""
    parts = x.double().unflatten(1, (-1, BLOCK[fmt]))
    top = parts.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        scale = torch.clamp(top * gs.double() / 6, max=448).to(torch.float8_e4m3fn).double()
        return torch.where(scale > 0, _exact_rounded(parts * gs.double() / scale) * scale, 0.0).flatten(1)
    scale = torch.exp2(torch.ceil(torch.log2(top / 6)).clamp(-127, 128))
    return torch.where(scale > 2.0 ** -127, _exact_rounded(parts / scale) * scale, 0.0).flatten(1)


def _exact_rope(x, gamma, turns, interleaved):
    """Norm, then a complex product with each frequency's turn."""
    y = x.double() * torch.rsqrt(x.double().square().mean(-1, keepdim=True) + EPS) * gamma.double()
    return _exact_turned(y, turns, interleaved)


def _exact_turned(y, turns, interleaved):
    y, half = y.clone(), turns.shape[-1]
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    z = torch.complex(y[..., first], y[..., second]) * turns.unsqueeze(1)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_turns(s, half):
    place = s["positions"].reshape(-1, s["positions"].shape[-1])
    sections = s["sections"] or (half,)
    parts, at = [], 0
    for axis, count in enumerate(sections):
        rows = place[axis]
        parts.append(torch.complex(s["cos"][rows, at:at + count].double(), s["sin"][rows, at:at + count].double()))
        at += count
    return torch.cat(parts, -1)


def _exact_gradient(dy, x, gamma, turns, interleaved):
    xd = x.double()
    r = torch.rsqrt(xd.square().mean(-1, keepdim=True) + EPS)
    back = _exact_turned(dy.double(), turns.conj(), interleaved)
    dgamma = torch.einsum("thd,thd->d", back, xd * r)
    back *= gamma.double()
    along = torch.einsum("thd,thd->th", back, xd).unsqueeze(-1) / xd.shape[-1]
    return r * back - r ** 3 * along * xd, dgamma


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("matmul", "quant_matmul"):
        fmt = case["format"]
        w = _exact_operand(s["w"], s["w_scale"], fmt)
        if op == "matmul":
            a, gs = _exact_operand(s["a"], s["a_scale"], fmt), s["a_global"]
        else:
            gs = 2688.0 / s["x"].abs().max().float() if fmt == "nvfp4" else None
            a = _exact_quantised(s["x"], fmt, gs)
        out = torch.einsum("mk,nk->mn", a, w)
        if gs is not None:
            out /= gs.double() * s["w_global"].double()
        return {"out": out if s["bias"] is None else out + s["bias"].double()}
    if op == "qkv":
        x = s["x"] + s["residual"]
        y = x.double()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["gamma"].double()
        out = torch.einsum("mk,nk->mn", _exact_quantised(y, "nvfp4", s["x_global"]),
                           _exact_operand(s["w"], s["w_scale"], "nvfp4"))
        out = (out / (s["x_global"].double() * s["w_global"].double())).to(x.dtype)
        q, k, v = out.split([case["heads"] * case["dim"]] + [case["kv_heads"] * case["dim"]] * 2, 1)
        shape, turns = (case["tokens"], -1, case["dim"]), _exact_turns(s, case["dim"] // 2)
        return {"q": _exact_rope(q.reshape(shape), s["gq"], turns, False),
                "k": _exact_rope(k.reshape(shape), s["gk"], turns, False), "v": v.reshape(shape).double(),
                "residual": x.double()}
    turns, turn = _exact_turns(s, case["rotated"] // 2), case["interleaved"]
    if op == "rmsnorm_rope":
        return {"q": _exact_rope(s["q"], s["gq"], turns, turn), "k": _exact_rope(s["k"], s["gk"], turns, turn)}
    dq, dgq = _exact_gradient(s["dq"], s["q"], s["gq"], turns, turn)
    dk, dgk = _exact_gradient(s["dk"], s["k"], s["gk"], turns, turn)
    return {"dq": dq, "dk": dk, "dgq": dgq, "dgk": dgk}
