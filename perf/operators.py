"""The layer-norm and 8-bit-integer operators as a user's program calls them, with plain forms.

layernorm           s = RN(x + r), y = (s - mean) * rstd * (gamma + offset) + beta
layernorm_backward  the gradients of s (with the residual stream's own gradient added), gamma, beta
matmul_int8         out = (q @ w^T) * q_scale[:, None] * w_scale[None, :] + bias, q and w int8
norm_matmul         a projection behind a norm: layernorm_quant_int8 or rmsnorm_quant_int8 (one
                    scale per token, amax / 127), then matmul_int8 on its codes

Where `own` is false, run() computes these with elementary torch operations in 32 bits; where it is
true, with the package's calls. Both take what prepare() gives.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5

# Ranges that draw() covers: no drawn case costs more than the largest listed one of its operator.
MOST_ELEMENTS = 16384 * 8192
MOST_PRODUCTS = 8192 ** 3


def listed():
    return [
        # one decoded token through the norm in front of a block, with its residual
        {"name": "ln_token", "op": "layernorm", "rows": 1, "hidden": 8192, "dtype": "bf16",
         "residual": True, "stats": False, "offset": 0.0},
        # a training step's forward norm, statistics kept for the backward pass
        {"name": "ln_step", "op": "layernorm", "rows": 8192, "hidden": 4096, "dtype": "bf16",
         "residual": True, "stats": True, "offset": 0.0},
        # a model in 32 bits whose width is no multiple of a vector
        {"name": "ln_odd", "op": "layernorm", "rows": 4099, "hidden": 5121, "dtype": "fp32",
         "residual": False, "stats": True, "offset": 0.0},
        # rows too wide for one thread block
        {"name": "ln_wide", "op": "layernorm", "rows": 2048, "hidden": 65536, "dtype": "fp16",
         "residual": False, "stats": False, "offset": 1.0},
        # a fine-tuning step on one short sequence
        {"name": "lnb_short", "op": "layernorm_backward", "rows": 64, "hidden": 4096,
         "dtype": "bf16", "residual": True, "offset": 0.0},
        # a training step's backward norm on a full batch
        {"name": "lnb_step", "op": "layernorm_backward", "rows": 16384, "hidden": 8192,
         "dtype": "fp16", "residual": True, "offset": 1.0},
        # the backward pass in 32 bits at a width that is no multiple of a vector
        {"name": "lnb_odd", "op": "layernorm_backward", "rows": 5003, "hidden": 2051,
         "dtype": "fp32", "residual": False, "offset": 0.0},
        # one decoded token through a projection
        {"name": "mm_token", "op": "matmul_int8", "m": 1, "n": 7168, "k": 8192, "out": "bf16",
         "bias": False},
        # a decode batch of ragged size, an output width that is no multiple of a tile
        {"name": "mm_batch", "op": "matmul_int8", "m": 100, "n": 5001, "k": 5120, "out": "fp16",
         "bias": True},
        # a long prompt through a square projection
        {"name": "mm_prompt", "op": "matmul_int8", "m": 8192, "n": 8192, "k": 8192, "out": "bf16",
         "bias": False},
        # a decode batch through RMS norm, quantisation and an up projection
        {"name": "norm_mm_batch", "op": "norm_matmul", "norm": "rms", "m": 16, "n": 16384,
         "k": 4096, "dtype": "bf16", "residual": True, "bias": False},
        # a prompt through layer norm, quantisation and an up projection with bias
        {"name": "norm_mm_prompt", "op": "norm_matmul", "norm": "layer", "m": 4096, "n": 16384,
         "k": 5120, "dtype": "bf16", "residual": True, "bias": True},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["layernorm", "layernorm_backward", "matmul_int8", "norm_matmul"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op in ("layernorm", "layernorm_backward"):
        hidden = _log(rng, 64, 65536)
        if rng.random() < 0.7:
            hidden = max(64, hidden // 8 * 8)
        rows = _log(rng, 1, min(65536, MOST_ELEMENTS // hidden // (2 if dtype == "fp32" else 1)))
        case = {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype,
                "residual": rng.random() < 0.5, "offset": rng.choice([0.0, 1.0])}
        if op == "layernorm":
            case["stats"] = rng.random() < 0.5
        return case
    k = 16 * _log(rng, 8, 1024)
    n = _log(rng, 64, 16384)
    m = _log(rng, 1, min(8192, MOST_PRODUCTS // (n * k)))
    if op == "matmul_int8":
        return {"op": op, "m": m, "n": n, "k": k, "out": dtype, "bias": rng.random() < 0.5}
    return {"op": op, "norm": rng.choice(["rms", "layer"]), "m": m, "n": n, "k": k,
            "dtype": rng.choice(["bf16", "fp16"]), "residual": rng.random() < 0.5,
            "bias": rng.random() < 0.5}


def _normal(g, shape, mean, std, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _weight(g, n, k):
    """A projection's weight in 8 bits with one scale per output channel."""
    w = torch.randn((n, k), generator=g, device="cuda")
    amax = w.abs().amax(1, keepdim=True)
    q = torch.round(w * (127.0 / amax)).to(torch.int8)
    return q, (amax[:, 0] * (0.02 / 127.0)).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op in ("layernorm", "layernorm_backward"):
        dt, shape = DTYPES[case["dtype"]], (case["rows"], case["hidden"])
        s["gamma"] = _normal(g, shape[1:], 1.0 - case["offset"], 0.1, dt)
        # a residual stream: rows of differing size, off centre
        x = torch.randn(shape, generator=g, device="cuda") + 0.25
        s["x"] = (x * (0.5 + torch.rand((shape[0], 1), generator=g, device="cuda"))).to(dt)
        del x
        if op == "layernorm":
            s["beta"] = _normal(g, shape[1:], 0.0, 0.1, dt)
            s["residual"] = _normal(g, shape, 0.0, 1.0, dt) if case["residual"] else None
        else:
            x = s["x"].float()
            mean = x.mean(1, keepdim=True)
            s["mean"] = mean[:, 0].contiguous()
            s["rstd"] = torch.rsqrt((x - mean).square().mean(1) + EPS)
            s["dy"] = _normal(g, shape, 0.0, 1.0, dt)
            s["dres"] = _normal(g, shape, 0.0, 1.0, dt) if case["residual"] else None
        return s
    m, n, k = case["m"], case["n"], case["k"]
    s["w"], s["w_scale"] = _weight(g, n, k)
    if op == "matmul_int8":
        a = torch.randn((m, k), generator=g, device="cuda")
        amax = a.abs().amax(1, keepdim=True)
        s["q"] = torch.round(a * (127.0 / amax)).to(torch.int8)
        s["q_scale"] = (amax[:, 0] / 127.0).contiguous()
        dt = DTYPES[case["out"]]
    else:
        dt = DTYPES[case["dtype"]]
        s["gamma"] = _normal(g, (k,), 1.0, 0.1, dt)
        s["beta"] = _normal(g, (k,), 0.0, 0.1, dt) if case["norm"] == "layer" else None
        s["x"] = _normal(g, (m, k), 0.1, 1.0, dt)
        s["residual"] = _normal(g, (m, k), 0.0, 1.0, dt) if case["residual"] else None
    s["bias"] = _normal(g, (n,), 0.0, 0.1, dt) if case["bias"] else None
    return s


def _add(x, r):
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def _plain_layernorm(s, gamma, beta, offset):
    f = s.float()
    mean = f.mean(1, keepdim=True)
    d = f - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    y = d * rstd * (gamma.float() + offset)
    if beta is not None:
        y = y + beta.float()
    return y, mean[:, 0], rstd[:, 0]


def _plain_rmsnorm(s, gamma):
    f = s.float()
    return f * (1.0 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)) * gamma.float()


def _plain_backward(dy, s, gamma, mean, rstd, dres, offset):
    xhat = (s.float() - mean[:, None]) * rstd[:, None]
    f = dy.float()
    g = f * (gamma.float() + offset)
    ds = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * rstd[:, None]
    if dres is not None:
        ds = ds + dres.float()
    return ds.to(s.dtype), (f * xhat).sum(0).to(gamma.dtype), f.sum(0).to(gamma.dtype)


def _plain_matmul(q, q_scale, w, w_scale, bias, dtype):
    out = (q.float() @ w.float().t()) * q_scale[:, None] * w_scale[None, :]
    return (out if bias is None else out + bias.float()).to(dtype)


def _plain_quantise(y):
    scale = y.abs().amax(1, keepdim=True) / 127.0
    q = torch.round(y / torch.where(scale > 0, scale, 1.0)).clamp(-127.0, 127.0)
    return q, scale[:, 0]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import rmsnorm_precision_activation_gb300 as rq
        if op == "layernorm":
            y, res, mean, rstd = rq.layernorm(
                state["x"], state["gamma"], state["beta"], residual=state["residual"],
                epsilon=EPS, weight_offset=case["offset"], stats=case["stats"])
            return {"y": y, "residual": res, "mean": mean, "rstd": rstd}
        if op == "layernorm_backward":
            ds, dgamma, dbeta = rq.layernorm_backward(
                state["dy"], state["x"], state["gamma"], state["mean"], state["rstd"],
                grad_residual=state["dres"], weight_offset=case["offset"])
            return {"ds": ds, "dgamma": dgamma, "dbeta": dbeta}
        if op == "matmul_int8":
            return {"out": rq.matmul_int8(state["q"], state["q_scale"], state["w"],
                                          state["w_scale"], bias=state["bias"],
                                          out_dtype=DTYPES[case["out"]])}
        if case["norm"] == "layer":
            q, scale, res = rq.layernorm_quant_int8(state["x"], state["gamma"], state["beta"],
                                                    residual=state["residual"], epsilon=EPS)
        else:
            q, scale, res = rq.rmsnorm_quant_int8(state["x"], state["gamma"],
                                                  residual=state["residual"], epsilon=EPS)
        out = rq.matmul_int8(q, scale, state["w"], state["w_scale"], bias=state["bias"],
                             out_dtype=DTYPES[case["dtype"]])
        return {"out": out, "residual": res}
    if op == "layernorm":
        s = _add(state["x"], state["residual"])
        y, mean, rstd = _plain_layernorm(s, state["gamma"], state["beta"], case["offset"])
        return {"y": y.to(s.dtype), "residual": s if case["residual"] else None,
                "mean": mean if case["stats"] else None, "rstd": rstd if case["stats"] else None}
    if op == "layernorm_backward":
        ds, dgamma, dbeta = _plain_backward(state["dy"], state["x"], state["gamma"], state["mean"],
                                            state["rstd"], state["dres"], case["offset"])
        return {"ds": ds, "dgamma": dgamma, "dbeta": dbeta}
    if op == "matmul_int8":
        return {"out": _plain_matmul(state["q"], state["q_scale"], state["w"], state["w_scale"],
                                     state["bias"], DTYPES[case["out"]])}
    s = _add(state["x"], state["residual"])
    if case["norm"] == "layer":
        y = _plain_layernorm(s, state["gamma"], state["beta"], 0.0)[0]
    else:
        y = _plain_rmsnorm(s, state["gamma"])
    q, scale = _plain_quantise(y)
    out = _plain_matmul(q, scale, state["w"], state["w_scale"], state["bias"],
                        DTYPES[case["dtype"]])
    return {"out": out, "residual": s if case["residual"] else None}


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] in ("layernorm", "layernorm_backward"):
        rows, hidden, e = case["rows"], case["hidden"], size[case["dtype"]]
        n = rows * hidden
        if case["op"] == "layernorm":
            # x and y, with a residual r and s too; gamma and beta; mean and rstd where kept
            return {"bytes": n * e * (4 if case["residual"] else 2) + 2 * hidden * e
                    + (8 * rows if case["stats"] else 0), "flops": 8 * n}
        # dy, s and ds, with a residual its gradient; mean and rstd; gamma, dgamma and dbeta
        return {"bytes": n * e * (4 if case["residual"] else 3) + 8 * rows + 3 * hidden * e,
                "flops": 14 * n}
    m, n, k = case["m"], case["n"], case["k"]
    e = size[case["out"] if case["op"] == "matmul_int8" else case["dtype"]]
    moved = n * k + 4 * n + m * n * e + (n * e if case["bias"] else 0)
    if case["op"] == "matmul_int8":
        return {"bytes": moved + m * k + 4 * m, "flops": 2 * m * n * k}
    # x, with a residual r and s too; gamma, and beta for layer norm; the codes stay on the chip
    moved += m * k * e * (3 if case["residual"] else 1) + k * e * (2 if case["norm"] == "layer" else 1)
    return {"bytes": moved, "flops": 2 * m * n * k + 10 * m * k}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def d(t):
        return t.double()

    if op == "layernorm":
        x = s["x"] if s["residual"] is None else s["x"] + s["residual"]
        xd = d(x)
        var, mean = torch.var_mean(xd, dim=-1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.einsum("rh,r,h->rh", xd - mean.unsqueeze(-1), rstd, d(s["gamma"]) + case["offset"])
        return {"y": y + d(s["beta"]), "residual": xd if s["residual"] is not None else None,
                "mean": mean if case["stats"] else None, "rstd": rstd if case["stats"] else None}
    if op == "layernorm_backward":
        dy, h = d(s["dy"]), case["hidden"]
        centred = (d(s["x"]) - d(s["mean"]).unsqueeze(-1)) * d(s["rstd"]).unsqueeze(-1)
        dgamma, dbeta = torch.einsum("rh,rh->h", dy, centred), torch.einsum("rh->h", dy)
        dy *= d(s["gamma"]) + case["offset"]
        along = torch.einsum("rh,rh->r", dy, centred) / h
        dy -= dy.sum(-1, keepdim=True) / h
        dy -= along.unsqueeze(-1) * centred
        dy *= d(s["rstd"]).unsqueeze(-1)
        return {"ds": dy if s["dres"] is None else dy + d(s["dres"]), "dgamma": dgamma,
                "dbeta": dbeta}
    if op == "matmul_int8":
        out = torch.einsum("mk,nk->mn", d(s["q"]), d(s["w"]))
        out = out * torch.outer(d(s["q_scale"]), d(s["w_scale"]))
        return {"out": out if s["bias"] is None else out + d(s["bias"])}
    x = s["x"] if s["residual"] is None else s["x"] + s["residual"]
    y = d(x)
    if case["norm"] == "layer":
        var, mean = torch.var_mean(y, dim=-1, correction=0)
        y = (y - mean.unsqueeze(-1)) * ((var + EPS) ** -0.5).unsqueeze(-1) * d(s["gamma"]) + d(s["beta"])
    else:
        y = y * (torch.einsum("mk,mk->m", y, y) / case["k"] + EPS).pow(-0.5).unsqueeze(-1) * d(s["gamma"])
    step = y.abs().amax(-1) / 127
    codes = torch.round(y / step.unsqueeze(-1))
    out = torch.einsum("mk,nk->mn", codes, d(s["w"])) * torch.outer(step, d(s["w_scale"]))
    return {"out": out if s["bias"] is None else out + d(s["bias"]),
            "residual": d(x) if s["residual"] is not None else None}
