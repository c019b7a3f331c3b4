"""The operators around the FP8 linear layer, as cases that can be timed and compared.

Three groups, in the order a fine-tuning step meets them: the norm in front of
a quantized activation (forward and backward), the FP8 linear layer with bias,
activation and residual in its epilogue (forward, and the epilogue's backward),
and the global norm and clipping of the adapter gradients.

`run` computes a case in its plain form (elementary torch operations in 32
bits, 64 for the long sums) or, where `own` is true, through the library.
`exact` computes the same outputs in 64 bits from the operators' definitions.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
ACTS = ("none", "relu", "gelu_erf", "gelu_tanh", "silu")
EPS = 1e-5

# Output widths and input widths of the linear layers of one Llama-7B block
# (q, k, v, o, gate, up, down), as in synthetic/workloads.py.
BLOCK_N = (4096, 4096, 4096, 4096, 11008, 11008, 4096)
BLOCK_K = (4096, 4096, 4096, 4096, 4096, 4096, 11008)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm in front of the attention projections: 4 x 1024 tokens of a Llama-7B block
        {"name": "norm_fwd_rms_4096x4096", "op": "norm_fwd", "kind": "rms", "rows": 4096, "cols": 4096,
         "dtype": "bf16", "params": "bf16", "affine": True},
        # one token while a tuned model is sampled from: latency
        {"name": "norm_fwd_layer_1x4096", "op": "norm_fwd", "kind": "layer", "rows": 1, "cols": 4096,
         "dtype": "bf16", "params": "bf16", "affine": True},
        # float32 residual stream, odd row length (no row but the first is 16-byte aligned)
        {"name": "norm_fwd_layer_f32_3001x1537", "op": "norm_fwd", "kind": "layer", "rows": 3001, "cols": 1537,
         "dtype": "f32", "params": "f32", "affine": True},
        # the backward of the MLP's norm at 8192 tokens, joined by the residual branch's gradient
        {"name": "norm_bwd_rms_8192x4096", "op": "norm_bwd", "kind": "rms", "rows": 8192, "cols": 4096,
         "dtype": "bf16", "params": "bf16", "dres": True},
        # ragged batch, row length not a multiple of 8, float32 master parameters
        {"name": "norm_bwd_layer_777x2050", "op": "norm_bwd", "kind": "layer", "rows": 777, "cols": 2050,
         "dtype": "bf16", "params": "f32", "dres": False},
        # MLP up-projection at 4096 tokens with its activation, the pre-activation kept for the backward
        {"name": "linear_gelu_4096x11008x4096", "op": "linear_fwd", "M": 4096, "N": 11008, "K": 4096,
         "bias": "bf16", "act": "gelu_tanh", "residual": False, "save_z": True},
        # MLP down-projection at 8192 tokens, added to the residual stream: the largest call
        {"name": "linear_residual_8192x4096x11008", "op": "linear_fwd", "M": 8192, "N": 4096, "K": 11008,
         "bias": "bf16", "act": "none", "residual": True, "save_z": False},
        # one token through an attention-sized projection: the weight is the work
        {"name": "linear_token_1x4096x4096", "op": "linear_fwd", "M": 1, "N": 4096, "K": 4096,
         "bias": "f32", "act": "silu", "residual": True, "save_z": False},
        # backward of the activation and the bias at the MLP's width
        {"name": "linear_bwd_gelu_8192x11008", "op": "linear_bwd", "M": 8192, "N": 11008, "act": "gelu_tanh"},
        # the same at a small ragged size: latency
        {"name": "linear_bwd_silu_200x272", "op": "linear_bwd", "M": 200, "N": 272, "act": "silu"},
        # one attention layer's gradients (dA, dB and a norm's weight): latency
        {"name": "clip_layer_r64", "op": "clip", "blocks": 0, "rank": 64, "width": 4096, "with_a": True},
        # every adapter gradient of a 32-block stack at rank 64: 448 tensors, more than the L2 holds
        {"name": "clip_stack_32x7_r64", "op": "clip", "blocks": 32, "rank": 64, "width": 0, "with_a": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _of16(v):
    return max(16, v // 16 * 16)


def draw(rng):
    op = rng.choice(("norm_fwd", "norm_bwd", "linear_fwd", "linear_bwd", "clip"))
    if op in ("norm_fwd", "norm_bwd"):
        cols = _log(rng, 16, 16384)
        cols = cols if rng.random() < 0.3 else _of16(cols)
        rows = _log(rng, 1, min(16384, 8192 * 11008 // cols))
        case = {"op": op, "kind": rng.choice(("layer", "rms")), "rows": rows, "cols": cols,
                "dtype": rng.choice(("bf16", "bf16", "f32")), "params": rng.choice(("bf16", "f32"))}
        if op == "norm_fwd":
            case["affine"] = rng.random() < 0.8
        else:
            case["dres"] = rng.random() < 0.5
        return case
    if op == "linear_fwd":
        N, K = _of16(_log(rng, 16, 11008)), _of16(_log(rng, 16, 11008))
        M = _log(rng, 1, min(8192, 8192 * 4096 * 11008 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "bias": rng.choice(("", "bf16", "f32")), "act": rng.choice(ACTS),
                "residual": rng.random() < 0.5, "save_z": rng.random() < 0.5}
    if op == "linear_bwd":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _of16(_log(rng, 16, 11008)), "act": rng.choice(ACTS)}
    return {"op": op, "blocks": rng.choice((0, 0, 1, 2, 4, 8, 16, 32)), "rank": 16 * rng.randint(1, 4),
            "width": _log(rng, 16, 11008), "with_a": rng.random() < 0.5}


def _clip_sizes(case):
    """(elements of each bf16 gradient, elements of each float32 gradient)."""
    r = case["rank"]
    if case["blocks"]:
        per = [n * r for n in BLOCK_N] + ([k * r for k in BLOCK_K] if case["with_a"] else [])
        return per * case["blocks"], []
    w = case["width"]
    return [w * r] + ([w * r] if case["with_a"] else []), [w, w + 1]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _hidden(g, rows, cols, dtype):
    """Hidden states: unit normal, a few columns far larger than the rest, rows of different size."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= 1.0 + 20.0 * (torch.rand((1, cols), generator=g, device=DEV) < 0.004)
    x *= 0.5 + torch.rand((rows, 1), generator=g, device=DEV)
    return (x + 0.1).to(dtype)


def _quantized(x):
    """Codes and scale of per-tensor max-abs E4M3 quantization."""
    s = 448.0 / x.abs().amax().float().clamp_min(1e-30)
    codes = (x.float() * s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, s.reshape(1)


def _views(flat, sizes):
    """16-byte aligned views of `sizes` elements each, laid one after another in `flat`."""
    out, at, step = [], 0, 16 // flat.element_size()
    for n in sizes:
        out.append(flat[at:at + n])
        at += -(-n // step) * step
    return out


def _flat_size(sizes, step):
    return sum(-(-n // step) * step for n in sizes)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op in ("norm_fwd", "norm_bwd"):
        rows, cols, dt, pt = case["rows"], case["cols"], DTYPES[case["dtype"]], DTYPES[case["params"]]
        layer = case["kind"] == "layer"
        s["x"] = _hidden(g, rows, cols, dt)
        affine = case.get("affine", True)
        s["gamma"] = (1.0 + _normal(g, cols, 0.1)).to(pt) if affine else None
        s["beta"] = _normal(g, cols, 0.1, pt) if affine and layer else None
        if op == "norm_bwd":
            s["dy"] = _normal(g, (rows, cols), 1e-3, dt)
            s["dres"] = _normal(g, (rows, cols), 1e-3, dt) if case["dres"] else None
            x = s["x"].double()  # the statistics that the forward pass kept
            mean = x.mean(1) if layer else torch.zeros(rows, dtype=torch.float64, device=DEV)
            s["mean"] = mean.float() if layer else None
            s["rstd"] = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
            if own:
                import fp8_quantized_lora_b200 as F
                s["workspace"] = F.workspace(F.OP_NORM_BWD, rows, 0, cols)
    elif op == "linear_fwd":
        M, N, K = case["M"], case["N"], case["K"]
        s["xq"], s["s_x"] = _quantized(_normal(g, (M, K)))
        s["wq"], s["s_w"] = _quantized(_normal(g, (N, K), 0.02))
        s["bias"] = _normal(g, N, 0.1, DTYPES[case["bias"]]) if case["bias"] else None
        s["residual"] = _normal(g, (M, N), 1.0, torch.bfloat16) if case["residual"] else None
    elif op == "linear_bwd":
        M, N = case["M"], case["N"]
        s["dy"] = _normal(g, (M, N), 1e-3, torch.bfloat16)
        s["z"] = _normal(g, (M, N), 1.3, torch.bfloat16) if case["act"] != "none" else None
        if own:
            import fp8_quantized_lora_b200 as F
            s["workspace"] = F.workspace(F.OP_LINEAR_EPILOGUE_BWD, M, N)
    else:
        n16, n32 = _clip_sizes(case)
        s["g16"] = torch.zeros(_flat_size(n16, 8), dtype=torch.bfloat16, device=DEV)
        s["g32"] = torch.zeros(_flat_size(n32, 4), device=DEV)
        views = _views(s["g16"], n16) + _views(s["g32"], n32)
        for k, v in enumerate(views):
            v.copy_(_normal(g, v.shape, 1e-3 * (1 + k % 7)))
        s["out16"], s["out32"] = torch.zeros_like(s["g16"]), torch.zeros_like(s["g32"])
        # about half of the norm of these inputs: the clip is in force
        s["max_norm"] = 1e-3 * math.sqrt(sum(n * (1 + k % 7) ** 2 for k, n in enumerate(n16 + n32))) / 2
        s["factor"] = -1e-2  # minus the learning rate: the increments of B that the proxy update takes
        if own:
            import fp8_quantized_lora_b200 as F
            s["grads"] = F.GradList(views)
            s["outs"] = F.GradList(_views(s["out16"], n16) + _views(s["out32"], n32))
            s["workspace"] = F.workspace(F.OP_CLIP_GRADS)
    return s


# ------------------------------------------------------------------ one pass
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu_erf":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain_norm_fwd(s):
    case, x = s["case"], s["x"].float()
    layer = case["kind"] == "layer"
    mean = x.mean(1) if layer else None
    xc = x - mean[:, None] if layer else x
    rstd = 1 / torch.sqrt((xc * xc).mean(1) + EPS)
    y = xc * rstd[:, None]
    y = y * s["gamma"].float() if s["gamma"] is not None else y
    y = y + s["beta"].float() if s["beta"] is not None else y
    out = {"y": y.to(s["x"].dtype), "rstd": rstd}
    return {**out, "mean": mean} if layer else out


def _plain_norm_bwd(s):
    case, x, dy, rstd = s["case"], s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    layer = case["kind"] == "layer"
    xh = (x - s["mean"][:, None]) * rstd if layer else x * rstd
    g = dy * s["gamma"].float()
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    dx = (dx - g.mean(1, keepdim=True) if layer else dx) * rstd
    dx = dx + s["dres"].float() if s["dres"] is not None else dx
    out = {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0)}
    return {**out, "dbeta": dy.sum(0)} if layer else out


def _plain_linear_fwd(s):
    case = s["case"]
    x = s["xq"].view(torch.float8_e4m3fn).float()
    w = s["wq"].view(torch.float8_e4m3fn).float()
    z = (x @ w.t()) / (s["s_x"] * s["s_w"])
    z = z + s["bias"].float() if s["bias"] is not None else z
    y = _act(z, case["act"])
    y = y + s["residual"].float() if s["residual"] is not None else y
    out = {"y": y.to(torch.bfloat16)}
    return {**out, "z": z.to(torch.bfloat16)} if case["save_z"] else out


def _plain_linear_bwd(s):
    act, dy = s["case"]["act"], s["dy"].float()
    if act == "none":  # dZ is dY itself
        return {"dbias": dy.sum(0)}
    dz = dy * _act_slope(s["z"].float(), act)
    return {"dz": dz.to(torch.bfloat16), "dbias": dz.sum(0)}


def _plain_clip(s):
    total = s["g16"].double().square().sum() + s["g32"].double().square().sum()
    norm = total.sqrt()
    coef = torch.clamp(s["max_norm"] / norm, max=1.0)
    by = (s["factor"] * coef).float()
    return {"out16": (s["g16"].float() * by).to(torch.bfloat16), "out32": s["g32"] * by,
            "norm": norm.float().reshape(1), "coef": coef.float().reshape(1)}


def _own_run(s):
    import fp8_quantized_lora_b200 as F

    case, op = s["case"], s["case"]["op"]
    if op in ("norm_fwd", "norm_bwd"):
        layer = case["kind"] == "layer"
        kind = F.NORM_LAYER if layer else F.NORM_RMS
        if op == "norm_fwd":
            y, mean, rstd = F.falqon_norm_fwd(s["x"], s["gamma"], s["beta"], EPS, kind)
            return {"y": y, "rstd": rstd, "mean": mean} if layer else {"y": y, "rstd": rstd}
        dx, dgamma, dbeta = F.falqon_norm_bwd(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], kind, dres=s["dres"],
                                              workspace=s["workspace"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta} if layer else {"dx": dx, "dgamma": dgamma}
    if op in ("linear_fwd", "linear_bwd"):
        act = {"none": F.ACT_NONE, "relu": F.ACT_RELU, "gelu_erf": F.ACT_GELU_ERF, "gelu_tanh": F.ACT_GELU_TANH,
               "silu": F.ACT_SILU}[case["act"]]
        if op == "linear_fwd":
            y, z = F.falqon_linear_fwd_epilogue(s["xq"], s["s_x"], s["wq"], s["s_w"], bias=s["bias"], act=act,
                                                residual=s["residual"], z=True if case["save_z"] else None)
            return {"y": y, "z": z} if case["save_z"] else {"y": y}
        dz, dbias = F.falqon_linear_epilogue_bwd(s["dy"], s["z"], act, dz=None if case["act"] == "none" else True,
                                                 workspace=s["workspace"])
        return {"dbias": dbias} if dz is None else {"dz": dz, "dbias": dbias}
    _, norm, coef = F.falqon_clip_grads(s["grads"], s["max_norm"], s["factor"], out=s["outs"],
                                        workspace=s["workspace"])
    return {"out16": s["out16"], "out32": s["out32"], "norm": norm, "coef": coef}


def run(state):
    if own:
        return _own_run(state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "linear_fwd": _plain_linear_fwd,
            "linear_bwd": _plain_linear_bwd, "clip": _plain_clip}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        R, C, e, p = case["rows"], case["cols"], BYTES[case["dtype"]], BYTES[case["params"]]
        layer = case["kind"] == "layer"
        if op == "norm_fwd":
            params = (2 if layer else 1) * p * C if case["affine"] else 0
            return {"bytes": 2 * e * R * C + params + 4 * R * (2 if layer else 1), "flops": 8 * R * C}
        return {"bytes": (4 if case["dres"] else 3) * e * R * C + p * C + 4 * (R + C) * (2 if layer else 1),
                "flops": 14 * R * C}
    if op == "linear_fwd":
        M, N, K = case["M"], case["N"], case["K"]
        outs = 1 + bool(case["residual"]) + bool(case["save_z"])
        return {"bytes": M * K + N * K + 2 * outs * M * N + N * BYTES.get(case["bias"], 0), "flops": 2 * M * N * K}
    if op == "linear_bwd":
        M, N = case["M"], case["N"]
        return {"bytes": (2 if case["act"] == "none" else 6) * M * N + 4 * N, "flops": 16 * M * N}
    n16, n32 = _clip_sizes(case)
    return {"bytes": 4 * sum(n16) + 8 * sum(n32), "flops": 3 * (sum(n16) + sum(n32))}


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op == "norm_fwd":
        x = d["x"]
        var, mean = torch.var_mean(x, dim=1, correction=0)
        moment = var if case["kind"] == "layer" else x.pow(2).sum(1) / x.shape[1]
        rstd = torch.pow(moment + EPS, -0.5)
        y = torch.einsum("rc,r->rc", x - mean[:, None] if case["kind"] == "layer" else x, rstd)
        if d["gamma"] is not None:
            y = torch.einsum("rc,c->rc", y, d["gamma"])
        if d["beta"] is not None:
            y = y + d["beta"][None]
        return {"y": y, "rstd": rstd, "mean": mean} if case["kind"] == "layer" else {"y": y, "rstd": rstd}
    if op == "norm_bwd":
        # dx = J^T (gamma dy) with the Jacobian of the normalised row: J = rstd (I - [1 1^T] / C - xh xh^T / C)
        layer, C = case["kind"] == "layer", case["cols"]
        xh = (d["x"] - (d["mean"][:, None] if layer else 0.0)) * d["rstd"][:, None]
        v = torch.einsum("rc,c->rc", d["dy"], d["gamma"])
        along = torch.einsum("rc,rc->r", v, xh) / C
        dx = v - torch.einsum("r,rc->rc", along, xh)
        if layer:
            dx = dx - (torch.einsum("rc->r", v) / C)[:, None]
        dx = torch.einsum("rc,r->rc", dx, d["rstd"])
        if d["dres"] is not None:
            dx = dx + d["dres"]
        out = {"dx": dx, "dgamma": torch.einsum("rc,rc->c", d["dy"], xh)}
        return {**out, "dbeta": torch.einsum("rc->c", d["dy"])} if layer else out
    if op == "linear_fwd":
        table = torch.arange(256, dtype=torch.uint8, device=DEV)
        sign, e, m = 1 - 2 * (table >> 7).double(), ((table >> 3) & 15).double(), (table & 7).double()
        values = sign * torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), torch.exp2(e - 6) * (m / 8))
        z = values[s["xq"].long()] @ values[s["wq"].long()].T / (d["s_x"] * d["s_w"])
        if d["bias"] is not None:
            z = z + d["bias"]
        y = _exact_act(z, case["act"])[0]
        if d["residual"] is not None:
            y = y + d["residual"]
        return {"y": y, "z": z} if case["save_z"] else {"y": y}
    if op == "linear_bwd":
        if case["act"] == "none":
            return {"dbias": torch.einsum("mn->n", d["dy"])}
        dz = d["dy"] * _exact_act(d["z"], case["act"])[1]
        return {"dz": dz, "dbias": torch.einsum("mn->n", dz)}
    norm = torch.sqrt(torch.dot(d["g16"], d["g16"]) + torch.dot(d["g32"], d["g32"]))
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    return {"out16": d["g16"] * (s["factor"] * coef), "out32": d["g32"] * (s["factor"] * coef),
            "norm": norm.reshape(1), "coef": coef.reshape(1)}


def _exact_act(z, act):
    """(value, derivative) in 64 bits; the derivative by the chain rule on the normal or logistic distribution."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return z.clamp_min(0.0), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu_erf":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z.pow(2) / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":  # (1 + tanh u) / 2 is the logistic function of 2 u
        u2 = math.sqrt(8 / math.pi) * (z + 0.044715 * z.pow(3))
        p = torch.sigmoid(u2)
        return z * p, p + z * p * torch.sigmoid(-u2) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z.pow(2))
    p = torch.sigmoid(z)
    return z * p, p + z * p * torch.sigmoid(-z)
