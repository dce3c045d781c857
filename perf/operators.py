"""Cases that time the operators for experts of one's own: grouping rows by expert, products grouped by
expert (bias, activation and residual in the epilogue, gradients), 8-bit activation checkpoints, and the combine.

``run`` computes a case either in plain torch operations (``own`` false) or through the framework's calls.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BLOCK = 64        # columns that share one scale of an 8-bit checkpoint
_E4M3_MAX = 448.0  # largest finite E4M3 value
_TINY = 1e-30      # smallest block maximum that a scale is made from


def listed():
    return [
        # a decode step of 32 sequences: the index work between the router and the experts
        dict(name="group_decode", op="group", T=32, k=2, N=8, skew=0.0, capacity=0),
        # a long prefill under a skewed router with a capacity that drops the hot experts' extras
        dict(name="group_prefill_skew", op="group", T=16384, k=8, N=128, skew=1.2, capacity=2048),
        # one new token through two FP8 experts: streaming their gate and up weights
        dict(name="up_one_token_fp8", op="linear", T=1, k=2, N=8, d_in=4096, d_out=14336, dtype="bf16",
             fp8=True, act="swiglu", gather=True, bias=False, residual=False, save=False, skew=0.0),
        # a decode step of 32 sequences: every expert's gate and up weights, a few rows each
        dict(name="up_decode", op="linear", T=32, k=2, N=8, d_in=4096, d_out=14336, dtype="bf16",
             fp8=False, act="swiglu", gather=True, bias=False, residual=False, save=False, skew=0.0),
        # training prefill, gate and up projections in one product, the checkpoint written by its epilogue
        dict(name="up_train", op="linear", T=4096, k=2, N=8, d_in=4096, d_out=14336, dtype="bf16",
             fp8=False, act="swiglu", gather=True, bias=False, residual=False, save=True, skew=0.0),
        # many small experts: the down projection of 256 experts with about 256 ragged rows each, with bias and residual
        dict(name="down_many_experts", op="linear", T=8192, k=8, N=256, d_in=2048, d_out=7168, dtype="bf16",
             fp8=False, act="none", gather=False, bias=True, residual=True, save=False, skew=0.0),
        # a small fp32 layer (the numerics reference of a port): GELU experts with bias
        dict(name="back_small_f32", op="linear_back", T=64, k=2, N=4, d_in=128, d_out=256, dtype="f32",
             act="gelu", gather=True, bias=True, skew=0.0),
        # the backward of up_train from its 8-bit checkpoint
        dict(name="back_train", op="linear_back", T=4096, k=2, N=8, d_in=4096, d_out=14336, dtype="bf16",
             act="swiglu", gather=True, bias=False, skew=0.0),
        # the layer's input kept in 8 bits for the backward
        dict(name="pack_input", op="pack", R=4096, C=4096, dtype="bf16"),
        # reading gate and up activations of a training batch back
        dict(name="unpack_hidden", op="unpack", R=8192, C=28672, dtype="bf16"),
        # weighted sum of eight experts' rows a token, 8192 tokens
        dict(name="combine_prefill", op="combine", T=8192, k=8, N=256, d=7168, dtype="bf16", gated=True),
        # its gradient for top-2 experts: every row's and every gate's
        dict(name="combine_back", op="combine_back", T=4096, k=2, N=8, d=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi):
    return 64 * max(1, _log(rng, lo, hi) // 64)


def draw(rng):
    op = rng.choice(["group", "linear", "linear", "linear", "linear_back", "linear_back", "pack", "unpack",
                     "combine", "combine_back"])
    N = _log(rng, 1, 256)
    k = rng.randint(1, min(N, 8))
    T = _log(rng, 1, 16384)
    skew = rng.choice([0.0, 0.0, 0.6, 1.2])
    if op == "group":
        return dict(op=op, T=T, k=k, N=N, skew=skew, capacity=rng.choice([0, 0, 1 + T * k // N]))
    if op in ("pack", "unpack"):
        C = _dim(rng, 64, 28672)
        R = _log(rng, 1, min(65536, 8192 * 28672 // C))
        return dict(op=op, R=R, C=C, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op in ("combine", "combine_back"):
        d = _dim(rng, 64, 8192)
        T = min(T, max(1, (1 << 28) // (d * k)))
        c = dict(op=op, T=T, k=k, N=N, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "combine":
            c["gated"] = rng.random() < 0.7
        return c
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    act = rng.choice(["none", "relu", "gelu", "silu", "swiglu", "swiglu"])
    d_in, d_out = _dim(rng, 64, 8192), _dim(rng, 64, 8192)
    width = d_out * (2 if act == "swiglu" else 1)
    N = max(1, min(N, (1 << 30) // (d_in * width)))
    k = min(k, N)
    most = 1.5e12 if dtype == "bf16" else 1e11  # operations of a forward; a backward has twice as many
    T = max(1, min(T, int(most / (2.0 * k * d_in * width))))
    c = dict(op=op, T=T, k=k, N=N, d_in=d_in, d_out=d_out, dtype=dtype, act=act, gather=rng.random() < 0.5,
             bias=rng.random() < 0.5, skew=skew)
    if op == "linear":
        c["fp8"] = dtype == "bf16" and rng.random() < 0.3
        c["residual"] = act != "swiglu" and rng.random() < 0.5
        c["save"] = act != "none" and rng.random() < 0.4
    return c


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype, std=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // max(1, math.prod(shape[1:])))  # fp32 temporaries of at most 512 MiB
    for i in range(0, shape[0], step):
        part = torch.randn((min(step, shape[0] - i), *shape[1:]), generator=gen, device="cuda")
        out[i:i + step] = part.mul_(std)
    return out


def _route(gen, c):
    """Experts of every token, distinct, from random scores with a Zipf-shaped offset."""
    score = torch.randn((c["T"], c["N"]), generator=gen, device="cuda")
    score -= c.get("skew", 0.0) * torch.log(torch.arange(1, c["N"] + 1, device="cuda"))
    return torch.topk(score, c["k"], dim=1).indices.to(torch.int32).contiguous()


def _grouped(gen, c):
    """Offsets, source token of every row and row of every slot, as a program has them after grouping."""
    idx = _route(gen, c).reshape(-1).long()
    order = torch.argsort(idx, stable=True)
    counts = torch.bincount(idx, minlength=c["N"])
    offsets = torch.zeros(c["N"] + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.arange(order.numel(), device="cuda")
    return dict(offsets=offsets, row_token=(order // c["k"]).to(torch.int32),
                slot_row=slot_row.to(torch.int32).reshape(c["T"], c["k"]), bounds=offsets.tolist())


def _to_e4m3(x):
    return x.to(torch.float8_e4m3fn)


def _fp8_weights(w):
    """Weights [N, out, in] as E4M3 codes (bytes) and one scale for each output channel."""
    codes = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty(w.shape[:2], device="cuda")
    for i in range(w.shape[0]):
        wf = w[i].float()
        scale[i] = wf.abs().amax(1).clamp_min(_TINY) / _E4M3_MAX
        codes[i] = _to_e4m3(wf / scale[i][:, None]).view(torch.uint8)
    return codes, scale


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case=c)
    op = c["op"]
    if op == "group":
        T, k, N = c["T"], c["k"], c["N"]
        s["idx"] = _route(gen, c)
        s["offsets"] = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
        s["row_token"] = torch.zeros(T * k, dtype=torch.int32, device="cuda")
        s["slot_row"] = torch.zeros((T, k), dtype=torch.int32, device="cuda")
        return s
    dt = _DTYPES[c["dtype"]]
    if op in ("pack", "unpack"):
        x = _normal(gen, (c["R"], c["C"]), dt, 1.5)
        s["codes"] = torch.zeros((c["R"], c["C"]), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.zeros((c["R"], c["C"] // _BLOCK), device="cuda")
        if op == "pack":
            s["x"] = x
        else:
            q, s["scale"] = _pack(x)
            s["codes"] = q.view(torch.uint8)
            s["x"] = torch.empty_like(x)
        return s
    T, k, N = c["T"], c["k"], c["N"]
    g = _grouped(gen, c)
    R = T * k
    s.update(g)
    if op in ("combine", "combine_back"):
        s["rows"] = _normal(gen, (R, c["d"]), dt)
        gate = torch.rand((T, k), generator=gen, device="cuda") + 0.1
        s["gate"] = gate / gate.sum(1, keepdim=True) if c.get("gated", True) else None
        s["y"] = torch.zeros((T, c["d"]), dtype=dt, device="cuda")
        if op == "combine_back":
            s["dy"] = _normal(gen, (T, c["d"]), dt)
            s["drows"] = torch.zeros_like(s["rows"])
            s["dgate"] = torch.zeros((T, k), device="cuda")
        return s
    d_in, d_out = c["d_in"], c["d_out"]
    width = d_out * (2 if c["act"] == "swiglu" else 1)
    s["x"] = _normal(gen, (T if c["gather"] else R, d_in), dt)
    s["w"] = _normal(gen, (N, width, d_in), dt, d_in ** -0.5)
    s["w_scale"] = None
    if c.get("fp8"):
        s["w"], s["w_scale"] = _fp8_weights(s["w"])
    s["bias"] = torch.randn((N, width), generator=gen, device="cuda") * 0.1 if c["bias"] else None
    if op == "linear":
        s["residual"] = _normal(gen, (R, d_out), dt) if c["residual"] else None
        s["y"] = torch.zeros((R, d_out), dtype=dt, device="cuda")
        s["codes"] = s["scale"] = None
        if c["save"]:
            s["codes"] = torch.zeros((R, width), dtype=torch.uint8, device="cuda")
            s["scale"] = torch.zeros((R, width // _BLOCK), device="cuda")
        return s
    s["dy"] = _normal(gen, (R, d_out), dt)
    s["codes"] = s["scale"] = None
    if c["act"] != "none":
        q, s["scale"] = _pack(_normal(gen, (R, width), torch.bfloat16))
        s["codes"] = q.view(torch.uint8)
    s["dx"] = torch.zeros((R, d_in), dtype=dt, device="cuda")
    s["dw"] = torch.zeros((N, width, d_in), dtype=dt, device="cuda")
    s["dbias"] = torch.zeros((N, width), device="cuda") if c["bias"] else None
    return s


# ------------------------------------------------------------------ the plain form
def _pack(x):
    """E4M3 codes of x (as a float8 tensor) and the fp32 scale of each block of 64 columns."""
    v = x.float().reshape(x.shape[0], -1, _BLOCK)
    top = v.abs().amax(2).clamp_min(_TINY)
    q = _to_e4m3(v * (_E4M3_MAX / top)[:, :, None])
    return q.reshape(x.shape), top / _E4M3_MAX


def _unpack(codes, scale):
    v = codes.view(torch.float8_e4m3fn).float().reshape(codes.shape[0], -1, _BLOCK)
    return (v * scale[:, :, None]).reshape(codes.shape)


def _activation(act, z):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "swiglu":
        a, b = z.chunk(2, 1)
        return a * torch.sigmoid(a) * b
    return z


def _activation_back(act, z, dy):
    if act == "relu":
        return dy * (z > 0)
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return dy * (cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    if act == "silu":
        p = torch.sigmoid(z)
        return dy * p * (1 + z * (1 - p))
    a, b = z.chunk(2, 1)
    p = torch.sigmoid(a)
    return torch.cat([dy * b * p * (1 + a * (1 - p)), dy * a * p], 1)


def _plain_group(s):
    c = s["case"]
    T, k, N = c["T"], c["k"], c["N"]
    idx = s["idx"].reshape(-1).long()
    order = torch.argsort(idx, stable=True)
    counts = torch.bincount(idx, minlength=N)
    start = torch.cumsum(counts, 0) - counts
    rank = torch.arange(T * k, device="cuda") - start[idx[order]]
    kept = counts.clamp_max(c["capacity"]) if c["capacity"] else counts
    offsets = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(kept, 0)
    fits = rank < kept[idx[order]]
    row = torch.where(fits, offsets[idx[order]] + rank, -1)
    slot_row = torch.empty(T * k, dtype=torch.int32, device="cuda")
    slot_row[order] = row.to(torch.int32)
    row_token = torch.zeros(T * k + 1, dtype=torch.int32, device="cuda")  # the last entry takes the dropped ones
    row_token[torch.where(fits, row, T * k)] = (order // k).to(torch.int32)
    row_token[T * k] = 0
    return offsets, row_token[:T * k], slot_row.reshape(T, k)


def _plain_linear(s):
    c = s["case"]
    x = s["x"]
    y = torch.zeros_like(s["y"])
    save = c["save"]
    codes = torch.zeros(s["codes"].shape, dtype=torch.float8_e4m3fn, device="cuda") if save else None
    scale = torch.zeros_like(s["scale"]) if save else None
    for e in range(c["N"]):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        if a == b:
            continue
        xe = (x[s["row_token"][a:b].long()] if c["gather"] else x[a:b]).float()
        if c["fp8"]:
            w = s["w"][e].view(torch.float8_e4m3fn).float() * s["w_scale"][e][:, None]
        else:
            w = s["w"][e].float()
        z = xe @ w.t()
        if c["bias"]:
            z = z + s["bias"][e]
        h = _activation(c["act"], z)
        if c["residual"]:
            h = h + s["residual"][a:b].float()
        y[a:b] = h
        if save:
            q, scale[a:b] = _pack(z)
            codes.view(torch.uint8)[a:b] = q.view(torch.uint8)
    return [y] + ([codes, scale] if save else [])


def _plain_linear_back(s):
    c = s["case"]
    dx, dw = torch.zeros_like(s["dx"]), torch.zeros_like(s["dw"])
    dbias = torch.zeros_like(s["dbias"]) if c["bias"] else None
    for e in range(c["N"]):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        if a == b:
            continue
        xe = (s["x"][s["row_token"][a:b].long()] if c["gather"] else s["x"][a:b]).float()
        dz = s["dy"][a:b].float()
        if c["act"] != "none":
            dz = _activation_back(c["act"], _unpack(s["codes"][a:b], s["scale"][a:b]), dz)
        dx[a:b] = dz @ s["w"][e].float()
        dw[e] = dz.t() @ xe
        if c["bias"]:
            dbias[e] = dz.sum(0)
    return [dx, dw] + ([dbias] if c["bias"] else [])


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "group":
        return _plain_group(s)
    if op == "pack":
        return _pack(s["x"])
    if op == "unpack":
        return _unpack(s["codes"], s["scale"]).to(s["x"].dtype)
    if op == "linear":
        return _plain_linear(s)
    if op == "linear_back":
        return _plain_linear_back(s)
    rows = s["rows"][s["slot_row"].reshape(-1).long()].float().reshape(c["T"], c["k"], c["d"])
    if op == "combine":
        if s["gate"] is not None:
            rows = rows * s["gate"][:, :, None]
        return rows.sum(1).to(s["y"].dtype)
    dy = s["dy"].float()
    drows = torch.empty_like(s["drows"])
    drows[s["slot_row"].reshape(-1).long()] = (
        s["gate"][:, :, None] * dy[:, None, :]).reshape(-1, c["d"]).to(drows.dtype)
    return drows, (rows * dy[:, None, :]).sum(2)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import sparse_mixture_experts_router_amd as moe

    c = s["case"]
    op = c["op"]
    if op == "group":
        if "ws" not in s:
            s["ws"] = moe.alloc_group_workspace(c["T"], c["N"], c["k"], "cuda")
        moe.moe_group_rows(s["idx"], c["N"], s["offsets"], s["row_token"], s["slot_row"],
                           capacity=c["capacity"], workspace=s["ws"])
        return s["offsets"], s["row_token"], s["slot_row"]
    if op == "pack":
        moe.moe_checkpoint_pack(s["x"], s["codes"], s["scale"])
        return s["codes"].view(torch.float8_e4m3fn), s["scale"]
    if op == "unpack":
        moe.moe_checkpoint_unpack(s["codes"], s["scale"], s["x"])
        return s["x"]
    if op == "combine":
        moe.moe_combine(s["rows"], s["slot_row"], s["y"], gate=s["gate"])
        return s["y"]
    if op == "combine_back":
        moe.moe_combine_backward(s["rows"], s["slot_row"], s["gate"], s["dy"], s["drows"], s["dgate"])
        return s["drows"], s["dgate"]
    R = c["T"] * c["k"]
    cfg = moe.make_linear_config(R, c["N"], c["d_in"], c["d_out"], dtype=_DTYPES[c["dtype"]],
                                 activation=c["act"], x_rows=c["T"] if c["gather"] else 0,
                                 weight_format=(moe.MOE_WEIGHTS_FP8_E4M3 if c.get("fp8")
                                                else moe.MOE_WEIGHTS_DTYPE))
    index = s["row_token"] if c["gather"] else None
    if op == "linear":
        if "ws" not in s:
            s["ws"] = moe.alloc_linear_workspace(cfg, "cuda")
        moe.moe_grouped_linear(cfg, s["x"], s["offsets"], s["w"], s["y"], row_index=index,
                               w_scale=s["w_scale"], bias=s["bias"], residual=s["residual"],
                               z_codes=s["codes"], z_scale=s["scale"], workspace=s["ws"])
        return [s["y"]] + ([s["codes"].view(torch.float8_e4m3fn), s["scale"]] if c["save"] else [])
    if "ws" not in s:
        s["ws"] = moe.alloc_linear_backward_workspace(cfg, "cuda")
    moe.moe_grouped_linear_backward(cfg, s["x"], s["offsets"], s["w"], s["dy"], row_index=index,
                                    z_codes=s["codes"], z_scale=s["scale"], dx=s["dx"], dw=s["dw"],
                                    dbias=s["dbias"], workspace=s["ws"])
    return [s["dx"], s["dw"]] + ([s["dbias"]] if c["bias"] else [])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work and the definition in 64 bits
def work(case):
    """Bytes and operations that a pass cannot do without (weights of every expert that can have rows)."""
    c = case
    op = c["op"]
    if op == "group":
        n = c["T"] * c["k"]
        return {"bytes": 4.0 * (n + c["N"] + 1 + 2 * n), "flops": 0.0}
    b = 2 if c["dtype"] == "bf16" else 4
    if op in ("pack", "unpack"):
        n = c["R"] * c["C"]
        return {"bytes": float(n * (b + 1) + 4 * n // _BLOCK), "flops": 3.0 * n}
    T, k = c["T"], c["k"]
    R = T * k
    if op == "combine":
        return {"bytes": float((R + T) * c["d"] * b + 4 * R * (2 if c["gated"] else 1)), "flops": 2.0 * R * c["d"]}
    if op == "combine_back":
        return {"bytes": float((2 * R + T) * c["d"] * b + 12 * R), "flops": 3.0 * R * c["d"]}
    width = c["d_out"] * (2 if c["act"] == "swiglu" else 1)
    groups = c["N"] * (1 - (1 - k / c["N"]) ** T)  # experts that get rows, on average
    wb = 1 if c.get("fp8") else b
    x = (T if c["gather"] else R) * c["d_in"] * b
    weights = groups * width * c["d_in"] * wb
    if op == "linear":
        y = R * c["d_out"] * b * (2 if c["residual"] else 1)
        saved = R * width * (1 + 4 / _BLOCK) if c["save"] else 0
        return {"bytes": float(x + weights + y + saved), "flops": 2.0 * R * c["d_in"] * width}
    saved = R * width * (1 + 4 / _BLOCK) if c["act"] != "none" else 0
    grads = R * c["d_in"] * b + c["N"] * width * c["d_in"] * b
    return {"bytes": float(x + weights + R * c["d_out"] * b + saved + grads), "flops": 4.0 * R * c["d_in"] * width}


def _e4m3_value(byte):
    """What an E4M3 byte stands for: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    v = byte.long()
    sign = 1.0 - 2.0 * (v >> 7).double()
    exponent, mantissa = (v >> 3) & 15, (v & 7).double()
    power = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=v.device), (exponent.clamp_min(1) - 7).double())
    value = sign * power * (torch.where(exponent > 0, 1.0, 0.0) + mantissa / 8)
    return torch.where((v & 127) == 127, float("nan"), value)


def _e4m3_nearest(v):
    """v (64 bits, |v| <= 448) to the nearest E4M3 value, ties to the even mantissa."""
    exponent = torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent - 1
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=v.device), (exponent - 3).double())
    return torch.round(v / step) * step


def _blocks64(z):
    v = z.reshape(z.shape[0], -1, _BLOCK)
    top = torch.clamp(v.abs().max(2).values, min=_TINY)
    return _e4m3_nearest(v * (_E4M3_MAX / top).unsqueeze(2)).reshape(z.shape), top / _E4M3_MAX


def _exact_forward(act, z):
    half = z.shape[1] // 2
    if act == "relu":
        return torch.maximum(z, torch.zeros_like(z))
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        return z[:, :half] / (1 + torch.exp(-z[:, :half])) * z[:, half:]
    return z


def _exact_slope(act, z, dy):
    half = z.shape[1] // 2
    if act == "none":
        return dy
    if act == "relu":
        return torch.where(z > 0, dy, torch.zeros_like(dy))
    if act == "gelu":
        return dy * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    g = z if act == "silu" else z[:, :half]
    p = 1 / (1 + torch.exp(-g))
    slope = p + g * p * (1 - p)
    if act == "silu":
        return dy * slope
    return torch.cat((dy * z[:, half:] * slope, dy * g * p), dim=1)


def exact(case, seed):
    c = case
    op = c["op"]
    if op == "group":
        return None
    s = prepare(case, seed)
    if op == "pack":
        return _blocks64(s["x"].double())
    if op == "unpack":
        scale = s["scale"].double().repeat_interleave(_BLOCK, dim=1)
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for i in range(0, c["R"], 1024):  # the 64-bit temporaries of a thousand rows at a time
            out[i:i + 1024] = _e4m3_value(s["codes"][i:i + 1024]) * scale[i:i + 1024]
        return out
    if op in ("combine", "combine_back"):
        T, k, d = c["T"], c["k"], c["d"]
        slot = s["slot_row"].long()
        if op == "combine":
            y = torch.zeros((T, d), dtype=torch.float64, device="cuda")
            for j in range(k):
                g = 1.0 if s["gate"] is None else s["gate"][:, j:j + 1].double()
                y += g * s["rows"][slot[:, j]].double()
            return y
        dy = s["dy"].double()
        drows = torch.zeros((T * k, d), dtype=torch.float64, device="cuda")
        dgate = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        for j in range(k):
            drows[slot[:, j]] = s["gate"][:, j:j + 1].double() * dy
            dgate[:, j] = (s["rows"][slot[:, j]].double() * dy).sum(1)
        return drows, dgate
    bounds, N = s["bounds"], c["N"]
    R = c["T"] * c["k"]
    width = c["d_out"] * (2 if c["act"] == "swiglu" else 1)
    src = s["row_token"].long() if c["gather"] else torch.arange(R, device="cuda")
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if op == "linear":
        y, codes, scale = zeros(R, c["d_out"]), None, None
        if c["save"]:
            codes, scale = zeros(R, width), zeros(R, width // _BLOCK)
        for e in range(N):
            r = slice(bounds[e], bounds[e + 1])
            if r.start == r.stop:
                continue
            w = (_e4m3_value(s["w"][e]) * s["w_scale"][e].double().unsqueeze(1) if c["fp8"]
                 else s["w"][e].double())
            z = torch.matmul(s["x"][src[r]].double(), w.T)
            if c["bias"]:
                z += s["bias"][e].double()
            y[r] = _exact_forward(c["act"], z)
            if c["residual"]:
                y[r] += s["residual"][r].double()
            if c["save"]:
                codes[r], scale[r] = _blocks64(z)
        return [y] + ([codes, scale] if c["save"] else [])
    dx, dw = zeros(R, c["d_in"]), zeros(N, width, c["d_in"])
    dbias = zeros(N, width) if c["bias"] else None
    for e in range(N):
        r = slice(bounds[e], bounds[e + 1])
        if r.start == r.stop:
            continue
        z = None
        if c["act"] != "none":
            z = _e4m3_value(s["codes"][r]) * s["scale"][r].double().repeat_interleave(_BLOCK, dim=1)
        dz = _exact_slope(c["act"], z, s["dy"][r].double())
        dx[r] = torch.matmul(dz, s["w"][e].double())
        dw[e] = torch.matmul(dz.T, s["x"][src[r]].double())
        if c["bias"]:
            dbias[e] = dz.sum(0)
    return [dx, dw] + ([dbias] if c["bias"] else [])
