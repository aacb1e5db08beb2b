"""Cases of the feed-forward block's FP8 operators around the a8w8 GEMM, with
their plain forms:

  rmsnorm   residual addition, root-mean-square norm and FP8 output in one
            call (hq_rmsnorm_fp8): the operand of the next FP8 GEMM
  norm_bwd  its backward pass (hq_rmsnorm_backward): the gradient of the
            residual stream and of the gain
  gemm_act  the a8w8 GEMM with bias, activation and residual in its epilogue
            and, for training, the pre-activation kept as block-wise FP8
            (hq_gemm_a8w8_act)
  act_bwd   the activation's backward pass from that 8-bit checkpoint, with
            the bias gradient (hq_act_backward_fp8)

`run` takes the plain form (f32 torch arithmetic, one rounding at the end)
unless `own` is set, when it calls the library.  FP8 codes come back as
float8 tensors beside their f32 scales.
"""
import math

import torch

own = False

EPS = 1e-5
FMAX = 448.0          # E4M3
Z_BLOCK = 32          # columns per scale of the GEMM's 8-bit checkpoint
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases
def _norm(name, rows, cols, dtype, wdtype, residual, block, y_out):
    return {"name": name, "op": "rmsnorm", "rows": rows, "cols": cols, "dtype": dtype, "wdtype": wdtype,
            "residual": residual, "block": block, "y_out": y_out}


def _norm_bwd(name, rows, cols, dtype, wdtype, dres):
    return {"name": name, "op": "norm_bwd", "rows": rows, "cols": cols, "dtype": dtype, "wdtype": wdtype,
            "dres": dres}


def _gemm(name, m, n, k, act, bias, residual, ckpt):
    return {"name": name, "op": "gemm_act", "m": m, "n": n, "k": k, "act": act, "bias": bias,
            "residual": residual, "ckpt": ckpt}


def _act_bwd(name, rows, cols, dtype, act, block, dbias):
    return {"name": name, "op": "act_bwd", "rows": rows, "cols": cols, "dtype": dtype, "act": act,
            "block": block, "dbias": dbias}


def listed():
    return [
        # one decode step of 16 sequences: the norm ahead of the layer's first GEMM, where launch latency counts
        _norm("norm_decode16", 16, 8192, "bf16", "bf16", True, 0, False),
        # the large layer's input, residual stream in and out, one scale per token
        _norm("norm_large", 16384, 8192, "bf16", "bf16", True, 0, False),
        # a ragged batch normed into block-wise codes for the block-scaled GEMM, the normed values kept for training
        _norm("norm_block_ragged", 5003, 1408, "f16", "f32", False, 32, True),
        # backward of the norm at the linear stack's width
        _norm_bwd("norm_bwd_stack", 2048, 1024, "bf16", "bf16", True),
        # backward of the large layer's norm
        _norm_bwd("norm_bwd_large", 16384, 8192, "bf16", "bf16", True),
        # a master-precision backward with a ragged width and no residual gradient
        _norm_bwd("norm_bwd_f32_ragged", 777, 4100, "f32", "f32", False),
        # decode, one sequence: the down projection added to the residual stream
        _gemm("down_decode1", 1, 8192, 28672, "none", True, True, False),
        # decode, 16 sequences: the up projection with its activation
        _gemm("up_decode16", 16, 28672, 8192, "gelu_tanh", True, False, False),
        # the linear stack's down projection, a ragged batch
        _gemm("stack_down_ragged", 2047, 1024, 4096, "silu", False, True, False),
        # training, the large layer's up projection: activation and the 8-bit checkpoint of what it was applied to
        _gemm("up_train_large", 16384, 28672, 8192, "gelu", True, False, True),
        # the stack's activation backward
        _act_bwd("act_bwd_stack", 2047, 4096, "f16", "silu", 128, False),
        # the large layer's activation backward with the bias gradient
        _act_bwd("act_bwd_large", 16384, 28672, "bf16", "gelu", 32, True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["rmsnorm", "norm_bwd", "gemm_act", "act_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "rmsnorm":
        block = rng.choice([0, 0, 32, 64, 128])
        cols = _log_int(rng, 64, 28672, 16 if block else rng.choice([1, 8, 64]))
        rows = _log_int(rng, 1, min(16384, 16384 * 8192 // cols))
        c = _norm("", rows, cols, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.7, block, rng.random() < 0.3)
    elif op == "norm_bwd":
        cols = _log_int(rng, 64, 28672, rng.choice([1, 8, 64]))
        rows = _log_int(rng, 1, min(16384, 16384 * 8192 // cols))
        c = _norm_bwd("", rows, cols, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.7)
    elif op == "gemm_act":
        ckpt = rng.random() < 0.4
        m = _log_int(rng, 1, 8192)
        n = _log_int(rng, 64, 28672, 32 if ckpt else 8)
        # the checkpoint belongs to an up projection, whose K is the model's width
        k = _log_int(rng, 64, min(8192 if ckpt else 28672, max(64, (1 << 40) // (m * n))), 16)
        c = _gemm("", m, n, k, rng.choice(sorted(ACTS)), rng.random() < 0.6, rng.random() < 0.5, ckpt)
    else:
        cols = _log_int(rng, 64, 28672, 16)
        rows = _log_int(rng, 1, 16384)
        c = _act_bwd("", rows, cols, dtype, rng.choice(["relu", "gelu", "gelu_tanh", "silu"]),
                     rng.choice([32, 64, 128]), rng.random() < 0.6)
    c.pop("name")
    return c


# ------------------------------------------------------------------ inputs
def _blocks(t, block):
    """t [rows, cols] as [rows, blocks, block], the last block filled up with zeros."""
    rows, cols = t.shape
    nb = -(-cols // block)
    if nb * block != cols:
        full = t.new_zeros((rows, nb * block))
        full[:, :cols] = t
        t = full
    return t.reshape(rows, nb, block)


def _quantize(y, block):
    """E4M3 codes of f32 y and f32 dequant scales [rows, blocks]; block 0: one per row."""
    rows, cols = y.shape
    b = _blocks(y, block or cols)
    amax = b.abs().amax(-1)
    m = FMAX / amax
    m = torch.where(torch.isfinite(m), m, torch.ones_like(m))
    q = (b * m[..., None]).clamp(-FMAX, FMAX).to(torch.float8_e4m3fn).reshape(rows, -1)[:, :cols].contiguous()
    s = 1.0 / m
    return q, s if block else s.reshape(rows)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(std)

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=dev)

    s = dict(case)
    op = case["op"]
    if op in ("rmsnorm", "norm_bwd"):
        rows, cols = case["rows"], case["cols"]
        t, wt = DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        s["weight"] = normal((cols,), 0.1).add_(1.0).to(wt)
        # a residual stream: a few channels carry values far above the rest
        chan = 1.0 + 15.0 * (torch.rand((cols,), generator=gen, device=dev) < 0.005).float()
        if op == "rmsnorm":
            s["x"] = normal((rows, cols)).to(t)
            s["residual"] = (normal((rows, cols), 2.0) * chan).to(t) if case["residual"] else None
            s["q"] = empty((rows, cols), torch.uint8)
            nb = -(-cols // case["block"]) if case["block"] else 0
            s["scales"] = empty((rows, nb) if nb else (rows,), torch.float32)
            s["h_out"] = empty((rows, cols), t) if case["residual"] else None
            s["y"] = empty((rows, cols), t) if case["y_out"] else None
            s["rstd"] = empty((rows,), torch.float32)
        else:
            s["h"] = (normal((rows, cols), 2.0) * chan).to(t)
            s["dy"] = normal((rows, cols), 1e-2).to(t)
            s["dres"] = normal((rows, cols), 1e-2).to(t) if case["dres"] else None
            s["rstd"] = 1.0 / torch.sqrt((s["h"].float() ** 2).mean(-1) + EPS)
            s["dx"] = empty((rows, cols), t)
            s["dweight"] = empty((cols,), wt)
    elif op == "gemm_act":
        m, n, k = case["m"], case["n"], case["k"]
        xq, s["x_scale"] = _quantize(normal((m, k)), 0)
        wq, s["w_scale"] = _quantize(normal((n, k), 0.02), 0)
        s["xq"], s["wq"] = xq.view(torch.uint8), wq.view(torch.uint8)
        s["bias_t"] = normal((n,), 0.3).to(torch.bfloat16) if case["bias"] else None
        s["res"] = normal((m, n)).to(torch.bfloat16) if case["residual"] else None
        s["out"] = empty((m, n), torch.bfloat16)
        s["zq"] = empty((m, n), torch.uint8) if case["ckpt"] else None
        s["zs"] = empty((m, n // Z_BLOCK), torch.float32) if case["ckpt"] else None
    else:
        rows, cols = case["rows"], case["cols"]
        t = DTYPES[case["dtype"]]
        zq, s["zs"] = _quantize(normal((rows, cols), 1.5), case["block"])
        s["zq"] = zq.view(torch.uint8)
        s["g"] = normal((rows, cols), 1e-2).to(t)
        s["dz"] = empty((rows, cols), t)
        s["db"] = empty((cols,), t) if case["dbias"] else None
    return s


# -------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
        return 0.5 * z * (1.0 + torch.tanh(u))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * z * z)
    sg = 1.0 / (1.0 + torch.exp(-z))
    return sg * (1.0 + z * (1.0 - sg))


def _plain_rmsnorm(s):
    t = DTYPES[s["dtype"]]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(-1) + EPS)
    y = h * rstd[:, None] * s["weight"].float()
    q, scales = _quantize(y, s["block"])
    return {"q": q, "scales": scales, "rstd": rstd, "h": h.to(t) if s["residual"] is not None else None,
            "y": y.to(t) if s["y_out"] else None}


def _plain_norm_bwd(s):
    t = DTYPES[s["dtype"]]
    dy, w = s["dy"].float(), s["weight"].float()
    xhat = s["h"].float() * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(t), "dweight": (dy * xhat).sum(0).to(s["weight"].dtype)}


def _plain_gemm_act(s):
    x = s["xq"].view(torch.float8_e4m3fn).float()
    w = s["wq"].view(torch.float8_e4m3fn).float()
    z = (x @ w.t()) * s["x_scale"][:, None] * s["w_scale"][None, :]
    if s["bias_t"] is not None:
        z = z + s["bias_t"].float()
    out = _act(z, s["act"])
    if s["res"] is not None:
        out = out + s["res"].float()
    r = {"out": out.to(torch.bfloat16)}
    if s["ckpt"]:
        r["zq"], r["zs"] = _quantize(z, Z_BLOCK)
    return r


def _plain_act_bwd(s):
    rows, cols = s["zq"].shape
    z = _blocks(s["zq"].view(torch.float8_e4m3fn).float(), s["block"]) * s["zs"][..., None]
    z = z.reshape(rows, -1)[:, :cols]
    dz = s["g"].float() * _act_grad(z, s["act"])
    return {"dz": dz.to(s["g"].dtype), "db": dz.sum(0).to(s["g"].dtype) if s["dbias"] else None}


def _own_run(s):
    import fp8_dynamic_quantization_amax_b200 as hq
    f8 = torch.float8_e4m3fn
    op = s["op"]
    if op == "rmsnorm":
        q, scales, h = hq.hq_rmsnorm_fp8(s["x"], s["weight"], EPS, residual=s["residual"], fmt=hq.E4M3,
                                         block=s["block"], q=s["q"], scales=s["scales"], residual_out=s["h_out"],
                                         y_out=s["y"], rstd_out=s["rstd"])
        return {"q": q.view(f8), "scales": scales, "rstd": s["rstd"], "h": h if s["residual"] is not None else None,
                "y": s["y"]}
    if op == "norm_bwd":
        dx, dw = hq.hq_rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dres=s["dres"], dx=s["dx"],
                                        dweight=s["dweight"])
        return {"dx": dx, "dweight": dw}
    if op == "gemm_act":
        r = hq.hq_gemm_a8w8_act(s["xq"], s["wq"], s["x_scale"], s["w_scale"], hq.E4M3, bias=s["bias_t"],
                                act=ACTS[s["act"]], residual=s["res"], out=s["out"], z_q=s["zq"], z_scales=s["zs"])
        if not s["ckpt"]:
            return {"out": r}
        return {"out": r[0], "zq": r[1].view(f8), "zs": r[2]}
    dz, db = hq.hq_act_backward_fp8(s["g"], s["zq"], s["zs"], ACTS[s["act"]], fmt=hq.E4M3, block=s["block"],
                                    dz=s["dz"], dbias=s["db"], need_dbias=s["dbias"])
    return {"dz": dz, "db": db}


def run(state):
    if own:
        return _own_run(state)
    return {"rmsnorm": _plain_rmsnorm, "norm_bwd": _plain_norm_bwd, "gemm_act": _plain_gemm_act,
            "act_bwd": _plain_act_bwd}[state["op"]](state)


# ------------------------------------------------------------ what it needs
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    op = case["op"]
    if op == "rmsnorm":
        n, e = case["rows"] * case["cols"], size[case["dtype"]]
        per = e + (2 * e if case["residual"] else 0) + 1 + (e if case["y_out"] else 0)
        ns = case["rows"] * (-(-case["cols"] // case["block"]) if case["block"] else 1)
        return {"bytes": n * per + 4 * ns + 4 * case["rows"] + case["cols"] * size[case["wdtype"]], "flops": 8 * n}
    if op == "norm_bwd":
        n, e = case["rows"] * case["cols"], size[case["dtype"]]
        return {"bytes": n * e * (4 if case["dres"] else 3) + 4 * case["rows"] + 2 * case["cols"] * size[case["wdtype"]],
                "flops": 10 * n}
    if op == "gemm_act":
        m, n, k = case["m"], case["n"], case["k"]
        b = m * k + n * k + 4 * (m + n) + 2 * m * n
        b += (2 * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
        b += m * n + 4 * m * (n // Z_BLOCK) if case["ckpt"] else 0
        return {"bytes": b, "flops": 2 * m * n * k}
    n, e = case["rows"] * case["cols"], size[case["dtype"]]
    ns = case["rows"] * -(-case["cols"] // case["block"])
    return {"bytes": n * (2 * e + 1) + 4 * ns + (case["cols"] * e if case["dbias"] else 0), "flops": 15 * n}


# ----------------------------------------------------------- 64-bit oracle
def _exact_quantized(y, block):
    """What the codes stand for before their rounding, and the dequant scales, in 64 bits."""
    cols = y.shape[1]
    width = block if block else cols
    group = torch.arange(cols, device=y.device) // width
    top = torch.zeros((y.shape[0], int(group[-1]) + 1), dtype=y.dtype, device=y.device)
    top.scatter_reduce_(1, group.expand(y.shape[0], cols), y.abs(), "amax")
    scale = torch.where(top > 0, top / FMAX, torch.ones_like(top))
    return y / scale[:, group], (scale if block else scale[:, 0])


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    op = case["op"]
    if op == "rmsnorm":
        h = s["x"].to(d)
        if case["residual"]:
            h = h + s["residual"].to(d)
        rstd = (h.square().sum(1) / case["cols"] + EPS).rsqrt()
        y = (h * s["weight"].to(d)) * rstd.unsqueeze(1)
        q, scales = _exact_quantized(y, case["block"])
        return {"q": q, "scales": scales, "rstd": rstd, "h": h if case["residual"] else None,
                "y": y if case["y_out"] else None}
    if op == "norm_bwd":
        dy, h, w, r = s["dy"].to(d), s["h"].to(d), s["weight"].to(d), s["rstd"].to(d).unsqueeze(1)
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = dy * w * r - h * (r ** 3) * dot / case["cols"]
        if case["dres"]:
            dx = dx + s["dres"].to(d)
        return {"dx": dx, "dweight": (dy * h * r).sum(0)}
    if op == "gemm_act":
        z = torch.matmul(s["xq"].view(torch.float8_e4m3fn).to(d), s["wq"].view(torch.float8_e4m3fn).to(d).t())
        z.mul_(s["x_scale"].to(d).unsqueeze(1)).mul_(s["w_scale"].to(d))
        if case["bias"]:
            z.add_(s["bias_t"].to(d))
        out = _exact_act(z, case["act"])
        if case["residual"]:
            out = out + s["res"].to(d)
        r = {"out": out}
        if case["ckpt"]:
            r["zq"], r["zs"] = _exact_quantized(z, Z_BLOCK)
        return r
    group = torch.arange(case["cols"], device="cuda") // case["block"]
    z = s["zq"].view(torch.float8_e4m3fn).to(d)
    z.mul_(s["zs"].to(d)[:, group])
    dz = _exact_slope(z, case["act"]).mul_(s["g"].to(d))
    return {"dz": dz, "db": dz.sum(0) if case["dbias"] else None}


def _exact_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def _exact_slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if act == "silu":
        return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    du = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
    return torch.sigmoid(u) + z * du * torch.sigmoid(u) * torch.sigmoid(-u)
