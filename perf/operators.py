"""Cases that measure the layer operators around the NVFP4 products.

The operators are those of one pre-norm linear block trained or served in NVFP4:
add + RMS norm with a quantized output, its backward pass, the NVFP4 product with bias,
activation and residual in its epilogue, the backward pass of bias and activation, and
the clipping of a list of gradients by their global norm.

`run` computes an operator either in its plain form (elementary torch operations in
FP32, rounded once at the end) or, where `own` is true, through this package's entry
points.  `exact` evaluates the definitions in FP64.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
EPS = 1e-5
E4M3_MAX = 448.0
BOUND = 448.0          # E4M3 bound of the NVFP4 operands
FACTOR = BOUND * 6.0   # amax of a line over the value of its largest code and scale
GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715
SCALE_BLOCK = 128      # columns per scale of the blockwise 8-bit output
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token's hidden state, quantized for the next product
        dict(name="norm_token", kind="norm", rows=1, cols=8192, dtype="bf16", residual=True,
             out="fp8_row"),
        # the activations of the linear layer of the benchmark
        dict(name="norm_train", kind="norm", rows=16384, cols=8192, dtype="bf16", residual=True,
             out="fp8_row"),
        # a row count and a row length that no tile divides, an FP32 residual stream
        dict(name="norm_ragged", kind="norm", rows=4000, cols=5000, dtype="fp32", residual=True,
             out="fp8_block"),
        # the same layer's norm backward, with the gradient of the residual stream
        dict(name="norm_backward_train", kind="norm_backward", rows=16384, cols=8192,
             dtype="bf16", dh=True),
        # a first layer: no gradient arrives beside the norm's
        dict(name="norm_backward_ragged", kind="norm_backward", rows=4000, cols=5000,
             dtype="fp32", dh=False),
        # the linear layer's weight applied to one decoded token
        dict(name="linear_token", kind="linear", m=1, n=28672, k=8192, bias=True, act="silu",
             residual=False, save_z=False, out="bf16"),
        # its training step's forward product; the pre-activation is kept for the backward
        dict(name="linear_train", kind="linear", m=16384, n=28672, k=8192, bias=True, act="gelu",
             residual=False, save_z=True, out="bf16"),
        # a prompt of 300 tokens: norm into NVFP4, then the product back into the stream
        dict(name="norm_linear_prompt", kind="norm_linear", m=300, n=2048, k=7168, bias=True,
             act="none", residual=True, out="bf16"),
        # the gradient of the linear layer's activation and bias, with the maxima that the
        # quantization of dz takes
        dict(name="act_backward_train", kind="act_backward", rows=16384, cols=28672,
             dtype="bf16", act="gelu"),
        dict(name="act_backward_ragged", kind="act_backward", rows=4000, cols=5000,
             dtype="fp32", act="silu"),
        # the vectors and small matrices of a model, BF16 and FP32 side by side
        dict(name="clip_small", kind="clip", count=48, total=1_000_003, dtype="mixed"),
        # the gradients of a few layers of large matrices
        dict(name="clip_train", kind="clip", count=12, total=973_000_000, dtype="bf16"),
    ]


def _size(rng, lo, hi, multiple=1):
    """A size whose logarithm is uniform between lo and hi."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / multiple)) * multiple
    n = max(lo, min(hi, n))
    return n - multiple if n == 3072 else n


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_backward", "linear", "linear", "norm_linear",
                       "act_backward", "clip"])
    if kind in ("norm", "norm_backward"):
        cols = _size(rng, 64, 16384, rng.choice([1, 8, 128]))
        rows = _size(rng, 1, min(16384, 134_000_000 // cols))
        c = dict(kind=kind, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp32"]))
        if kind == "norm":
            c.update(residual=rng.random() < 0.75, out=rng.choice(["fp8_row", "fp8_block", "y"]))
        else:
            c.update(dh=rng.random() < 0.5)
        return c
    if kind in ("linear", "norm_linear"):
        n, k = _size(rng, 64, 28672, rng.choice([1, 8, 64])), _size(rng, 64, 8192, 32)
        m = _size(rng, 1, 64) if rng.random() < 0.4 else _size(rng, 64, 8192)
        c = dict(kind=kind, m=m, n=n, k=k, bias=rng.random() < 0.75,
                 act=rng.choice(["none", "relu", "gelu", "silu"]),
                 residual=rng.random() < 0.5, out="bf16")
        if kind == "linear":
            c.update(save_z=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "fp32"]))
        return c
    if kind == "act_backward":
        cols = _size(rng, 64, 28672, rng.choice([1, 8, 128]))
        rows = _size(rng, 1, min(16384, 235_000_000 // cols))
        return dict(kind=kind, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    act=rng.choice(["none", "relu", "gelu", "silu"]))
    return dict(kind="clip", count=rng.randint(1, 48), total=_size(rng, 100_003, 400_000_000),
                dtype=rng.choice(["bf16", "fp32", "mixed"]))


def _clip_sizes(case):
    """Sizes of a gradient list: matrices and vectors of a model, far apart in size."""
    r = random.Random(case["count"] * 1_000_003 + case["total"])
    w = [math.exp(r.uniform(0.0, 6.0)) for _ in range(case["count"])]
    left, sizes = case["total"] - case["count"], []
    for x in w[:-1]:
        sizes.append(1 + int(left * x / sum(w)))
    return sizes + [case["total"] - sum(sizes)]


def _clip_dtype(case, i):
    return DTYPES[case["dtype"] if case["dtype"] != "mixed" else ("bf16", "fp32")[i % 2]]


# ---------------------------------------------------------------- NVFP4 in torch

def _e2m1_codes(v):
    """Codes of the nearest E2M1 values (ties to the even code), as int32."""
    a = v.abs()
    code = ((a > 0.25).to(torch.int32) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    return code + 8 * torch.signbit(v)


def _e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quantize_rows(x):
    """Codes (one per element, int32), E4M3 block scales (as FP32) and amax of the rows of
    the FP32 x: row-scaled NVFP4 with 1x16 blocks."""
    rows, cols = x.shape
    amax = x.abs().amax(dim=1)
    s = torch.where(amax > 0, FACTOR / amax, torch.ones_like(amax))
    blocks = x.reshape(rows, cols // 16, 16)
    scale = _e4m3(blocks.abs().amax(dim=2) / 6.0 * s[:, None]).float()
    enc = torch.where(scale > 0, s[:, None] / scale, torch.zeros_like(scale))
    codes = _e2m1_codes(blocks * enc[:, :, None]).reshape(rows, cols)
    return codes, scale, amax


def _operand(rows, cols, generator, std):
    """A row-scaled NVFP4 operand of normal values: packed codes, scale bytes, amax."""
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=DEVICE)
    scales = torch.empty(rows, cols // 16, dtype=torch.uint8, device=DEVICE)
    amax = torch.empty(rows, dtype=torch.float32, device=DEVICE)
    for r in range(0, rows, 4096):
        x = torch.randn(min(4096, rows - r), cols, generator=generator, device=DEVICE) * std
        c, s, a = _quantize_rows(x)
        codes[r:r + 4096] = (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8)
        scales[r:r + 4096] = _e4m3(s).view(torch.uint8)
        amax[r:r + 4096] = a
    return codes, scales, amax


def _code_values(dtype):
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(mags + [-m for m in mags], dtype=dtype, device=DEVICE)


def _pair_values(dtype):
    """[256][2]: the two E2M1 values of each code byte, low nibble first."""
    v, byte = _code_values(dtype), torch.arange(256, device=DEVICE)
    return torch.stack([v[byte & 15], v[byte >> 4]], dim=1)


def _dequantize(codes, scales, amax):
    """FP32 values of an NVFP4 operand: code * decode(scale) * (amax / FACTOR)."""
    rows = codes.shape[0]
    v = _pair_values(torch.float32)[codes.int()].reshape(rows, -1, 16)
    d = scales.view(torch.float8_e4m3fn).float() * (amax * (1.0 / FACTOR))[:, None]
    return (v * d[:, :, None]).reshape(rows, -1)


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _stream_values(rows, cols, g, dtype):
    """A residual stream: rows of different magnitude, a few channels much larger."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEVICE))
    channel = torch.rand(cols, generator=g, device=DEVICE)
    return x.mul_(1.0 + 20.0 * (channel > 0.999)).to(dtype)


def _normal(shape, g, std, dtype):
    return (torch.randn(shape, generator=g, device=DEVICE) * std).to(dtype)


def prepare(case, seed):
    g, kind, s = _generator(seed), case["kind"], dict(case)
    if kind in ("norm", "norm_backward"):
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device=DEVICE)).to(dt)
        if kind == "norm":
            s["x"] = _stream_values(rows, cols, g, dt)
            s["rstd"] = torch.empty(rows, device=DEVICE)
            if case["residual"]:
                s["skip"] = _stream_values(rows, cols, g, dt)
                s["h"] = torch.empty_like(s["x"])
            if case["out"] == "y":
                s["y"] = torch.empty_like(s["x"])
            else:
                per_row = 1 if case["out"] == "fp8_row" else -(-cols // SCALE_BLOCK)
                s["codes"] = torch.empty(rows, cols, dtype=torch.uint8, device=DEVICE)
                s["scale"] = torch.empty(rows, per_row, device=DEVICE)
        else:
            s["h"] = _stream_values(rows, cols, g, dt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + EPS)
            s["dy"] = _normal((rows, cols), g, 0.01, dt)
            if case["dh"]:
                s["grad_h"] = _normal((rows, cols), g, 0.01, dt)
            s["dx"] = torch.empty_like(s["h"])
            s["dweight"] = torch.empty(cols, device=DEVICE)
            s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEVICE)
    elif kind in ("linear", "norm_linear"):
        m, n, k, dt = case["m"], case["n"], case["k"], DTYPES[case["out"]]
        s["w"] = _operand(n, k, g, 0.02)
        if kind == "linear":
            s["a"] = _operand(m, k, g, 1.0)
        else:
            s["x"], s["skip"] = (_stream_values(m, k, g, torch.bfloat16) for _ in range(2))
            s["weight"] = (1.0 + 0.1 * torch.randn(k, generator=g, device=DEVICE)).bfloat16()
            s["h"] = torch.empty_like(s["x"])
            s["rstd"] = torch.empty(m, device=DEVICE)
            s["a"] = (torch.empty(m, k // 2, dtype=torch.uint8, device=DEVICE),
                      torch.empty(m, k // 16, dtype=torch.uint8, device=DEVICE),
                      torch.empty(m, device=DEVICE))
        s["bias_values"] = _normal((n,), g, 0.1, torch.float32) if case["bias"] else None
        s["add"] = _normal((m, n), g, 1.0, dt) if case["residual"] else None
        s["d"] = torch.empty(m, n, dtype=dt, device=DEVICE)
        s["z"] = torch.empty_like(s["d"]) if case.get("save_z") else None
        s["workspace"] = torch.empty((256 << 20) + 4 * (m + n) * k // 8, dtype=torch.uint8,
                                     device=DEVICE)
    elif kind == "act_backward":
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["z"] = _normal((rows, cols), g, 1.5, dt)
        s["dd"] = _normal((rows, cols), g, 0.01, dt)
        s["dz"] = torch.empty_like(s["z"])
        s["dbias"] = torch.empty(cols, device=DEVICE)
        s["amax"] = torch.empty(rows + cols, device=DEVICE)  # of the rows, of the columns
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEVICE)
    else:
        s["grads"] = [_normal((n,), g, 0.02, _clip_dtype(case, i))
                      for i, n in enumerate(_clip_sizes(case))]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = torch.empty(1, device=DEVICE)
        s["max_norm"] = 1.0
        s["workspace"] = torch.empty(1 << 20, dtype=torch.uint8, device=DEVICE)
    return s


# ---------------------------------------------------------------- plain forms

def _norm_plain(s):
    h = s["x"].float() + s["skip"].float() if s.get("skip") is not None else s["x"].float()
    rstd = torch.rsqrt(h.square().mean(dim=1) + EPS)
    return h, rstd, h * s["weight"].float() * rstd[:, None]


def _plain_norm(s):
    h, rstd, y = _norm_plain(s)
    r = {"rstd": rstd}
    if s["residual"]:
        r["h"] = h.to(s["x"].dtype)
    if s["out"] == "y":
        r["y"] = y.to(s["x"].dtype)
        return r
    rows, cols = y.shape
    block = cols if s["out"] == "fp8_row" else SCALE_BLOCK
    padded = torch.nn.functional.pad(y, (0, -cols % block)).reshape(rows, -1, block)
    amax = padded.abs().amax(dim=2)
    r["scale"] = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    codes = _e4m3(padded / r["scale"][:, :, None]).reshape(rows, -1)
    r["codes"] = codes[:, :cols].contiguous()
    return r


def _plain_norm_backward(s):
    dy, n = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = (g - n * (g * n).mean(dim=1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"]:
        dx = dx + s["grad_h"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * n).sum(dim=0)}


def _act_plain(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + GELU_A * z * z * z)))
    return z * torch.sigmoid(z) if act == "silu" else z


def _plain_linear(s, a, w):
    z = torch.matmul(a, w.t())
    if s["bias"]:
        z = z + s["bias_values"]
    d = _act_plain(z, s["act"])
    if s["residual"]:
        d = d + s["add"].float()
    r = {"d": d.to(s["d"].dtype)}
    if s["z"] is not None:
        r["z"] = z.to(s["d"].dtype)
    return r


def _plain_norm_linear(s):
    h, rstd, y = _norm_plain(s)
    codes, scale, amax = _quantize_rows(y)
    v = _code_values(torch.float32)[codes].reshape(*scale.shape, 16)
    a = v * (scale * (amax * (1.0 / FACTOR))[:, None])[:, :, None]
    r = _plain_linear(s, a.reshape(y.shape), _dequantize(*s["w"]))
    return dict(r, h=h.to(s["x"].dtype), rstd=rstd, amax=amax)


def _plain_act_backward(s):
    z, dd, act = s["z"].float(), s["dd"].float(), s["act"]
    if act == "relu":
        dd = dd * (z > 0)
    elif act == "gelu":
        t = torch.tanh(GELU_C * (z + GELU_A * z * z * z))
        dd = dd * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * z * z))
    elif act == "silu":
        sig = torch.sigmoid(z)
        dd = dd * (sig * (1 + z * (1 - sig)))
    dz = dd.to(s["z"].dtype)
    a = dz.abs()
    return {"dz": dz, "dbias": dd.sum(dim=0), "amax": torch.cat([a.amax(dim=1), a.amax(dim=0)])}


def _plain_clip(s):
    norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm.reshape(1), "grads": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


# ---------------------------------------------------------------- the framework's operators

def _own_norm(s):
    import nvfp4_precision_quantization_gb300 as nv
    r = {"rstd": s["rstd"]}
    fp8 = None
    if s["out"] != "y":
        fp8 = nv.Fp8Out(s["codes"], s["scale"], 0 if s["out"] == "fp8_row" else SCALE_BLOCK)
        r.update(codes=s["codes"].view(torch.float8_e4m3fn), scale=s["scale"])
    nv.nvfp4_add_rmsnorm(s["x"], s["weight"], EPS, residual=s.get("skip"), h=s.get("h"),
                         y=s.get("y"), rstd=s["rstd"], fp8=fp8)
    r.update({k: s[k] for k in ("h", "y") if k in s})
    return r


def _own_norm_backward(s):
    import nvfp4_precision_quantization_gb300 as nv
    nv.nvfp4_add_rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"],
                                  dweight=s["dweight"], dh=s.get("grad_h"),
                                  workspace=s["workspace"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_linear(s):
    import nvfp4_precision_quantization_gb300 as nv
    r = {}
    if s["kind"] == "norm_linear":
        nv.nvfp4_add_rmsnorm(s["x"], s["weight"], EPS, residual=s["skip"], h=s["h"],
                             rstd=s["rstd"], row=nv.Out(*s["a"]),
                             cfg=nv.Config(nv.NVFP4_ROW_SCALED, BOUND, 0, 0))
        r = {"h": s["h"], "rstd": s["rstd"], "amax": s["a"][2]}
    act = {"none": nv.NVFP4_ACT_NONE, "relu": nv.NVFP4_ACT_RELU, "gelu": nv.NVFP4_ACT_GELU,
           "silu": nv.NVFP4_ACT_SILU}[s["act"]]
    nv.nvfp4_gemm_bias_act(nv.Operand(*s["a"], nv.NVFP4_ROW_SCALED, BOUND),
                           nv.Operand(*s["w"], nv.NVFP4_ROW_SCALED, BOUND), s["d"],
                           bias=s["bias_values"], act=act, residual=s["add"], z=s["z"],
                           workspace=s["workspace"])
    r["d"] = s["d"]
    if s["z"] is not None:
        r["z"] = s["z"]
    return r


def _own_act_backward(s):
    import nvfp4_precision_quantization_gb300 as nv
    act = {"none": nv.NVFP4_ACT_NONE, "relu": nv.NVFP4_ACT_RELU, "gelu": nv.NVFP4_ACT_GELU,
           "silu": nv.NVFP4_ACT_SILU}[s["act"]]
    rows = s["rows"]
    nv.nvfp4_bias_act_backward(s["dd"], s["z"], act, s["dz"], dbias=s["dbias"],
                               row_amax=s["amax"][:rows], col_amax=s["amax"][rows:],
                               workspace=s["workspace"])
    # the maxima of values of dz's type are values of that type
    return {"dz": s["dz"], "dbias": s["dbias"], "amax": s["amax"].to(s["dz"].dtype)}


def _own_clip(s):
    import nvfp4_precision_quantization_gb300 as nv
    nv.nvfp4_clip_grad_norm(s["grads"], s["max_norm"], s["norm"], out=s["out"],
                            workspace=s["workspace"])
    return {"norm": s["norm"], "grads": s["out"]}


def run(state):
    kind = state["kind"]
    if own:
        return {"norm": _own_norm, "norm_backward": _own_norm_backward, "linear": _own_linear,
                "norm_linear": _own_linear, "act_backward": _own_act_backward,
                "clip": _own_clip}[kind](state)
    if kind == "linear":
        return _plain_linear(state, _dequantize(*state["a"]), _dequantize(*state["w"]))
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward,
            "norm_linear": _plain_norm_linear, "act_backward": _plain_act_backward,
            "clip": _plain_clip}[kind](state)


# ---------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    if kind == "norm":
        n, b = case["rows"] * case["cols"], BYTES[case["dtype"]]
        bytes_ = n * b * (3 if case["residual"] else 1) + case["cols"] * b + 4 * case["rows"]
        if case["out"] == "y":
            bytes_ += n * b
        else:
            blocks = 1 if case["out"] == "fp8_row" else -(-case["cols"] // SCALE_BLOCK)
            bytes_ += n + 4 * case["rows"] * blocks
        return {"bytes": bytes_, "flops": 6 * n}
    if kind == "norm_backward":
        n, b = case["rows"] * case["cols"], BYTES[case["dtype"]]
        return {"bytes": n * b * (4 if case["dh"] else 3) + case["cols"] * (b + 4)
                + 4 * case["rows"], "flops": 10 * n}
    if kind in ("linear", "norm_linear"):
        m, n, k = case["m"], case["n"], case["k"]
        line = k // 2 + k // 16 + 4
        bytes_ = n * line + BYTES[case["out"]] * m * n * (
            1 + bool(case["residual"]) + bool(case.get("save_z"))) + (4 * n if case["bias"] else 0)
        bytes_ += m * line if kind == "linear" else 6 * m * k + 2 * k + 8 * m
        return {"bytes": bytes_, "flops": 2 * m * n * k}
    if kind == "act_backward":
        n = case["rows"] * case["cols"]
        return {"bytes": n * BYTES[case["dtype"]] * (2 if case["act"] == "none" else 3)
                + 4 * case["rows"] + 8 * case["cols"], "flops": 12 * n}
    sizes = _clip_sizes(case)
    return {"bytes": 4 + sum(2 * n * torch.empty((), dtype=_clip_dtype(case, i)).element_size()
                             for i, n in enumerate(sizes)), "flops": 3 * case["total"]}


# ---------------------------------------------------------------- 64 bits

def _round64(x, mantissa, lowest, largest):
    """x rounded to `mantissa` fraction bits with the exponent at least `lowest` (ties to
    even), saturated at `largest`."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=lowest) - mantissa)
    return (torch.round(x / step) * step).clamp(-largest, largest)


def _exact_norm(s):
    h = s["x"].double()
    if s.get("skip") is not None:
        h = h + s["skip"].double()
    rstd = 1.0 / ((h * h).sum(dim=1) / h.shape[1] + EPS).sqrt()
    return h, rstd, torch.einsum("rc,c,r->rc", h, s["weight"].double(), rstd)


def _exact_operand(codes, scales, amax):
    pair = _pair_values(torch.float64)[codes.int()].flatten(1)
    sf = scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=1)
    return pair * sf * amax.double()[:, None] / FACTOR


def _exact_linear(s, a):
    z = torch.mm(a, _exact_operand(*s["w"]).t())
    if s["bias"]:
        z += s["bias_values"].double()
    if s["act"] == "gelu":
        d = z / (1.0 + torch.exp(-2.0 * GELU_C * (z + GELU_A * z ** 3)))
    elif s["act"] == "silu":
        d = z / (1.0 + torch.exp(-z))
    else:
        d = torch.relu(z) if s["act"] == "relu" else z
    if s["residual"]:
        d = d + s["add"].double()
    return {"d": d, "z": z} if s["z"] is not None else {"d": d}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        h, rstd, y = _exact_norm(s)
        r = {"rstd": rstd}
        if case["residual"]:
            r["h"] = h
        if case["out"] == "y":
            return dict(r, y=y)
        parts = y.split(y.shape[1] if case["out"] == "fp8_row" else SCALE_BLOCK, dim=1)
        scale = torch.stack([p.abs().amax(dim=1) / E4M3_MAX for p in parts], dim=1)
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        codes = [_round64(p / scale[:, i:i + 1], 3, -6, E4M3_MAX) for i, p in enumerate(parts)]
        return dict(r, scale=scale, codes=torch.cat(codes, dim=1))
    if kind == "norm_backward":
        dy, h, w = s["dy"].double(), s["h"].double(), s["weight"].double()
        inv = s["rstd"].double()[:, None]
        dot = ((dy * w) * h).sum(dim=1, keepdim=True)
        dx = inv * (dy * w) - h * dot * inv ** 3 / h.shape[1]
        if case["dh"]:
            dx = dx + s["grad_h"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc,r->c", dy, h, inv[:, 0])}
    if kind == "linear":
        return _exact_linear(s, _exact_operand(*s["a"]))
    if kind == "norm_linear":
        h, rstd, y = _exact_norm(s)
        amax = y.abs().amax(dim=1)
        g = torch.where(amax > 0, FACTOR / amax, torch.ones_like(amax))[:, None]
        top = y.abs().unflatten(1, (-1, 16)).amax(dim=2)
        sf = _round64(top / 6.0 * g, 3, -6, E4M3_MAX).repeat_interleave(16, dim=1)
        v = torch.where(sf > 0, _round64(y * g / sf, 1, 0, 6.0), torch.zeros_like(y))
        return dict(_exact_linear(s, v * sf * amax[:, None] / FACTOR), h=h, rstd=rstd, amax=amax)
    if kind == "act_backward":
        z, dz = s["z"].double(), s["dd"].double()
        if case["act"] == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        elif case["act"] in ("gelu", "silu"):
            gelu = case["act"] == "gelu"
            u = 2.0 * GELU_C * (z + GELU_A * z ** 3) if gelu else z
            du = 2.0 * GELU_C * (1.0 + 3.0 * GELU_A * z ** 2) if gelu else 1.0
            p = 1.0 / (1.0 + torch.exp(-u))
            dz = dz * (p + z * p * (1.0 - p) * du)
        # the maxima are those of dz as it is stored
        a = dz.to(s["z"].dtype).abs().double()
        return {"dz": dz, "dbias": dz.sum(dim=0),
                "amax": torch.cat([a.max(dim=1).values, a.max(dim=0).values])}
    norm = sum(float(t.double().pow(2).sum()) for t in s["grads"]) ** 0.5
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64, device=DEVICE),
            "grads": [t.double() * coef for t in s["grads"]]}
