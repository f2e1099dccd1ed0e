"""Cases that measure the operators of a gated feed-forward block in NVFP4.

The operators are those between the attention output and the next block of a pre-norm
transformer: dropout of the sublayer's output (a counter-based generator, no mask stored)
with the residual addition and the layer norm that follow it, the gated product act(A Wg^T +
bg) * (A Wu^T + bu) of NVFP4 operands, and the backward pass of each.

`run` computes an operator either in its plain form (elementary torch operations in FP32,
rounded once at the end) or, where `own` is true, through this package's entry points.
`exact` evaluates the definitions in FP64.
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
        # one decoded token through the gate and up projections of a wide block
        dict(name="gated_token", kind="gated", m=1, n=28672, k=8192, bias=False, act="silu",
             save=False, out="bf16"),
        # a training step's forward product: stacked weights of the benchmark's linear layer;
        # both pre-activations are kept, and the maxima that the quantization of d takes
        dict(name="gated_train", kind="gated", m=16384, n=14336, k=8192, bias=False, act="silu",
             save=True, out="bf16"),
        # a prompt of 300 tokens: norm into NVFP4, then the gated product; odd width, biases
        dict(name="norm_gated_prompt", kind="norm_gated", m=300, n=5000, k=7168, bias=True,
             act="gelu", save=False, out="bf16"),
        # the gradients of gate and up in that step, their sums and maxima
        dict(name="gated_backward_train", kind="gated_backward", rows=16384, cols=14336,
             dtype="bf16", act="silu"),
        # a shape that no tile divides, FP32 activations
        dict(name="gated_backward_ragged", kind="gated_backward", rows=4000, cols=5000,
             dtype="fp32", act="gelu"),
        # one decoded token's hidden state, quantized for the next product
        dict(name="layernorm_token", kind="layernorm", rows=1, cols=8192, dtype="bf16",
             residual=True, p=0.0, bias=True, out="fp8_row"),
        # a training step's activations: dropout, residual, norm, 8-bit output
        dict(name="layernorm_train", kind="layernorm", rows=16384, cols=8192, dtype="bf16",
             residual=True, p=0.1, bias=True, out="fp8_row"),
        # a row count and a row length that no tile divides, FP32, the norm as it is
        dict(name="layernorm_ragged", kind="layernorm", rows=4000, cols=5000, dtype="fp32",
             residual=True, p=0.0, bias=True, out="y"),
        # that training step's backward pass, with the gradient of the residual stream
        dict(name="layernorm_backward_train", kind="layernorm_backward", rows=16384, cols=8192,
             dtype="bf16", dh=True, p=0.1),
        # a first layer: no gradient arrives beside the norm's, nothing was dropped
        dict(name="layernorm_backward_ragged", kind="layernorm_backward", rows=4000, cols=5000,
             dtype="fp32", dh=False, p=0.0),
        # the sublayer's output added to the stream where no norm follows
        dict(name="dropout_train", kind="dropout", rows=16384, cols=8192, dtype="bf16",
             residual=True, p=0.1),
        # the gradient of a small odd matrix: the same mask, no residual
        dict(name="dropout_small", kind="dropout", rows=333, cols=1001, dtype="fp32",
             residual=False, p=0.25),
    ]


def _size(rng, lo, hi, multiple=1):
    """A size whose logarithm is uniform between lo and hi."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / multiple)) * multiple
    return max(-(-lo // multiple) * multiple, min(hi // multiple * multiple, n))


def draw(rng):
    kind = rng.choice(["gated", "gated", "norm_gated", "gated_backward", "layernorm",
                       "layernorm", "layernorm_backward", "dropout"])
    if kind in ("gated", "norm_gated"):
        n, k = _size(rng, 64, 14336, rng.choice([1, 8, 64])), _size(rng, 64, 8192, 32)
        m = _size(rng, 1, 64) if rng.random() < 0.4 else _size(rng, 64, 8192)
        return dict(kind=kind, m=m, n=n, k=k, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu", "silu", "silu"]),
                    save=rng.random() < 0.5,
                    out="bf16" if kind == "norm_gated" else rng.choice(["bf16", "bf16", "fp32"]))
    if kind == "gated_backward":
        cols = _size(rng, 64, 14336, rng.choice([1, 8, 128]))
        rows = _size(rng, 1, min(16384, 117_000_000 // cols))
        return dict(kind=kind, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    act=rng.choice(["none", "relu", "gelu", "silu"]))
    cols = _size(rng, 64, 16384, rng.choice([1, 8, 128]))
    rows = _size(rng, 1, min(16384, 134_000_000 // cols))
    c = dict(kind=kind, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp32"]),
             p=rng.choice([0.0, 0.05, 0.1, 0.5]))
    if kind == "layernorm":
        c.update(residual=rng.random() < 0.75, bias=rng.random() < 0.75,
                 out=rng.choice(["fp8_row", "fp8_block", "y"]))
    elif kind == "layernorm_backward":
        c.update(dh=rng.random() < 0.5)
    else:
        c.update(residual=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------- the counter-based mask

# Philox4x32 with ten rounds (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
# 2011).  Element i of a call takes 16 bits: of the block of counter (i / 8, offset) under the
# key `seed`, the half (i % 2) of word (i % 8) / 2, low half first.

def _philox_words(blocks, seed, offset):
    """The four 32-bit words (as int64) of the blocks 0 .. blocks - 1, [blocks][4]."""
    low = 0xFFFFFFFF
    i = torch.arange(blocks, dtype=torch.int64, device=DEVICE)
    c = [i & low, i >> 32, torch.full_like(i, offset & low), torch.full_like(i, offset >> 32)]
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # modulo 2^64: the high half is right
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack(c, dim=1)


def _threshold(p):
    """An element is dropped where its 16 bits are below this."""
    return int(math.floor(p * 65536.0 + 0.5))


def _keep(rows, cols, p, seed, offset):
    """The mask [rows][cols] and the factor of what is kept."""
    t = _threshold(p)
    w = _philox_words(-(-rows * cols // 8), seed, offset)
    bits = torch.stack([w & 0xFFFF, w >> 16], dim=2).reshape(-1)[:rows * cols]
    return (bits >= t).reshape(rows, cols), 65536.0 / (65536 - t)


def _dropped(x, s):
    """x in FP32 with the state's mask applied (none where p is 0)."""
    x = x.float()
    if s["p"] == 0.0:
        return x
    keep, factor = _keep(*x.shape, s["p"], s["seed"], s["offset"])
    return torch.where(keep, x * factor, torch.zeros_like(x))


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
    """A residual stream: rows of different magnitude and mean, a few channels much larger."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    x += 0.5 * torch.randn(rows, 1, generator=g, device=DEVICE)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEVICE))
    channel = torch.rand(cols, generator=g, device=DEVICE)
    return x.mul_(1.0 + 20.0 * (channel > 0.999)).to(dtype)


def _normal(shape, g, std, dtype):
    return (torch.randn(shape, generator=g, device=DEVICE) * std).to(dtype)


def _seeds(s, seed):
    """The generator's seed and the call's number, as a training program counts them."""
    r = random.Random(seed)
    s["seed"], s["offset"] = r.getrandbits(64), r.getrandbits(40)


def _prepare_norm(s, rows, cols, dt, g, bias, residual):
    s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device=DEVICE)).to(dt)
    s["shift"] = _normal((cols,), g, 0.1, dt) if bias else None
    s["x"] = _stream_values(rows, cols, g, dt)
    s["skip"] = _stream_values(rows, cols, g, dt) if residual else None
    s["h"] = torch.empty_like(s["x"]) if residual or s.get("p") else None
    s["mean"], s["rstd"] = (torch.empty(rows, device=DEVICE) for _ in range(2))


def prepare(case, seed):
    g, kind, s = _generator(seed), case["kind"], dict(case)
    _seeds(s, seed)
    if kind in ("gated", "norm_gated"):
        m, n, k, dt = case["m"], case["n"], case["k"], DTYPES[case["out"]]
        s["w"] = _operand(2 * n, k, g, 0.02)  # the gate's lines, then the up projection's
        if kind == "gated":
            s["a"] = _operand(m, k, g, 1.0)
        else:
            _prepare_norm(s, m, k, torch.bfloat16, g, True, True)
            s["p"] = 0.0
            s["a"] = (torch.empty(m, k // 2, dtype=torch.uint8, device=DEVICE),
                      torch.empty(m, k // 16, dtype=torch.uint8, device=DEVICE),
                      torch.empty(m, device=DEVICE))
        s["bias_values"] = _normal((2 * n,), g, 0.1, torch.float32) if case["bias"] else None
        s["d"] = torch.empty(m, n, dtype=dt, device=DEVICE)
        s["gu"] = torch.empty(m, 2 * n, dtype=dt, device=DEVICE) if case["save"] else None
        s["amax"] = torch.empty(m + n, device=DEVICE) if case["save"] else None
        s["workspace"] = torch.empty((256 << 20) + 4 * (m + 2 * n) * k // 8, dtype=torch.uint8,
                                     device=DEVICE)
    elif kind == "gated_backward":
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["gu"] = _normal((rows, 2 * cols), g, 1.5, dt)
        s["dd"] = _normal((rows, cols), g, 0.01, dt)
        s["dgu"] = torch.empty_like(s["gu"])
        s["dbias"] = torch.empty(2 * cols, device=DEVICE)
        s["amax"] = torch.empty(rows + 2 * cols, device=DEVICE)  # of the rows, of the columns
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEVICE)
    elif kind == "layernorm":
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        _prepare_norm(s, rows, cols, dt, g, case["bias"], case["residual"])
        if case["out"] == "y":
            s["y"] = torch.empty_like(s["x"])
        else:
            per_row = 1 if case["out"] == "fp8_row" else -(-cols // SCALE_BLOCK)
            s["codes"] = torch.empty(rows, cols, dtype=torch.uint8, device=DEVICE)
            s["scale"] = torch.empty(rows, per_row, device=DEVICE)
    elif kind == "layernorm_backward":
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device=DEVICE)).to(dt)
        s["h"] = _stream_values(rows, cols, g, dt)
        h = s["h"].float()
        s["mean"] = h.mean(dim=1)
        s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(dim=1) + EPS)
        s["dy"] = _normal((rows, cols), g, 0.01, dt)
        s["grad_h"] = _normal((rows, cols), g, 0.01, dt) if case["dh"] else None
        s["dx"] = torch.empty_like(s["h"])
        s["dskip"] = torch.empty_like(s["h"]) if case["p"] else None
        s["dweight"], s["dbias"] = (torch.empty(cols, device=DEVICE) for _ in range(2))
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEVICE)
    else:
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        s["x"] = _stream_values(rows, cols, g, dt)
        s["skip"] = _stream_values(rows, cols, g, dt) if case["residual"] else None
        s["y"] = torch.empty_like(s["x"])
    return s


# ---------------------------------------------------------------- plain forms

def _norm_plain(s):
    h = _dropped(s["x"], s)
    if s["skip"] is not None:
        h = h + s["skip"].float()
    mean = h.mean(dim=1)
    centred = h - mean[:, None]
    rstd = torch.rsqrt(centred.square().mean(dim=1) + EPS)
    y = centred * rstd[:, None] * s["weight"].float()
    if s["shift"] is not None:
        y = y + s["shift"].float()
    r = {"mean": mean, "rstd": rstd}
    if s["h"] is not None:
        r["h"] = h.to(s["x"].dtype)
    return r, y


def _plain_layernorm(s):
    r, y = _norm_plain(s)
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


def _plain_layernorm_backward(s):
    dy, dt = s["dy"].float(), s["h"].dtype
    n = (s["h"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    d = (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True)) \
        * s["rstd"][:, None]
    if s["dh"]:
        d = d + s["grad_h"].float()
    r = {"dx": _dropped(d, s).to(dt), "dweight": (dy * n).sum(dim=0), "dbias": dy.sum(dim=0)}
    if s["p"]:
        r["dskip"] = d.to(dt)
    return r


def _plain_dropout(s):
    y = _dropped(s["x"], s)
    if s["skip"] is not None:
        y = y + s["skip"].float()
    return {"y": y.to(s["x"].dtype)}


def _act_plain(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + GELU_A * z * z * z)))
    return z * torch.sigmoid(z) if act == "silu" else z


def _plain_gated(s, a, w):
    gu = torch.matmul(a, w.t())
    if s["bias"]:
        gu = gu + s["bias_values"]
    d = (_act_plain(gu[:, :s["n"]], s["act"]) * gu[:, s["n"]:]).to(s["d"].dtype)
    r = {"d": d}
    if s["save"]:
        m = d.abs()
        r.update(gu=gu.to(d.dtype), amax=torch.cat([m.amax(dim=1), m.amax(dim=0)]))
    return r


def _plain_norm_gated(s):
    r, y = _norm_plain(s)
    codes, scale, amax = _quantize_rows(y)
    v = _code_values(torch.float32)[codes].reshape(*scale.shape, 16)
    a = v * (scale * (amax * (1.0 / FACTOR))[:, None])[:, :, None]
    return dict(r, row_amax=amax, **_plain_gated(s, a.reshape(y.shape), _dequantize(*s["w"])))


def _plain_gated_backward(s):
    n, act, dd = s["cols"], s["act"], s["dd"].float()
    g, u = s["gu"][:, :n].float(), s["gu"][:, n:].float()
    if act == "relu":
        slope = (g > 0).float()
    elif act == "gelu":
        t = torch.tanh(GELU_C * (g + GELU_A * g * g * g))
        slope = 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * g * g)
    elif act == "silu":
        sig = torch.sigmoid(g)
        slope = sig * (1 + g * (1 - sig))
    else:
        slope = torch.ones_like(g)
    both = torch.cat([dd * u * slope, dd * _act_plain(g, act)], dim=1)
    dgu = both.to(s["gu"].dtype)
    a = dgu.abs()
    return {"dgu": dgu, "dbias": both.sum(dim=0),
            "amax": torch.cat([a.amax(dim=1), a.amax(dim=0)])}


# ---------------------------------------------------------------- the framework's operators

def _mask(nv, s):
    return nv.Mask(s["p"], s["seed"], s["offset"]) if s["p"] else None


def _own_layernorm(s):
    import nvfp4_precision_quantization_gb300 as nv
    r = {"mean": s["mean"], "rstd": s["rstd"]}
    fp8 = None
    if s["out"] != "y":
        fp8 = nv.Fp8Out(s["codes"], s["scale"], 0 if s["out"] == "fp8_row" else SCALE_BLOCK)
        r.update(codes=s["codes"].view(torch.float8_e4m3fn), scale=s["scale"])
    nv.nvfp4_add_layernorm(s["x"], s["weight"], EPS, bias=s["shift"], residual=s["skip"],
                           mask=_mask(nv, s), h=s["h"], y=s.get("y"), mean=s["mean"],
                           rstd=s["rstd"], fp8=fp8)
    if s["h"] is not None:
        r["h"] = s["h"]
    if s["out"] == "y":
        r["y"] = s["y"]
    return r


def _own_layernorm_backward(s):
    import nvfp4_precision_quantization_gb300 as nv
    nv.nvfp4_add_layernorm_backward(s["dy"], s["h"], s["weight"], s["mean"], s["rstd"], s["dx"],
                                    dweight=s["dweight"], dbias=s["dbias"], dh=s["grad_h"],
                                    mask=_mask(nv, s), dresidual=s["dskip"],
                                    workspace=s["workspace"])
    r = {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if s["p"]:
        r["dskip"] = s["dskip"]
    return r


def _own_dropout(s):
    import nvfp4_precision_quantization_gb300 as nv
    nv.nvfp4_dropout(s["x"], nv.Mask(s["p"], s["seed"], s["offset"]), s["y"],
                     residual=s["skip"])
    return {"y": s["y"]}


def _own_gated(s):
    import nvfp4_precision_quantization_gb300 as nv
    r, m = {}, s["m"]
    if s["kind"] == "norm_gated":
        nv.nvfp4_add_layernorm(s["x"], s["weight"], EPS, bias=s["shift"], residual=s["skip"],
                               h=s["h"], mean=s["mean"], rstd=s["rstd"], row=nv.Out(*s["a"]),
                               cfg=nv.Config(nv.NVFP4_ROW_SCALED, BOUND, 0, 0))
        r = {"h": s["h"], "mean": s["mean"], "rstd": s["rstd"], "row_amax": s["a"][2]}
    act = {"none": nv.NVFP4_ACT_NONE, "relu": nv.NVFP4_ACT_RELU, "gelu": nv.NVFP4_ACT_GELU,
           "silu": nv.NVFP4_ACT_SILU}[s["act"]]
    amax = s["amax"]
    nv.nvfp4_gemm_gated(nv.Operand(*s["a"], nv.NVFP4_ROW_SCALED, BOUND),
                        nv.Operand(*s["w"], nv.NVFP4_ROW_SCALED, BOUND), s["d"],
                        bias=s["bias_values"], act=act, gu=s["gu"],
                        row_amax=amax[:m] if amax is not None else None,
                        col_amax=amax[m:] if amax is not None else None,
                        workspace=s["workspace"])
    r["d"] = s["d"]
    if s["save"]:
        # the maxima of values of d's type are values of that type
        r.update(gu=s["gu"], amax=amax.to(s["d"].dtype))
    return r


def _own_gated_backward(s):
    import nvfp4_precision_quantization_gb300 as nv
    act = {"none": nv.NVFP4_ACT_NONE, "relu": nv.NVFP4_ACT_RELU, "gelu": nv.NVFP4_ACT_GELU,
           "silu": nv.NVFP4_ACT_SILU}[s["act"]]
    rows = s["rows"]
    nv.nvfp4_gated_backward(s["dd"], s["gu"], act, s["dgu"], dbias=s["dbias"],
                            row_amax=s["amax"][:rows], col_amax=s["amax"][rows:],
                            workspace=s["workspace"])
    return {"dgu": s["dgu"], "dbias": s["dbias"], "amax": s["amax"].to(s["dgu"].dtype)}


def run(state):
    kind = state["kind"]
    if own:
        return {"layernorm": _own_layernorm, "layernorm_backward": _own_layernorm_backward,
                "dropout": _own_dropout, "gated": _own_gated, "norm_gated": _own_gated,
                "gated_backward": _own_gated_backward}[kind](state)
    if kind == "gated":
        return _plain_gated(state, _dequantize(*state["a"]), _dequantize(*state["w"]))
    return {"layernorm": _plain_layernorm, "layernorm_backward": _plain_layernorm_backward,
            "dropout": _plain_dropout, "norm_gated": _plain_norm_gated,
            "gated_backward": _plain_gated_backward}[kind](state)


# ---------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    if kind in ("gated", "norm_gated"):
        m, n, k = case["m"], case["n"], case["k"]
        line = k // 2 + k // 16 + 4
        bytes_ = 2 * n * line + BYTES[case["out"]] * m * n * (3 if case["save"] else 1)
        bytes_ += (8 * n if case["bias"] else 0) + (4 * (m + n) if case["save"] else 0)
        bytes_ += m * line if kind == "gated" else 6 * m * k + 4 * k + 12 * m
        return {"bytes": bytes_, "flops": 4 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    n, b = rows * cols, BYTES[case["dtype"]]
    if kind == "gated_backward":
        return {"bytes": 5 * n * b + 4 * rows + 16 * cols, "flops": 16 * n}
    if kind == "layernorm":
        moved = 1 + bool(case["residual"]) + bool(case["residual"] or case["p"])
        bytes_ = n * b * moved + cols * b * (1 + bool(case["bias"])) + 8 * rows
        if case["out"] == "y":
            bytes_ += n * b
        else:
            blocks = 1 if case["out"] == "fp8_row" else -(-cols // SCALE_BLOCK)
            bytes_ += n + 4 * rows * blocks
        return {"bytes": bytes_, "flops": 8 * n}
    if kind == "layernorm_backward":
        moved = 3 + bool(case["dh"]) + bool(case["p"])
        return {"bytes": n * b * moved + cols * (b + 8) + 8 * rows, "flops": 14 * n}
    return {"bytes": n * b * (3 if case["residual"] else 2), "flops": 2 * n}


# ---------------------------------------------------------------- 64 bits

def _round64(x, mantissa, lowest, largest):
    """x rounded to `mantissa` fraction bits with the exponent at least `lowest` (ties to
    even), saturated at `largest`."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=lowest) - mantissa)
    return (torch.round(x / step) * step).clamp(-largest, largest)


def _times32(a, m):
    """(high, low) 32 bits of a * m for a 32-bit tensor and constant, in 16-bit limbs."""
    lo, hi = a & 0xFFFF, a >> 16
    m0, m1 = m & 0xFFFF, m >> 16
    mid = (lo * m0 >> 16) + (lo * m1 & 0xFFFF) + hi * m0
    return hi * m1 + (lo * m1 >> 16) + (mid >> 16), (mid << 16 & 0xFFFF0000) | (lo * m0 & 0xFFFF)


def _exact_dropped(x, s):
    """The definition element by element, in runs so that it fits beside the data."""
    out = x.double().flatten()
    out = out.clone() if x.dtype == torch.float64 else out  # written below, the input is not
    t = _threshold(s["p"])
    if t == 0:
        return out.view(x.shape)
    for at in range(0, out.numel(), 1 << 25):
        i = torch.arange(at, min(at + (1 << 25), out.numel()), device=DEVICE)
        block = torch.arange(at // 8, int(i[-1]) // 8 + 1, device=DEVICE)
        v = [block % (1 << 32), block // (1 << 32), torch.zeros_like(block) + s["offset"] % 2 ** 32,
             torch.zeros_like(block) + s["offset"] // 2 ** 32]
        for r in range(10):
            key = [(k + r * w) % 2 ** 32 for k, w in ((s["seed"] % 2 ** 32, 0x9E3779B9),
                                                      (s["seed"] // 2 ** 32, 0xBB67AE85))]
            (h0, l0), (h2, l2) = _times32(v[0], 0xD2511F53), _times32(v[2], 0xCD9E8D57)
            v = [h2 ^ v[1] ^ key[0], l2, h0 ^ v[3] ^ key[1], l0]
        word = torch.stack(v)[i % 8 // 2, i // 8 - at // 8]
        bits = torch.where(i % 2 == 1, word // 65536, word % 65536)
        run_ = out[at:at + (1 << 25)]
        run_.copy_(torch.where(bits < t, torch.zeros_like(run_), run_ / (1.0 - t / 65536.0)))
    return out.view(x.shape)


def _exact_norm(s):
    h = _exact_dropped(s["x"], s)
    if s["skip"] is not None:
        h = h + s["skip"].double()
    mean = h.sum(dim=1) / h.shape[1]
    c = h - mean[:, None]
    rstd = 1.0 / ((c * c).sum(dim=1) / h.shape[1] + EPS).sqrt()
    y = torch.einsum("rc,c,r->rc", c, s["weight"].double(), rstd)
    if s["shift"] is not None:
        y = y + s["shift"].double()
    r = {"mean": mean, "rstd": rstd}
    if s["h"] is not None:
        r["h"] = h
    return r, y


def _exact_operand(codes, scales, amax):
    pair = _pair_values(torch.float64)[codes.int()].flatten(1)
    sf = scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=1)
    return pair * sf * amax.double()[:, None] / FACTOR


def _exact_act(z, act):
    """act(z) and its derivative, by the logistic function p of u."""
    if act == "relu":
        return torch.relu(z), torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
    if act == "none":
        return z, torch.ones_like(z)
    gelu = act == "gelu"
    u = 2.0 * GELU_C * (z + GELU_A * z ** 3) if gelu else z
    du = 2.0 * GELU_C * (1.0 + 3.0 * GELU_A * z ** 2) if gelu else 1.0
    p = 1.0 / (1.0 + torch.exp(-u))
    return z * p, p + z * p * (1.0 - p) * du


def _exact_gated(s, a):
    n = s["n"]
    w = _exact_operand(*s["w"])
    g, u = torch.mm(a, w[:n].t()), torch.mm(a, w[n:].t())
    if s["bias"]:
        g += s["bias_values"][:n].double()
        u += s["bias_values"][n:].double()
    d = _exact_act(g, s["act"])[0] * u
    if not s["save"]:
        return {"d": d}
    m = d.to(s["d"].dtype).abs().double()  # the maxima are those of d as it is stored
    return {"d": d, "gu": torch.cat([g, u], dim=1),
            "amax": torch.cat([m.max(dim=1).values, m.max(dim=0).values])}


def exact(case, seed):
    kind = case["kind"]
    if kind in ("gated", "norm_gated") and 4 * case["m"] * case["n"] * case["k"] > 1.2e13:
        return None
    s = prepare(case, seed)
    if kind == "layernorm":
        r, y = _exact_norm(s)
        if case["out"] == "y":
            return dict(r, y=y)
        parts = y.split(y.shape[1] if case["out"] == "fp8_row" else SCALE_BLOCK, dim=1)
        scale = torch.stack([p.abs().amax(dim=1) / E4M3_MAX for p in parts], dim=1)
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        codes = [_round64(p / scale[:, i:i + 1], 3, -6, E4M3_MAX) for i, p in enumerate(parts)]
        return dict(r, scale=scale, codes=torch.cat(codes, dim=1))
    if kind == "layernorm_backward":
        dy, w, inv = s["dy"].double(), s["weight"].double(), s["rstd"].double()[:, None]
        c, cols = s["h"].double() - s["mean"].double()[:, None], s["h"].shape[1]
        total = (dy * w).sum(dim=1, keepdim=True)
        dot = (dy * w * c).sum(dim=1, keepdim=True)
        d = inv * (dy * w) - inv * total / cols - c * dot * inv ** 3 / cols
        if case["dh"]:
            d = d + s["grad_h"].double()
        r = {"dx": _exact_dropped(d, s), "dweight": torch.einsum("rc,rc,r->c", dy, c, inv[:, 0]),
             "dbias": dy.sum(dim=0)}
        if case["p"]:
            r["dskip"] = d
        return r
    if kind == "dropout":
        y = _exact_dropped(s["x"], s)
        return {"y": y + s["skip"].double() if case["residual"] else y}
    if kind == "gated":
        return _exact_gated(s, _exact_operand(*s["a"]))
    if kind == "norm_gated":
        r, y = _exact_norm(s)
        amax = y.abs().amax(dim=1)
        g = torch.where(amax > 0, FACTOR / amax, torch.ones_like(amax))[:, None]
        top = y.abs().unflatten(1, (-1, 16)).amax(dim=2)
        sf = _round64(top / 6.0 * g, 3, -6, E4M3_MAX).repeat_interleave(16, dim=1)
        v = torch.where(sf > 0, _round64(y * g / sf, 1, 0, 6.0), torch.zeros_like(y))
        return dict(r, row_amax=amax, **_exact_gated(s, v * sf * amax[:, None] / FACTOR))
    n, dd = case["cols"], s["dd"].double()
    g, u = s["gu"][:, :n].double(), s["gu"][:, n:].double()
    value, slope = _exact_act(g, case["act"])
    both = torch.cat([dd * slope * u, dd * value], dim=1)
    a = both.to(s["gu"].dtype).abs().double()  # the maxima of dgu as it is stored
    return {"dgu": both, "dbias": both.sum(dim=0),
            "amax": torch.cat([a.max(dim=1).values, a.max(dim=0).values])}
