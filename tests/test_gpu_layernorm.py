"""Dropout + add + layer norm with its quantized outputs, and its backward pass, on the GPU
against the FP64 definitions.

Tolerances, derived from the FP32 arithmetic.  h: one product and one addition, 2^-23 of A =
|x factor| + |r|.  mean: at most 48 additions per chain (32 values in a thread, a warp tree of 5,
up to 32 warps counted with their growth), so within 2^-18 mean(A).  The squares are summed
around the warps' means, so their sum is within 2^-18 of itself, plus 2^-22 Q for h's error, with
Q = rms(A) / sqrt(var + eps), plus (2^-18 Q)^2 for the means' own; rstd takes half of that and
2^-23.  y: |w| rstd times the errors of h and the mean, |n w| times rstd's, and 2^-22 of |n w| and
|y| for the three products and sums.  Storing rounds once: 2^-8 (BF16) or 2^-24 (FP32) relative.
E4M3 keeps 3 fraction bits: half a step is 2^-4 relative, or 2^-10 of the scale below the normal
range.  The NVFP4 codes are compared byte for byte with the oracle's quantization of the FP32 y
that the same call returns.
"""
import numpy as np
import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv
import oracle
from block_reference import drop, layernorm, layernorm_backward, threshold
from layer_reference import at_offset, guarded, half_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float32]
EPS = 1e-5
# one row to enough of them for every CTA to walk several, at each width of a row's team; row
# lengths on, before and behind the teams' borders, odd ones among them
SHAPES = [(1, 1), (1, 16), (3, 17), (5, 100), (9, 128), (2, 511), (33, 512), (7, 1000), (4, 1024),
          (700, 1024), (65, 2056), (6, 4096), (2, 5000), (1, 8192), (400, 8192), (3, 8193),
          (310, 16384), (2, 28672), (1, 32768), (0, 64),
          (9001, 24), (7003, 512), (5003, 1000), (3001, 2048), (2777, 4096), (1501, 5008),
          (701, 12000), (400, 20000), (9001, 25), (3001, 1001), (1501, 4097), (601, 9001),
          (401, 17001)]


def _inputs(rows, cols, dtype, seed, wdtype=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x = (x + 3 * torch.randn(rows, 1, generator=g, device=DEV)) \
        * torch.exp(2 * torch.randn(rows, 1, generator=g, device=DEV))
    r = torch.randn(rows, cols, generator=g, device=DEV)
    w = 1 + 0.3 * torch.randn(cols, generator=g, device=DEV)
    b = 0.5 * torch.randn(cols, generator=g, device=DEV)
    return x.to(dtype), r.to(dtype), w.to(wdtype or dtype), b.to(wdtype or dtype)


def _bounds(x, r, w, h, rstd, y, mask):
    """Errors before the last rounding, as derived above: of h, mean, rstd and y."""
    a = (drop(x, *mask) if mask else x.double()).abs()
    if r is not None:
        a = a + r.double().abs()
    e_h, e_m = 2.0 ** -23 * a, 2.0 ** -18 * a.mean(dim=1)
    q = a.square().mean(dim=1).sqrt() * rstd
    rel = 2.0 ** -18 + 2.0 ** -22 * q + (2.0 ** -18 * q) ** 2
    w = w.double().abs()
    c = (h - h.mean(dim=1, keepdim=True)).abs() * rstd[:, None]
    e_y = w * rstd[:, None] * (e_h + e_m[:, None]) + c * w * (rel[:, None] + 2.0 ** -22) \
        + 2.0 ** -22 * y.abs()
    return e_h, e_m, rel, e_y


def _inside(got, want, tol, what):
    bad = (got.double() - want).abs() > tol + 1e-37
    assert not bool(bad.any()), (what, got[bad][:3].tolist(), want[bad][:3].tolist())


def _mask(p, seed):
    return (p, 12345 + seed, 977 * seed) if p else None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_and_sum(rows, cols, dtype):
    x, r, w, b = _inputs(rows, cols, dtype, rows * 31 + cols)
    half = half_ulp(dtype)
    for residual, bias, p in ((None, None, 0.0), (r, b, 0.1), (None, b, 0.6), (r, None, 0.0)):
        mask = _mask(p, cols)
        y, ok_y = guarded((rows, cols), dtype)
        h, ok_h = guarded((rows, cols), dtype)
        mean, ok_m = guarded((rows,), torch.float32)
        rstd, ok_s = guarded((rows,), torch.float32)
        keep = residual is not None or mask is not None
        nv.nvfp4_add_layernorm(x, w, EPS, bias=bias, residual=residual,
                               mask=nv.Mask(*mask) if mask else None, h=h if keep else None, y=y,
                               mean=mean, rstd=rstd)
        torch.cuda.synchronize()
        eh, em, es, ey = layernorm(x, residual, w, bias, EPS, mask)
        t_h, t_m, rel, t_y = _bounds(x, residual, w, eh, es, ey, mask)
        _inside(mean, em, t_m + 2.0 ** -23 * em.abs(), "mean")
        _inside(rstd, es, rel * es, "rstd")
        _inside(y, ey, t_y * (1 + half) + half * ey.abs(), "y")
        if keep:
            _inside(h, eh, t_h * (1 + half) + half * eh.abs(), "h")
        for ok in (ok_y, ok_h, ok_m, ok_s):
            ok()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_fp8_output(rows, cols, dtype, block):
    x, r, w, b = _inputs(rows, cols, dtype, rows + cols, torch.float32)
    mask = _mask(0.1, rows)
    blocks = -(-cols // 128) if block else 1
    codes, ok_c = guarded((rows, cols), torch.uint8)
    scale, ok_s = guarded((rows, blocks), torch.float32)
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, mask=nv.Mask(*mask),
                           fp8=nv.Fp8Out(codes, scale, block))
    torch.cuda.synchronize()
    eh, _, es, y = layernorm(x, r, w, b, EPS, mask)
    t_y = _bounds(x, r, w, eh, es, y, mask)[3]
    width = 128 if block else max(cols, 1)

    def in_blocks(t):
        return torch.nn.functional.pad(t, (0, blocks * width - cols)).reshape(rows, blocks, width)
    want = in_blocks(y).abs().amax(dim=2) / 448.0
    _inside(scale, want, in_blocks(t_y).amax(dim=2) / 448.0 + 2.0 ** -23 * want, "scale")
    s = scale.double().repeat_interleave(width, dim=1)[:, :cols]
    v = codes.view(torch.float8_e4m3fn).double() * s
    # (the scale rounds up or down: a value at the maximum stays within the last step)
    assert bool(((v - y).abs() <= 1.001 * (2.0 ** -4 * y.abs() + 2.0 ** -10 * s) + 2 * t_y).all())
    ok_c()
    ok_s()


@pytest.mark.parametrize("fos", [0, 1])
@pytest.mark.parametrize("bound", [448.0, 256.0])
@pytest.mark.parametrize("rows,cols", [s for s in SHAPES if 0 < s[0] < 800 or s[1] in (25, 1001)])
def test_nvfp4_output_is_the_quantize_of_y(rows, cols, bound, fos):
    x, r, w, b = _inputs(rows, cols, torch.float32, 7 * rows + cols)
    if rows > 2:  # a row of equal values: y is the bias
        x[2] = 1.5
        r[2] = 0
    y = torch.empty_like(x)
    codes, ok_c = guarded((rows, (cols + 1) // 2), torch.uint8)
    scales, ok_s = guarded((rows, (cols + 15) // 16), torch.uint8)
    amax, ok_a = guarded((rows,), torch.float32)
    cfg = nv.Config(nv.NVFP4_ROW_SCALED, bound, fos, 0)
    mask = nv.Mask(0.25, 9, cols) if cols % 2 else None
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, mask=mask, y=y,
                           row=nv.Out(codes, scales, amax), cfg=cfg)
    torch.cuda.synchronize()
    ref = oracle.quantize(y.cpu().numpy(), "fp32", mode=oracle.ROW_SCALED, bound=bound,
                          four_over_six=bool(fos), columnwise=False)["row"]
    assert np.array_equal(amax.cpu().numpy().view(np.uint32), ref[2].view(np.uint32))
    assert np.array_equal(scales.cpu().numpy(), ref[1])
    assert np.array_equal(codes.cpu().numpy(), ref[0])
    for ok in (ok_c, ok_s, ok_a):
        ok()


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 8192), (40, 512), (7003, 512), (3001, 1001), (4004, 1024),
                                       (2777, 2048), (2000, 4096), (1501, 5001), (1000, 8192),
                                       (1500, 8200), (701, 12000), (320, 20000), (330, 17001)])
def test_bf16_rows_to_nvfp4(rows, cols, masked):
    """BF16 rows, few ones and enough of them for the ring: the codes, scales and amax are the oracle's of
    the FP32 y.  That y is the one that the FP32 kernels give for the same values: a BF16 x is exact
    in FP32, and at these lengths neither the rows' teams nor the order of their sums depend on the type."""
    x, r, w, b = _inputs(rows, cols, torch.bfloat16, 3 * rows + cols)
    mask = nv.Mask(0.25, 9, cols) if masked else None
    out = nv.alloc_out(rows, cols, rows)
    cfg = nv.Config(nv.NVFP4_ROW_SCALED, 448.0, 0, 0)
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, mask=mask, row=out, cfg=cfg)
    y = torch.empty(rows, cols, device=DEV)
    nv.nvfp4_add_layernorm(x.float(), w, EPS, bias=b, residual=r.float(), mask=mask, y=y)
    torch.cuda.synchronize()
    ref = oracle.quantize(y.cpu().numpy(), "fp32", mode=oracle.ROW_SCALED, bound=448.0,
                          columnwise=False)["row"]
    assert np.array_equal(out.amax.cpu().numpy().view(np.uint32), ref[2].view(np.uint32))
    assert np.array_equal(out.scales.cpu().numpy(), ref[1])
    assert np.array_equal(out.codes.cpu().numpy(), ref[0])


def test_given_amax():
    x, _, w, b = _inputs(9, 320, torch.float32, 5)
    y = torch.empty_like(x)
    for mode, n in ((nv.NVFP4_ROW_SCALED, 9), (nv.NVFP4_PER_TENSOR, 1)):
        given = torch.full((n,), 3.25, device=DEV) + torch.arange(n, device=DEV)
        o = nv.alloc_out(9, 320, n)
        o.amax_in = given
        nv.nvfp4_add_layernorm(x, w, EPS, bias=b, y=y, row=o, cfg=nv.Config(mode, 448.0, 0, 0))
        torch.cuda.synchronize()
        ref = oracle.quantize(y.cpu().numpy(), "fp32", mode=mode, bound=448.0, columnwise=False,
                              row_amax_in=given.cpu().numpy())["row"]
        assert torch.equal(o.amax, given)
        assert np.array_equal(o.codes.cpu().numpy(), ref[0])
        assert np.array_equal(o.scales.cpu().numpy(), ref[1])


def test_rows_far_from_zero_keep_their_variance():
    """Values of 2^12 +- 1 (exact in FP32): sums of squares around zero would lose them all."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for cols in (64, 1000, 8192, 20000):
        x = 4096.0 + torch.randint(-1, 2, (6, cols), generator=g, device=DEV).float()
        w = torch.ones(cols, device=DEV)
        rstd, mean = torch.empty(6, device=DEV), torch.empty(6, device=DEV)
        nv.nvfp4_add_layernorm(x, w, 0.0, y=torch.empty_like(x), mean=mean, rstd=rstd)
        _, em, es, _ = layernorm(x, None, w, None, 0.0)
        # each mean is within 2^-18 4096 = 2^-6 of its own: 2^-12 of a variance of 2/3
        _inside(mean, em, 2.0 ** -6, "mean")
        _inside(rstd, es, (2.0 ** -11 + 2.0 ** -18) * es, "rstd")


@pytest.mark.parametrize("far", [2.0 ** 12, 2.0 ** 14, 2.0 ** 16, -2.0 ** 16])
@pytest.mark.parametrize("cols", [64, 511, 1000, 1024, 2056, 5000, 8192, 12000, 20000, 32768])
@pytest.mark.parametrize("rows", [6, 4100])
def test_variance_does_not_depend_on_the_mean(rows, cols, far):
    """Values far + {-1, 0, 1}: every difference to a mean near them is exact in FP32.

    A chain adds at most 16 pairs in a thread, its two halves, 5 steps in a warp, 2 and 5 in the join: g =
    29 2^-24.  A warp's mean is within shift = g |far| of its own, so its squares are within g (sigma + off
    + shift)^2 and its differences within g (mean|c| + off + shift), off being the distance of a warp's
    mean from the row's: no more than that of some 512 columns in a row.  The join moves them by at
    most 2 off + shift, to the first warp's mean, in products within 2^-21.  rstd takes half of the
    variance's error and 2^-23; the mean is rounded once and carries the differences' error."""
    if rows * cols > 5_000_000 and cols not in (2056, 20000):
        rows = 700
    g = torch.Generator(device=DEV)
    g.manual_seed(cols)
    x = far + torch.randint(-1, 2, (rows, cols), generator=g, device=DEV).float()
    w = torch.ones(cols, device=DEV)
    mean, rstd, y = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty_like(x)
    nv.nvfp4_add_layernorm(x, w, 0.0, y=y, mean=mean, rstd=rstd)
    _, em, es, _ = layernorm(x, None, w, None, 0.0)
    c = x.double() - em[:, None]
    var, spread = c.square().mean(dim=1), c.abs().mean(dim=1)
    block = torch.nn.functional.pad(c, (0, -cols % 512)).unflatten(1, (-1, 512)).sum(dim=2)
    count = torch.full((block.shape[1],), 512.0, dtype=torch.float64, device=DEV)
    count[-1] -= -cols % 512
    chain = 29 * 2.0 ** -24
    off = (block / count).abs().amax(dim=1)
    shift = chain * abs(far)
    moved = 2 * off + shift
    rel = ((chain + 2.0 ** -21) * (var.sqrt() + moved) ** 2
           + 2 * moved * chain * (spread + off + shift)) / var
    _inside(rstd, es, (rel / 2 + 2.0 ** -23) * es, "rstd")
    _inside(mean, em, 2.0 ** -24 * em.abs() + chain * (spread + off + shift) + 2.0 ** -21 * moved, "mean")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 9, 2500])
@pytest.mark.parametrize("cols", [64, 128, 1000, 1024, 2048, 5000, 7424, 8192, 12000, 20000])
def test_small_means_are_those_of_the_sum(rows, cols, dtype):
    """Integers of -3 .. 3: every sum is exact in FP32, so a mean, however near 0, is off by the roundings of 1 /
    cols and of one product alone: 2^-23 of itself."""
    g = torch.Generator(device=DEV)
    g.manual_seed(rows * cols)
    x = torch.randint(-3, 4, (rows, cols), generator=g, device=DEV).to(dtype)
    x[0, 1::2] = -x[0, 0::2]  # a row that sums to 0
    w = torch.ones(cols, device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    nv.nvfp4_add_layernorm(x, w, EPS, y=torch.empty_like(x), mean=mean, rstd=rstd)
    _, em, es, _ = layernorm(x, None, w, None, EPS)
    assert float(mean[0]) == 0.0
    _inside(mean, em, 2.0 ** -23 * em.abs(), "mean")
    _inside(rstd, es, 2.0 ** -18 * es, "rstd")


@pytest.mark.parametrize("cols", [2048, 1003])
def test_fused_is_the_two_operators(cols):
    """The fused sum is bit for bit that of nvfp4_dropout with the same mask, and in place."""
    for dtype in DTYPES:
        x, r, w, b = _inputs(700, cols, dtype, 4)
        mask = nv.Mask(0.3, 1 << 63, 5)
        h, y, both = (torch.empty_like(x) for _ in range(3))
        nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, mask=mask, h=h, y=y)
        nv.nvfp4_dropout(x, mask, both, residual=r)
        assert torch.equal(both, h)
        r2, x2 = r.clone(), x.clone()
        nv.nvfp4_add_layernorm(x2, w, EPS, bias=b, residual=r2, mask=mask, h=r2, y=x2)
        assert torch.equal(r2, h) and torch.equal(x2, y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_unaligned_starts(dtype, offset):
    x, r, w, b = _inputs(6, 1040, dtype, offset)
    mask = nv.Mask(0.2, 3, 4)
    want = torch.empty_like(x)
    codes, scale = torch.empty(6, 1040, dtype=torch.uint8, device=DEV), torch.empty(6, device=DEV)
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, mask=mask, y=want)
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, mask=mask, fp8=nv.Fp8Out(codes, scale, 0))
    y, ok = guarded((6, 1040), dtype, offset=offset)
    h, ok_h = guarded((6, 1040), dtype, offset=offset)
    c, ok_c = guarded((6, 1040), torch.uint8, offset=offset)
    s2 = torch.empty(6, device=DEV)
    xo, ro, wo, bo = (at_offset(t, offset) for t in (x, r, w, b))
    nv.nvfp4_add_layernorm(xo, wo, EPS, bias=bo, residual=ro, mask=mask, h=h, y=y)
    nv.nvfp4_add_layernorm(xo, wo, EPS, bias=bo, residual=ro, mask=mask, fp8=nv.Fp8Out(c, s2, 0))
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(c, codes) and torch.equal(s2, scale)
    for o in (ok, ok_h, ok_c):
        o()


def test_bad_values_stay_in_their_row():
    """A NaN or an infinity spoils its row alone, and not even that where it is dropped."""
    x, r, w, b = _inputs(5, 640, torch.float32, 9)
    y, y2, y3 = (torch.empty_like(x) for _ in range(3))
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, y=y)
    x[1, 3], x[3, 600] = float("nan"), float("inf")
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, y=y2)
    assert bool(y2[1].isnan().all()) and bool(y2[3].isnan().any())
    for i in (0, 2, 4):
        assert torch.equal(y[i], y2[i])
    h = torch.empty_like(x)
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, mask=nv.Mask(1.0, 1, 1), h=h, y=y3)
    assert torch.equal(h, r) and not bool(y3.isnan().any())


@pytest.mark.parametrize("cols", [48, 640, 8192])
def test_infinite_rows(cols):
    """The mean of a row with an infinity is that infinity (with both a NaN), its rstd and y are NaN."""
    x, _, w, b = _inputs(4, cols, torch.float32, 10)
    inf = float("inf")
    x[0, 0], x[1, cols - 1], x[2, 1], x[2, cols - 2] = inf, -inf, inf, -inf
    y, mean, rstd = torch.empty_like(x), torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, y=y, mean=mean, rstd=rstd)
    assert float(mean[0]) == inf and float(mean[1]) == -inf and bool(mean[2].isnan())
    assert bool(rstd[:3].isnan().all()) and bool(y[:3].isnan().all())
    assert bool(y[3].isfinite().all()) and bool(rstd[3].isfinite())


@pytest.mark.parametrize("far", [0.0, 1e27])
@pytest.mark.parametrize("cols", [48, 640, 1000, 5000, 8192, 20000])
def test_rows_whose_squares_overflow(cols, far):
    """Spreads above 2e19: the variance is infinite in FP32, so rstd is 0 and y the bias; the mean is not
    touched by that.  One block of columns far from the others overflows in the join alone.  (A row
    may come out as one value: its variance is 0, and its y the bias too.)"""
    x, _, w, b = _inputs(5, cols, torch.float32, 12)
    spread = torch.tensor([1e20, 1e22, 1e25, 1e30, 0.0], device=DEV)[:, None]
    x = far + torch.sign(x) * (1 + x.abs().clamp(max=1)) * spread
    x[4, cols // 2:] = -1e30
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device=DEV), torch.empty(5, device=DEV)
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, y=y, mean=mean, rstd=rstd)
    _, em, es, _ = layernorm(x, None, w, b, EPS)
    same = (x == x[:, :1]).all(dim=1)
    assert bool((rstd[~same] == 0).all()) and int(same.sum()) <= 1
    _inside(rstd[same], es[same], 2.0 ** -22 * es[same], "rstd")
    assert torch.equal(y, b.expand(5, cols))
    _inside(mean, em, 2.0 ** -18 * x.double().abs().mean(dim=1), "mean")


def test_rows_without_columns():
    x, w = torch.empty(3, 0, device=DEV), torch.empty(0, device=DEV)
    mean, rstd = torch.ones(3, device=DEV), torch.empty(3, device=DEV)
    nv.nvfp4_add_layernorm(x, w, 0.25, bias=w, y=torch.empty_like(x), mean=mean, rstd=rstd)
    assert mean.tolist() == [0.0] * 3 and rstd.tolist() == [2.0] * 3
    nv.nvfp4_add_layernorm_backward(x, x, w, mean, rstd, torch.empty_like(x), dweight=w, dbias=w)


# ---------------------------------------------------------------- backward


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, dtype):
    """dresidual: n is within 2^-22 (one difference, one product) of |h| + |mean| scaled, the two
    row means add at most 48 terms per chain: within 2^-18 of the terms' magnitude rstd (|g| +
    mean|g| + |n| mean|g n|) with |n| taken as (|h| + |mean|) rstd.  dweight, dbias: sums of
    `rows` terms, at most rows / CTAs + 80 additions per chain."""
    x, dy, w, _ = _inputs(rows, cols, dtype, rows + 3 * cols)
    h, dh = x, _inputs(rows, cols, dtype, 77)[1]
    _, mean, rstd, _ = layernorm(h, None, w, None, EPS)
    mean, rstd = mean.float(), rstd.float()
    half = half_ulp(dtype)
    for extra, p in ((None, 0.0), (dh, 0.1), (dh, 0.0), (None, 0.5)):
        mask = _mask(p, rows)
        dx, ok_x = guarded((rows, cols), dtype)
        dr, ok_r = guarded((rows, cols), dtype)
        dw, ok_w = guarded((cols,), torch.float32)
        db, ok_b = guarded((cols,), torch.float32)
        nv.nvfp4_add_layernorm_backward(dy, h, w, mean, rstd, dx, dweight=dw, dbias=db, dh=extra,
                                        mask=nv.Mask(*mask) if mask else None,
                                        dresidual=dr if mask else None)
        torch.cuda.synchronize()
        ex, er, ew, eb = layernorm_backward(dy, h, w, mean, rstd, extra, mask)
        s = rstd.double()[:, None]
        n = (h.double().abs() + mean.double().abs()[:, None]) * s
        g = (dy.double() * w.double()).abs()
        mag = s * (g + g.mean(1, keepdim=True) + n * (g * n).mean(1, keepdim=True))
        tol = 2.0 ** -18 * mag + (half + 2.0 ** -22) * er.abs()
        factor = 65536.0 / (65536 - threshold(p))
        # what is dropped is exactly 0 (a kept gradient of 0, as in a row of one column, is the
        # difference of rounded terms: within the terms' tolerance like any other)
        kept = drop(torch.ones_like(er), *mask) != 0 if mask else torch.ones_like(er, dtype=bool)
        _inside(dx, ex, torch.where(kept, tol * factor * (1 + 2.0 ** -22), 0.0), "dx")
        if mask:
            _inside(dr, er, tol, "dresidual")
        terms = rows * 2.0 ** -24 + 100 * 2.0 ** -24
        _inside(dw, ew, terms * (dy.double().abs() * n).sum(0), "dweight")
        _inside(db, eb, terms * dy.double().abs().sum(0), "dbias")
        for ok in (ok_x, ok_r, ok_w, ok_b):
            ok()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(9001, 24), (9001, 25), (7003, 512), (5003, 1000), (3001, 1001),
                                       (3001, 2048), (2777, 4096), (1501, 5008), (1501, 4097),
                                       (1300, 8192), (701, 12000), (401, 17001), (400, 20000), (5, 100)])
def test_parameter_gradients_of_small_integers_are_exact(rows, cols, dtype):
    """dy in {-2 .. 2}, h in {-3 .. 3}, mean 0, rstd 1, weight 1: n is h and every partial sum an integer
    below 6 * 9001 < 2^24, so no addition rounds, whatever their order: a row that is left out, counted
    twice or taken from its neighbour shows."""
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + cols)
    dy = torch.randint(-2, 3, (rows, cols), generator=g, device=DEV).to(dtype)
    h = torch.randint(-3, 4, (rows, cols), generator=g, device=DEV).to(dtype)
    w = torch.ones(cols, device=DEV, dtype=dtype)
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    dw, db, dx = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV), torch.empty_like(h)
    nv.nvfp4_add_layernorm_backward(dy, h, w, mean, rstd, dx, dweight=dw, dbias=db)
    assert torch.equal(dw.double(), (dy.double() * h.double()).sum(0))
    assert torch.equal(db.double(), dy.double().sum(0))


def test_backward_against_differences():
    """sum(dy * y) changes along a direction by the gradients' inner products (FP64 loss of
    the kernel's FP32 forward; the central difference's own error is of third order)."""
    _, x, w, b = _inputs(3, 200, torch.float32, 11)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    dy, vx, vr = (torch.randn(3, 200, generator=g, device=DEV) for _ in range(3))
    vw, vb = (torch.randn(200, generator=g, device=DEV) for _ in range(2))
    r, mask = torch.randn(3, 200, generator=g, device=DEV), nv.Mask(0.3, 4, 5)
    mean, rstd, y, h = (torch.empty(3, device=DEV), torch.empty(3, device=DEV),
                        torch.empty_like(x), torch.empty_like(x))
    nv.nvfp4_add_layernorm(x, w, EPS, bias=b, residual=r, mask=mask, h=h, y=y, mean=mean, rstd=rstd)
    dx, dr, dw, db = (torch.empty_like(t) for t in (x, x, w, w))
    nv.nvfp4_add_layernorm_backward(dy, h, w, mean, rstd, dx, dweight=dw, dbias=db, mask=mask,
                                    dresidual=dr)

    def loss(t):
        out = torch.empty_like(x)
        nv.nvfp4_add_layernorm(x + t * vx, w + t * vw, EPS, bias=b + t * vb, residual=r + t * vr,
                               mask=mask, y=out)
        return float((out.double() * dy.double()).sum())
    e = 2.0 ** -7
    slope = (loss(e) - loss(-e)) / (2 * e)
    want = sum(float((a.double() * v.double()).sum())
               for a, v in ((dx, vx), (dr, vr), (dw, vw), (db, vb)))
    # FP32 noise of the loss: 600 terms, 2^-22 each, over 2e; third order: e^2 of the terms, whose
    # third derivatives stay below 16 (n of up to 4, a step of |v| up to 4)
    scale = float((dy.double() * y.double()).abs().sum())
    assert abs(slope - want) <= scale * (2.0 ** -22 / e + 16 * e * e)


@pytest.mark.parametrize("cols", [1500, 1001])
def test_backward_in_place_and_repeatable(cols):
    x, dy, w, _ = _inputs(3700, cols, torch.bfloat16, 2)
    _, mean, rstd, _ = layernorm(x, None, w, None, EPS)
    mean, rstd, mask = mean.float(), rstd.float(), nv.Mask(0.1, 7, 8)
    dx, dr = torch.empty_like(x), torch.empty_like(x)
    dw, db, dw2, db2 = (torch.empty(cols, device=DEV) for _ in range(4))
    nv.nvfp4_add_layernorm_backward(dy, x, w, mean, rstd, dx, dweight=dw, dbias=db, dh=dy,
                                    mask=mask, dresidual=dr)
    dy2, x2 = dy.clone(), x.clone()
    nv.nvfp4_add_layernorm_backward(dy2, x2, w, mean, rstd, dy2, dweight=dw2, dbias=db2, dh=dy,
                                    mask=mask, dresidual=x2)
    assert torch.equal(dy2, dx) and torch.equal(x2, dr)
    assert torch.equal(dw2, dw) and torch.equal(db2, db)


def test_one_parameter_gradient_alone():
    x, dy, w, _ = _inputs(50, 300, torch.float32, 6)
    mean, rstd = torch.zeros(50, device=DEV), torch.ones(50, device=DEV)
    dw, db, dw1, db1 = (torch.empty(300, device=DEV) for _ in range(4))
    dx = torch.empty_like(x)
    nv.nvfp4_add_layernorm_backward(dy, x, w, mean, rstd, dx, dweight=dw, dbias=db)
    nv.nvfp4_add_layernorm_backward(dy, x, w, mean, rstd, dx, dweight=dw1)
    nv.nvfp4_add_layernorm_backward(dy, x, w, mean, rstd, dx, dbias=db1)
    assert torch.equal(dw, dw1) and torch.equal(db, db1)


def test_other_stream_and_workspace():
    x, dy, w, b = _inputs(640, 4096, torch.bfloat16, 8)
    _, mean, rstd, _ = layernorm(x, None, w, None, EPS)
    mean, rstd = mean.float(), rstd.float()
    dx, dx2, dw, dw2 = (torch.empty_like(t) for t in (x, x, mean.new_empty(4096), mean.new_empty(4096)))
    nv.nvfp4_add_layernorm_backward(dy, x, w, mean, rstd, dx, dweight=dw)
    ws, ok = guarded((nv.nvfp4_add_layernorm_backward_workspace_size(640, 4096),), torch.uint8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    nv.nvfp4_add_layernorm_backward(dy, x, w, mean, rstd, dx2, dweight=dw2, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    ok()
