"""Add + RMS norm with its quantized outputs, and its backward pass, on the GPU against
the FP64 definitions.

Tolerances, derived from the FP32 arithmetic: the sum of squares of a row takes at most
48 additions per chain (32 values in a thread, a warp tree of 5, up to 32 warps counted
with their growth), so mean(h^2) is within 2^-18 and rstd within 2^-19 + 2^-23 relative;
y adds two products: 2^-18 covers it.  Storing rounds once: 2^-8 (BF16) or 2^-24 (FP32)
relative.  E4M3 keeps 3 fraction bits: half a step is 2^-4 relative, or 2^-10 of the scale
below the normal range.  The NVFP4 codes are compared byte for byte with the oracle's
quantization of the FP32 y that the same call returns.
"""
import numpy as np
import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv
import oracle
from layer_reference import at_offset, guarded, half_ulp, norm, norm_backward

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 2.0 ** -18
SHAPES = [(1, 1), (1, 16), (3, 17), (5, 100), (9, 128), (2, 511), (33, 512), (7, 1000), (4, 1024),
          (700, 1024), (3, 2048), (65, 2056), (6, 4096), (2, 5000), (1, 8192), (400, 8192),
          (3, 8193), (2, 16384), (310, 16384), (2, 28672), (1, 32768), (0, 64)]
DTYPES = [torch.bfloat16, torch.float32]


def _inputs(rows, cols, dtype, seed, wdtype=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x = x * torch.exp(2 * torch.randn(rows, 1, generator=g, device=DEV))
    r = torch.randn(rows, cols, generator=g, device=DEV)
    w = 1 + 0.3 * torch.randn(cols, generator=g, device=DEV)
    return x.to(dtype), r.to(dtype), w.to(wdtype or dtype)


def _close(got, want, rel, what):
    err = (got.double() - want).abs()
    bad = err > rel * want.abs() + 1e-37
    assert not bool(bad.any()), f"{what}: {err[bad].max().item()} of {want[bad][:3].tolist()}"


# enough rows for every CTA to walk several, at each width of a row's team, with groups of
# rows cut by the last row
MANY = [(9001, 24), (7003, 512), (5003, 1000), (3001, 2048), (2777, 4096), (1501, 8192),
        (1501, 5008), (701, 16384), (701, 12000), (400, 20000), (9001, 25), (3001, 1001),
        (2501, 1002), (1501, 4097), (1001, 5004), (601, 9001), (401, 17001)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES + MANY)
def test_norm_and_sum(rows, cols, dtype):
    x, r, w = _inputs(rows, cols, dtype, rows * 31 + cols)
    for residual in (None, r):
        y, ok_y = guarded((rows, cols), dtype)
        rstd, ok_s = guarded((rows,), torch.float32)
        h, ok_h = guarded((rows, cols), dtype)
        nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=residual, h=h if residual is not None else None,
                             y=y, rstd=rstd)
        torch.cuda.synchronize()
        eh, es, ey = norm(x, residual, w, 1e-5)
        _close(rstd, es, REL, "rstd")
        _close(y, ey, REL + half_ulp(dtype), "y")
        if residual is not None:
            _close(h, eh, 2.0 ** -23 + half_ulp(dtype), "h")
        for ok in (ok_y, ok_s, ok_h):
            ok()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("rows,cols", SHAPES + MANY)
def test_fp8_output(rows, cols, dtype, block):
    x, r, w = _inputs(rows, cols, dtype, rows + cols, torch.float32)
    if rows > 2:
        x[1] = 0
        r[1] = 0
    blocks = -(-cols // 128) if block else 1
    codes, ok_c = guarded((rows, cols), torch.uint8)
    scale, ok_s = guarded((rows, blocks), torch.float32)
    nv.nvfp4_add_rmsnorm(x, w, 1e-6, residual=r, fp8=nv.Fp8Out(codes, scale, block))
    torch.cuda.synchronize()
    _, _, y = norm(x, r, w, 1e-6)
    width = 128 if block else max(cols, 1)
    pad = torch.nn.functional.pad(y, (0, blocks * width - cols)).reshape(rows, blocks, width)
    amax = pad.abs().amax(dim=2)
    want = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    _close(scale, want, 2 * REL, "scale")
    s = scale.double().repeat_interleave(width, dim=1)[:, :cols]
    v = codes.view(torch.float8_e4m3fn).double() * s
    assert bool(((v - y).abs() <= 2.0 ** -4 * 1.001 * y.abs() + 2.0 ** -10 * 1.001 * s).all())
    ok_c()
    ok_s()


@pytest.mark.parametrize("fos", [0, 1])
@pytest.mark.parametrize("bound", [448.0, 256.0])
@pytest.mark.parametrize("rows,cols", SHAPES + MANY[1:5] + MANY[10:16])
def test_nvfp4_output_is_the_quantize_of_y(rows, cols, bound, fos):
    if rows == 0:
        pytest.skip("no codes to compare")
    x, r, w = _inputs(rows, cols, torch.float32, 7 * rows + cols)
    if rows > 2:
        x[2] = 0
        r[2] = 0
    y = torch.empty_like(x)
    codes, ok_c = guarded((rows, (cols + 1) // 2), torch.uint8)
    scales, ok_s = guarded((rows, (cols + 15) // 16), torch.uint8)
    amax, ok_a = guarded((rows,), torch.float32)
    cfg = nv.Config(nv.NVFP4_ROW_SCALED, bound, fos, 0)
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=r, y=y, row=nv.Out(codes, scales, amax), cfg=cfg)
    torch.cuda.synchronize()
    ref = oracle.quantize(y.cpu().numpy(), "fp32", mode=oracle.ROW_SCALED, bound=bound,
                          four_over_six=bool(fos), columnwise=False)["row"]
    assert np.array_equal(amax.cpu().numpy().view(np.uint32), ref[2].view(np.uint32))
    assert np.array_equal(scales.cpu().numpy(), ref[1])
    assert np.array_equal(codes.cpu().numpy(), ref[0])
    for ok in (ok_c, ok_s, ok_a):
        ok()


def test_bf16_stream_gives_the_codes_of_its_fp32_copy():
    x, r, w = _inputs(40, 5008, torch.bfloat16, 3)
    cfg = nv.Config(nv.NVFP4_ROW_SCALED, 448.0, 0, 0)
    outs = []
    for cast in (lambda t: t, lambda t: t.float()):
        o = nv.alloc_out(40, 5008, 40)
        nv.nvfp4_add_rmsnorm(cast(x), cast(w), 1e-5, residual=cast(r), row=o, cfg=cfg)
        outs.append(o)
    torch.cuda.synchronize()
    for f in ("codes", "scales", "amax"):
        assert torch.equal(getattr(outs[0], f), getattr(outs[1], f))


def test_given_amax():
    x, _, w = _inputs(9, 320, torch.float32, 5)
    y = torch.empty_like(x)
    for mode, n in ((nv.NVFP4_ROW_SCALED, 9), (nv.NVFP4_PER_TENSOR, 1)):
        given = torch.full((n,), 3.25, device=DEV) + torch.arange(n, device=DEV)
        o = nv.alloc_out(9, 320, n)
        o.amax_in = given
        nv.nvfp4_add_rmsnorm(x, w, 1e-5, y=y, row=o, cfg=nv.Config(mode, 448.0, 0, 0))
        torch.cuda.synchronize()
        ref = oracle.quantize(y.cpu().numpy(), "fp32", mode=mode, bound=448.0, columnwise=False,
                              row_amax_in=given.cpu().numpy())["row"]
        assert torch.equal(o.amax, given)
        assert np.array_equal(o.codes.cpu().numpy(), ref[0])
        assert np.array_equal(o.scales.cpu().numpy(), ref[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_unaligned_starts(dtype, offset):
    x, r, w = _inputs(6, 1040, dtype, offset)
    want = torch.empty_like(x)
    codes, scale = torch.empty(6, 1040, dtype=torch.uint8, device=DEV), torch.empty(6, device=DEV)
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=r, y=want)
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=r, fp8=nv.Fp8Out(codes, scale, 0))
    y, ok = guarded((6, 1040), dtype, offset=offset)
    h, ok_h = guarded((6, 1040), dtype, offset=offset)
    c, ok_c = guarded((6, 1040), torch.uint8, offset=offset)
    s2 = torch.empty(6, device=DEV)
    xo, ro, wo = (at_offset(t, offset) for t in (x, r, w))
    nv.nvfp4_add_rmsnorm(xo, wo, 1e-5, residual=ro, h=h, y=y)
    nv.nvfp4_add_rmsnorm(xo, wo, 1e-5, residual=ro, fp8=nv.Fp8Out(c, s2, 0))
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(c, codes) and torch.equal(s2, scale)
    for o in (ok, ok_h, ok_c):
        o()


@pytest.mark.parametrize("cols", [2048, 1003])
def test_in_place_stream(cols):
    """The sum may replace x or the residual, y may replace x."""
    x, r, w = _inputs(12, cols, torch.bfloat16, 1)
    h, y = torch.empty_like(x), torch.empty_like(x)
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=r, h=h, y=y)
    r2, y2 = r.clone(), torch.empty_like(x)
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=r2, h=r2, y=y2)
    assert torch.equal(r2, h) and torch.equal(y2, y)
    x2, r3 = x.clone(), r.clone()
    nv.nvfp4_add_rmsnorm(x2, w, 1e-5, residual=r3, h=r3, y=x2)
    assert torch.equal(r3, h) and torch.equal(x2, y)


def test_extreme_rows():
    """Rows of zeros, of the smallest and the largest values the squares allow."""
    for dtype in DTYPES:
        x = torch.zeros(4, 64, dtype=dtype, device=DEV)
        x[1] = 1e-30
        x[2] = 1e17
        x[3, 5] = -2.0
        w = torch.ones(64, dtype=dtype, device=DEV)
        y, rstd = torch.empty_like(x), torch.empty(4, device=DEV)
        nv.nvfp4_add_rmsnorm(x, w, 1e-6, y=y, rstd=rstd)
        eh, es, ey = norm(x, None, w, 1e-6)
        _close(rstd, es, REL, "rstd")
        _close(y, ey, REL + half_ulp(dtype), "y")
        o = nv.alloc_out(4, 64, 4)
        nv.nvfp4_add_rmsnorm(x, w, 1e-6, row=o, cfg=nv.Config(nv.NVFP4_ROW_SCALED, 448.0, 0, 0))
        assert int(o.codes[0].sum()) == 0 and float(o.amax[0]) == 0.0


def test_a_bad_row_leaves_the_others_alone():
    x, r, w = _inputs(5, 640, torch.float32, 9)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=r, y=y)
    x[1, 3], x[3, 600] = float("nan"), float("inf")
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=r, y=y2)
    assert bool(y2[1].isnan().all()) and bool(y2[3, 600].isnan())
    for i in (0, 2, 4):
        assert torch.equal(y[i], y2[i])


# ---------------------------------------------------------------- backward


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES + [(2500, 96), (1300, 2048)] + MANY)
def test_backward(rows, cols, dtype):
    """dx: products of FP32 values and one row mean of at most 48 additions per chain:
    within 2^-18 of the terms' magnitude |g| + |n| mean|g n|; dweight: sums of `rows`
    products, at most rows / CTAs + 80 additions per chain."""
    h, dy, w = _inputs(rows, cols, dtype, rows + 3 * cols)
    dh = _inputs(rows, cols, dtype, 77)[1]
    _, rstd64, _ = norm(h, None, w, 1e-5)
    rstd = rstd64.float()
    for extra in (None, dh):
        dx, ok_x = guarded((rows, cols), dtype)
        dw, ok_w = guarded((cols,), torch.float32)
        nv.nvfp4_add_rmsnorm_backward(dy, h, w, rstd, dx, dweight=dw, dh=extra)
        torch.cuda.synchronize()
        ex, ew = norm_backward(dy, h, w, rstd, extra)
        n, g = h.double() * rstd.double()[:, None], dy.double() * w.double()
        mag = rstd.double()[:, None] * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
        tol = REL * mag + (half_ulp(dtype) + 2.0 ** -23) * ex.abs()
        assert bool(((dx.double() - ex).abs() <= tol + 1e-37).all())
        tol_w = (rows + 100) * 2.0 ** -24 * (dy.double() * n).abs().sum(0)
        assert bool(((dw.double() - ew).abs() <= tol_w + 1e-37).all())
        ok_x()
        ok_w()


def test_backward_against_differences():
    """sum(dy * y) changes along a direction by the gradients' inner products (FP64 loss of
    the kernel's FP32 forward; the central difference's own error is of third order)."""
    x, r, w = _inputs(3, 200, torch.float32, 11)
    x = r  # rows of unit size
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    dy, vx = (torch.randn(3, 200, generator=g, device=DEV) for _ in range(2))
    vw = torch.randn(200, generator=g, device=DEV)
    rstd, y = torch.empty(3, device=DEV), torch.empty_like(x)
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, y=y, rstd=rstd)
    dx, dw = torch.empty_like(x), torch.empty(200, device=DEV)
    nv.nvfp4_add_rmsnorm_backward(dy, x, w, rstd, dx, dweight=dw)

    def loss(t):
        out = torch.empty_like(x)
        nv.nvfp4_add_rmsnorm(x + t * vx, w + t * vw, 1e-5, y=out)
        return float((out.double() * dy.double()).sum())
    e = 2.0 ** -7
    slope = (loss(e) - loss(-e)) / (2 * e)
    want = float((dx.double() * vx.double()).sum() + (dw.double() * vw.double()).sum())
    # FP32 noise of the loss: 600 terms, 2^-22 each, over 2e; third order: e^2 of the terms
    scale = float((dy.double() * y.double()).abs().sum())
    assert abs(slope - want) <= scale * (2.0 ** -22 / e + 2 * e * e)


def test_backward_in_place_and_repeatable():
    h, dy, w = _inputs(700, 1500, torch.bfloat16, 2)
    rstd = norm(h, None, w, 1e-5)[1].float()
    dx, dw = torch.empty_like(h), torch.empty(1500, device=DEV)
    nv.nvfp4_add_rmsnorm_backward(dy, h, w, rstd, dx, dweight=dw, dh=dy)
    dy2, dw2 = dy.clone(), torch.empty_like(dw)
    nv.nvfp4_add_rmsnorm_backward(dy2, h, w, rstd, dy2, dweight=dw2, dh=dy)
    assert torch.equal(dy2, dx) and torch.equal(dw2, dw)


def test_other_stream():
    x, r, w = _inputs(64, 4096, torch.bfloat16, 8)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=r, y=y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=r, y=y2, stream=s)
    s.synchronize()
    assert torch.equal(y, y2)


# rows that start on any element, enough of them to run through shared memory in 16-byte
# units at each team width, with a last few bytes that fill no unit
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(50003, 25), (40009, 511), (20011, 513), (9001, 1001),
                                       (9003, 2047), (5003, 2049), (5003, 4097), (4001, 5001),
                                       (2003, 6145), (1501, 9001), (1301, 12002)])
def test_many_unaligned_rows(rows, cols, dtype):
    test_norm_and_sum(rows, cols, dtype)
    test_backward(rows, cols, dtype)
    if cols < 3000:
        test_fp8_output(rows, cols, dtype, 128)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_unaligned_rows_in_place(dtype):
    """h may be the residual, and dx may be dy: the units around a row's group hold its
    neighbours' elements, which may have been replaced by then."""
    x, r, w = _inputs(9001, 1001, dtype, 3)
    h, y = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(9001, device=DEV)
    nv.nvfp4_add_rmsnorm(x, w, 1e-6, residual=r, h=h, y=y, rstd=rstd)
    r2, y2 = r.clone(), torch.empty_like(x)
    nv.nvfp4_add_rmsnorm(x, w, 1e-6, residual=r2, h=r2, y=y2, rstd=rstd)
    assert torch.equal(r2, h) and torch.equal(y2, y)
    dx, dw = torch.empty_like(x), torch.empty(1001, device=DEV)
    nv.nvfp4_add_rmsnorm_backward(x, h, w, rstd, dx, dh=r, dweight=dw)
    dy, dw2 = x.clone(), torch.empty(1001, device=DEV)
    nv.nvfp4_add_rmsnorm_backward(dy, h, w, rstd, dy, dh=r, dweight=dw2)
    assert torch.equal(dy, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [3, 40000])
def test_rows_without_columns(rows, dtype):
    """Nothing to sum: rstd is 1/sqrt(eps), scales are 1, the amax is 0."""
    x, w = torch.empty(rows, 0, dtype=dtype, device=DEV), torch.empty(0, dtype=dtype, device=DEV)
    r, h, y = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    rstd, ok_r = guarded((rows,), torch.float32)
    for block in (0, 128):
        scale, ok = guarded((rows, 0 if block else 1), torch.float32)
        codes = torch.empty(rows, 0, dtype=torch.uint8, device=DEV)
        rstd.zero_()
        nv.nvfp4_add_rmsnorm(x, w, 0.25, residual=r, h=h, y=y, rstd=rstd,
                             fp8=nv.Fp8Out(codes, scale, block))
        torch.cuda.synchronize()
        assert bool((rstd == 2.0).all()) and bool((scale == 1.0).all())
        ok()
    amax, ok = guarded((rows,), torch.float32)
    none = torch.empty(rows, 0, dtype=torch.uint8, device=DEV)
    nv.nvfp4_add_rmsnorm(x, w, 0.25, row=nv.Out(none, none, amax),
                         cfg=nv.Config(nv.NVFP4_ROW_SCALED, 448.0, 0, 0))
    torch.cuda.synchronize()
    assert bool((amax == 0.0).all())
    ok()
    ok_r()
    # and back: no dx, no dweight
    nv.nvfp4_add_rmsnorm_backward(y, h, w, rstd, x, dweight=torch.empty(0, device=DEV))
    torch.cuda.synchronize()


def _fp8(x, w, r, block):
    """The FP32 y of a norm with its E4M3 codes and scale, from one call."""
    rows, cols = x.shape
    y = torch.empty_like(x)
    codes = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    scale = torch.empty(rows, -(-cols // 128) if block else 1, device=DEV)
    nv.nvfp4_add_rmsnorm(x, w, 1e-6, residual=r, y=y, fp8=nv.Fp8Out(codes, scale, block))
    torch.cuda.synchronize()
    each = scale.repeat_interleave(128 if block else cols, dim=1)[:, :cols]
    return y, codes.view(torch.float8_e4m3fn), each


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("rows,cols", [(3000, 4096), (2001, 4001), (4, 512)])
def test_fp8_codes_are_those_of_the_quotient(rows, cols, block):
    """code = E4M3(y / scale) with the stored scale: every code of the FP32 quotient."""
    x, r, w = _inputs(rows, cols, torch.float32, 13)
    y, codes, scale = _fp8(x, w, r, block)
    want = (y / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    assert torch.equal(codes.float(), want.float())


@pytest.mark.parametrize("block", [0, 128])
def test_fp8_of_tiny_values(block):
    """A row whose maximum lies below 448 * 2^-126, and blocks of such values in ordinary
    rows (weights of 1e-36): the scale stops at 2^-126, and code * scale is y within half a
    step of E4M3 all the same."""
    w = torch.ones(1024, device=DEV)
    w[128:256] = 1e-36
    w[512:640] = 3e-38
    x, _, _ = _inputs(6, 1024, torch.float32, 4)
    x[2] = x[2] / x[2].abs().max() * 1e-39  # y: about 1e-36
    x[4] = x[4] / x[4].abs().max() * 5e-39
    y, codes, scale = _fp8(x, w, None, block)
    assert float(scale[2].min()) >= 2.0 ** -126
    v, s, want = codes.double() * scale.double(), scale.double(), y.double()
    assert bool(((v - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * s).all())
    # the largest is not lost: its code times the scale is within half a step of it
    top = want[2].abs().max()
    assert top > 0 and abs(v[2].abs().max() - top) <= 2.0 ** -4 * top


def test_maxima_skip_nan():
    """A row with an infinity has rstd 0, so its other values are 0 and that one is NaN; rows of
    zeros with eps = 0 have an infinite rstd and are NaN throughout.  The maxima skip NaN:
    they are 0 and the scales 1, and the rows between are as they were."""
    x = torch.ones(4, 256, device=DEV)
    x[0, 200], x[2] = float("inf"), 0.0
    w = torch.full((256,), 2.0, device=DEV)
    for block in (0, 128):
        codes = torch.empty(4, 256, dtype=torch.uint8, device=DEV)
        scale = torch.empty(4, 2 if block else 1, device=DEV)
        y = torch.empty_like(x)
        nv.nvfp4_add_rmsnorm(x, w, 0.0, y=y, fp8=nv.Fp8Out(codes, scale, block))
        torch.cuda.synchronize()
        assert bool(y[0, 200].isnan()) and bool(y[2].isnan().all())
        assert float(y[0, :200].abs().max()) == 0.0
        assert bool((scale[0] == 1.0).all()) and bool((scale[2] == 1.0).all())
        for i in (1, 3):
            v = codes[i].view(torch.float8_e4m3fn).float() * scale[i].repeat_interleave(
                256 // scale.shape[1])
            assert bool(((v - y[i]).abs() <= 2.0 ** -4 * y[i].abs()).all())
    o = nv.alloc_out(4, 256, 4)
    nv.nvfp4_add_rmsnorm(x, w, 0.0, row=o, cfg=nv.Config(nv.NVFP4_ROW_SCALED, 448.0, 0, 0))
    torch.cuda.synchronize()
    assert float(o.amax[0]) == 0.0 and float(o.amax[2]) == 0.0 and float(o.amax[1]) > 0.0
