"""The NVFP4 product with bias, activation and residual in its epilogue, and the backward
pass of bias and activation, on the GPU against the FP64 definitions.

Tolerances.  The product: as in test_gpu_gemm, (k 2^-23 + 2^-21) sum|terms|.  Adding the
bias rounds once (2^-23 of |z|).  The activations' slopes are below 1.13, and their own
evaluation (one exponential, one reciprocal) is within 2^-20 (1 + |z|) of the value: the
exponential's relative error is 2^-22 + |u| 2^-23, which p (1 - p) |z| turns into less than
2^-20.  Storing rounds once.
"""
import numpy as np
import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv
import oracle
import workloads
from layer_reference import ACTS, act, act_slope, at_offset, guarded, half_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda"
RS, PT = nv.NVFP4_ROW_SCALED, nv.NVFP4_PER_TENSOR
DTYPES = [torch.bfloat16, torch.float32]


def _operands(m, n, k, seed, modes=(RS, RS), bounds=(448.0, 448.0)):
    host, dev = [], []
    for i, lines in enumerate((m, n)):
        c, s, a = workloads.nvfp4_operand(lines, k, seed + i, modes[i] == RS)
        a = a * (0.1 / a.max())  # values of order one for the activations
        host.append(dict(codes=c.numpy(), scales=s.numpy(), amax=a.numpy(),
                         row_scaled=modes[i] == RS, bound=bounds[i]))
        dev.append(nv.Operand(c.to(DEV), s.to(DEV), a.to(DEV), modes[i], bounds[i]))
    z, mag = oracle.gemm(host[0], host[1], with_abs=True)
    return dev, torch.from_numpy(z).to(DEV), torch.from_numpy(mag).to(DEV)


def _check(m, n, k, dtype, name, bias, residual, keep, seed, modes=(RS, RS),
           bounds=(448.0, 448.0), offset=0):
    (a, b), z, mag = _operands(m, n, k, seed, modes, bounds)
    scale = 1.0 / float(z.abs().max().clamp(min=1e-6)) * 4.0
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    b.amax = (b.amax * scale).float()  # |z| up to about 4
    z, mag = z * scale, mag * scale
    tol = (k * 2.0 ** -23 + 2.0 ** -20) * mag
    bv = torch.randn(n, generator=g, device=DEV).to(bias) if bias is not None else None
    if bv is not None:
        z = z + bv.double()
        tol = tol + 2.0 ** -23 * z.abs()
    d, ok_d = guarded((m, n), dtype, offset=offset)
    zz, ok_z = guarded((m, n), dtype, offset=offset)
    want = act(z, name)
    tol_d = 1.13 * tol + (2.0 ** -20 * (1 + z.abs()) if name in ("gelu", "silu") else 0)
    res = None
    if residual:
        res = at_offset(torch.randn(m, n, generator=g, device=DEV).to(dtype), offset)
        want = want + res.double()
        tol_d = tol_d + 2.0 ** -23 * want.abs()
    nv.nvfp4_gemm_bias_act(a, b, d, bias=bv, act=ACTS[name], residual=res, z=zz if keep else None)
    torch.cuda.synchronize()
    half = half_ulp(dtype)
    assert bool(((d.double() - want).abs() <= tol_d * (1 + half) + half * want.abs()).all())
    if keep:
        assert bool(((zz.double() - z).abs() <= tol * (1 + half) + half * z.abs()).all())
    ok_d()
    ok_z()


# one token to several tiles, odd sizes on both axes, K tails of a K tile
SIZES = [(1, 256, 256), (1, 1, 32), (1, 4097, 512), (2, 100, 96), (7, 300, 320), (8, 512, 1024),
         (16, 1000, 544), (17, 129, 64), (31, 64, 800), (33, 640, 256), (64, 255, 288),
         (65, 384, 512), (100, 77, 96), (128, 256, 128), (129, 257, 160), (200, 520, 992),
         (300, 500, 320),
         # past the few-rows kernel: row and tile counts that go to the tiled one
         (385, 6000, 64), (450, 5000, 96), (1000, 2561, 160)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_gemm_bias_act(m, n, k, dtype):
    name = list(ACTS)[(m + n + k // 32) % 4]
    _check(m, n, k, dtype, name, torch.float32, True, True, m + n + k)
    _check(m, n, k, dtype, "gelu", None, False, False, m + n + k + 1, (PT, RS), (256.0, 448.0))


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("bias", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual,keep", [(False, True), (True, False)])
@pytest.mark.parametrize("m", [1, 5, 40, 150])
def test_epilogue_combinations(m, name, bias, residual, keep):
    _check(m, 272, 160, torch.bfloat16, name, bias, residual, keep, 3 * m)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m", [1, 9, 140])
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_unaligned_outputs(m, offset, dtype):
    _check(m, 264, 128, dtype, "silu", torch.float32, True, True, m, offset=offset)


@pytest.mark.parametrize("m,n", [(1, 5000), (40, 20000), (1, 40000), (129, 10100)])
def test_tiles_cut_along_k(m, n):
    """More tiles than SMs with a rest that is cut along K, beside whole tiles."""
    _check(m, n, 2080, torch.bfloat16, "gelu", torch.float32, True, True, m)


@pytest.mark.parametrize("m", [1, 20, 130])
def test_long_k(m):
    """Long sums, every K tile of a split: the bound is still a small part of one term's
    block, because every operand value is drawn alike."""
    _check(m, 320, 8192 + 96, torch.float32, "none", torch.float32, False, True, 5)


def test_plain_epilogue_is_the_gemm():
    """Without bias, activation and residual d is nvfp4_gemm's (many rows: the same sums)."""
    (a, b), _, _ = _operands(1100, 2400, 512, 4)
    d, e = (torch.empty(1100, 2400, device=DEV) for _ in range(2))
    nv.nvfp4_gemm(a, b, d)
    nv.nvfp4_gemm_bias_act(a, b, e)
    assert torch.equal(d, e)


@pytest.mark.parametrize("m", [3, 150])
def test_residual_in_place_and_repeatable(m):
    (a, b), _, _ = _operands(m, 384, 2048, 6)
    res = torch.randn(m, 384, device=DEV).bfloat16()
    d, e = torch.empty_like(res), res.clone()
    nv.nvfp4_gemm_bias_act(a, b, d, act=nv.NVFP4_ACT_GELU, residual=res)
    nv.nvfp4_gemm_bias_act(a, b, e, act=nv.NVFP4_ACT_GELU, residual=e)
    assert torch.equal(d, e)
    for _ in range(3):
        nv.nvfp4_gemm_bias_act(a, b, e, act=nv.NVFP4_ACT_GELU, residual=res)
        assert torch.equal(d, e)


def test_empty_sum_and_empty_outputs():
    bias = torch.randn(40, device=DEV)
    empty = lambda lines: nv.Operand(torch.empty(lines, 0, dtype=torch.uint8, device=DEV),  # noqa: E731
                                     torch.empty(lines, 0, dtype=torch.uint8, device=DEV),
                                     torch.ones(lines, device=DEV), RS, 448.0)
    res = torch.randn(3, 40, device=DEV)
    d, z = torch.empty_like(res), torch.empty_like(res)
    nv.nvfp4_gemm_bias_act(empty(3), empty(40), d, bias=bias, act=nv.NVFP4_ACT_RELU, residual=res,
                           z=z)
    assert torch.equal(z, bias.expand(3, 40)) and torch.equal(d, bias.clamp(min=0) + res)
    (a, b), _, _ = _operands(4, 40, 64, 1)
    none = nv.Operand(a.codes[:0], a.scales[:0], a.amax[:0], RS, 448.0)
    nv.nvfp4_gemm_bias_act(none, b, torch.empty(0, 40, device=DEV), bias=bias)


@pytest.mark.parametrize("m", [2, 140])
def test_workspace_and_stream(m):
    """A given workspace of the stated size, on another stream."""
    (a, b), _, _ = _operands(m, 512, 1024, 9)
    d, e = (torch.empty(m, 512, device=DEV) for _ in range(2))
    nv.nvfp4_gemm_bias_act(a, b, d, act=nv.NVFP4_ACT_SILU)
    need = nv.nvfp4_gemm_bias_act_workspace_size(m, 512, 1024)
    ws, ok = guarded((max(need, 256),), torch.uint8)
    ws.random_(0, 256)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):  # what one call leaves in the workspace does not matter to the next
        e.zero_()
        torch.cuda.synchronize()
        nv.nvfp4_gemm_bias_act(a, b, e, act=nv.NVFP4_ACT_SILU, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(d, e)
    ok()


# ---------------------------------------------------------------- backward

BACK = [(1, 1), (1, 4096), (3, 16), (5, 17), (40, 64), (1000, 8), (129, 100), (300, 512),
        (77, 513), (64, 5000), (2000, 1024), (5, 28672), (700, 2056), (0, 8), (8, 0),
        (3000, 1001), (999, 515), (1200, 2050)]


def _backward_inputs(rows, cols, dtype, seed, spread=3.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    z = (spread * torch.randn(rows, cols, generator=g, device=DEV)).to(dtype)
    return z, torch.randn(rows, cols, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("rows,cols", BACK)
def test_backward(rows, cols, name, dtype):
    """act' is within 2^-19 (its terms p and z p (1 - p) u' are bounded by 1.2 and each
    within 2^-20); the sums take rows additions of values bounded by |dd| 1.2."""
    z, dd = _backward_inputs(rows, cols, dtype, rows + cols)
    dz, ok_z = guarded((rows, cols), dtype)
    dbias, ok_b = guarded((cols,), torch.float32)
    ra, ok_r = guarded((rows,), torch.float32)
    ca, ok_c = guarded((cols,), torch.float32)
    nv.nvfp4_bias_act_backward(dd, z if name != "none" else None, ACTS[name], dz, dbias=dbias,
                               row_amax=ra, col_amax=ca)
    torch.cuda.synchronize()
    want = dd.double() * act_slope(z.double(), name)
    tol = 2.0 ** -19 * dd.double().abs() + half_ulp(dtype) * 1.001 * want.abs()
    assert bool(((dz.double() - want).abs() <= tol).all())
    exact = name in ("none", "relu")
    tol_b = (rows * 2.0 ** -24 + (0 if exact else 2.0 ** -19)) * 1.2 * dd.double().abs().sum(0)
    assert bool(((dbias.double() - want.sum(0)).abs() <= tol_b).all())
    mags = torch.nn.functional.pad(dz.float().abs(), (0, 1, 0, 1))
    assert torch.equal(ra, mags.amax(dim=1)[:rows])
    assert torch.equal(ca, mags.amax(dim=0)[:cols])
    for ok in (ok_z, ok_b, ok_r, ok_c):
        ok()


def test_backward_against_differences():
    z, dd = _backward_inputs(20, 300, torch.float32, 3, 1.5)
    z, dd, e = z.double(), dd.double(), 2.0 ** -12
    for name in ("gelu", "silu"):
        dz, zf = torch.empty(20, 300, device=DEV), z.float()
        nv.nvfp4_bias_act_backward(dd.float(), zf, ACTS[name], dz)
        slope = (act(zf.double() + e, name) - act(zf.double() - e, name)) / (2 * e)
        # third derivatives below 2: e^2 / 6 * 2
        assert bool(((dz.double() - dd * slope).abs() <= dd.abs() * (2.0 ** -19 + e * e)).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_arguments_stay_finite(dtype):
    """Saturated activations: the slope is 0 or 1, with no product of 0 and infinity."""
    z = torch.tensor([[-3e38, -1e20, -1e4, -100.0, -20.0, 20.0, 100.0, 1e4, 1e20, 3e38]],
                     device=DEV).to(dtype)
    dd = torch.full_like(z, 2.0)
    for name in ("gelu", "silu", "relu"):
        dz = torch.empty_like(z)
        nv.nvfp4_bias_act_backward(dd, z, ACTS[name], dz)
        want = torch.tensor([[0.0] * 5 + [2.0] * 5], device=DEV)
        assert bool(((dz.float() - want).abs() <= 1e-6).all()), (name, dz)


def test_backward_feeds_the_quantization():
    """The maxima are the amax that the quantization of dz computes, so giving them
    changes no byte."""
    z, dd = _backward_inputs(260, 512, torch.bfloat16, 4)
    dz, ra, ca = torch.empty_like(z), torch.empty(260, device=DEV), torch.empty(512, device=DEV)
    nv.nvfp4_bias_act_backward(dd, z, nv.NVFP4_ACT_GELU, dz, row_amax=ra, col_amax=ca)
    cfg = nv.Config(RS, 448.0, 0, 0)
    outs = []
    for given in (False, True):
        r, c = nv.alloc_out(260, 512, 260), nv.alloc_out(512, 260, 512)
        if given:
            r.amax_in, c.amax_in = ra, ca
        nv.nvfp4_quantize_both(dz, cfg, r, c)
        outs.append((r, c))
    torch.cuda.synchronize()
    for x, y in zip(*outs):
        for f in ("codes", "scales", "amax"):
            assert np.array_equal(getattr(x, f).cpu().numpy(), getattr(y, f).cpu().numpy())


def test_backward_in_place_unaligned_and_partial():
    z, dd = _backward_inputs(90, 1000, torch.bfloat16, 6)
    dz, db = torch.empty_like(z), torch.empty(1000, device=DEV)
    nv.nvfp4_bias_act_backward(dd, z, nv.NVFP4_ACT_SILU, dz, dbias=db)
    for offset in (0, 1, 8):
        zo, do = at_offset(z, offset), at_offset(dd, offset)
        db2 = torch.empty_like(db)
        nv.nvfp4_bias_act_backward(do, zo, nv.NVFP4_ACT_SILU, do, dbias=db2)
        assert torch.equal(do, dz) and torch.equal(db, db2)
        zo2, do2 = at_offset(z, offset), at_offset(dd, offset)
        nv.nvfp4_bias_act_backward(do2, zo2, nv.NVFP4_ACT_SILU, zo2)
        assert torch.equal(zo2, dz)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("m,n", [(3, 41), (1, 1), (700, 513)])
def test_empty_sum_of_every_activation(m, n, name, dtype):
    """k == 0 against the definition, with the same evaluation as every other k: the values
    of a product with all-zero codes, byte for byte."""
    g = torch.Generator(device=DEV)
    g.manual_seed(m + n)
    bias = 6 * torch.randn(n, generator=g, device=DEV)
    res = torch.randn(m, n, generator=g, device=DEV).to(dtype)

    def zeros(lines, k):
        return nv.Operand(torch.zeros(lines, k // 2, dtype=torch.uint8, device=DEV),
                          torch.zeros(lines, k // 16, dtype=torch.uint8, device=DEV),
                          torch.ones(lines, device=DEV), RS, 448.0)
    out = []
    for k in (0, 64):
        d, ok_d = guarded((m, n), dtype)
        z, ok_z = guarded((m, n), dtype)
        nv.nvfp4_gemm_bias_act(zeros(m, k), zeros(n, k), d, bias=bias, act=ACTS[name],
                               residual=res, z=z)
        torch.cuda.synchronize()
        ok_d()
        ok_z()
        out.append((d, z))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    zz = bias.double().expand(m, n)
    want = act(zz, name) + res.double()
    tol = 2.0 ** -20 * (1 + zz.abs()) + (2.0 ** -23 + half_ulp(dtype)) * 1.01 * want.abs()
    assert bool(((out[0][0].double() - want).abs() <= tol).all())


def _moved(o, codes, scales, amax):
    """The operand with its tensors starting off their allocations' alignment."""
    return nv.Operand(at_offset(o.codes, codes), at_offset(o.scales, scales),
                      at_offset(o.amax, amax), o.mode, o.bound)


@pytest.mark.parametrize("m,n,k", [(1, 300, 544), (5, 129, 2080), (40, 1000, 96), (64, 256, 8224),
                                   (300, 500, 320), (129, 10100, 1056), (450, 5000, 96)])
@pytest.mark.parametrize("start", [1, 2, 8])
def test_scales_that_start_anywhere(m, n, k, start):
    """Scale tensors that start off 16 bytes are copied byte by byte, and change nothing: every
    scale reaches the place that it has otherwise."""
    (a, b), _, _ = _operands(m, n, k, m + n + k)
    bias = torch.randn(n, device=DEV)
    want = torch.empty(m, n, device=DEV)
    nv.nvfp4_gemm_bias_act(a, b, want, bias=bias, act=nv.NVFP4_ACT_GELU)
    for x, w in ((start, 0), (0, start), (start, start)):
        d, ok = guarded((m, n), torch.float32)
        nv.nvfp4_gemm_bias_act(_moved(a, 16, x, 1), _moved(b, 32, w, 3), d, bias=bias,
                               act=nv.NVFP4_ACT_GELU)
        torch.cuda.synchronize()
        assert torch.equal(d, want)
        ok()
