"""Refusals of the layer operators: argument checks that run before any CUDA call (no
GPU needed), and the binding's own checks."""
import ctypes

import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv

R = ctypes.byref
BF, FP = nv.NVFP4_IN_BF16, nv.NVFP4_IN_FP32
BASE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from nvfp4_precision_quantization_gb300 import build
    build.build()
    return nv.load_library()


def _norm(lib, x=BASE, residual=None, dtype=BF, weight=2 * BASE, wdtype=BF, rows=4, cols=64,
          eps=1e-5, h=None, y=3 * BASE, rstd=None, fp8=None, cfg=None, row=None):
    return lib.nvfp4_add_rmsnorm(x, residual, dtype, weight, wdtype, rows, cols, eps, h, y, rstd,
                                 fp8, cfg, row, None)


def test_norm_refusals(lib):
    inv, uns = nv.NVFP4_ERR_INVALID, nv.NVFP4_ERR_UNSUPPORTED
    row = nv._COut(5 * BASE, 6 * BASE, 7 * BASE, None)
    rs = nv.Config(nv.NVFP4_ROW_SCALED, 448.0, 0, 0)
    for want, word, kw in (
            (inv, "in_dtype", dict(dtype=7)), (inv, "weight_dtype", dict(wdtype=-1)),
            (inv, "rows and cols", dict(rows=-1)), (uns, "MAX_COLS", dict(cols=32769)),
            (inv, "weight is NULL", dict(weight=None)), (inv, "x is NULL", dict(x=None)),
            (inv, "eps", dict(eps=-1.0)), (inv, "eps", dict(eps=float("nan"))),
            (inv, "residual", dict(h=4 * BASE)), (inv, "no output", dict(y=None)),
            (inv, "aligned", dict(x=BASE + 1)), (inv, "aligned", dict(dtype=FP, x=BASE + 2)),
            (inv, "h overlaps y", dict(residual=8 * BASE, h=3 * BASE)),
            (inv, "without being it", dict(y=BASE + 2)),
            (inv, "without being it", dict(residual=8 * BASE, h=8 * BASE - 16)),
            (inv, "fp8->block", dict(fp8=R(nv._CFp8Out(BASE, BASE, 64)))),
            (inv, "fp8->codes", dict(fp8=R(nv._CFp8Out(None, BASE, 0)))),
            (inv, "fp8->scale", dict(fp8=R(nv._CFp8Out(BASE, None, 128)))),
            (uns, "one call", dict(fp8=R(nv._CFp8Out(BASE, BASE, 0)), row=R(row), cfg=R(rs))),
            (inv, "cfg is NULL", dict(row=R(row))),
            (inv, "bound", dict(row=R(row), cfg=R(nv.Config(nv.NVFP4_ROW_SCALED, 1.0, 0, 0)))),
            (uns, "16x16", dict(row=R(row), cfg=R(nv.Config(nv.NVFP4_PER_TENSOR, 448.0, 0, 1)))),
            (uns, "amax_in", dict(row=R(row), cfg=R(nv.Config(nv.NVFP4_PER_TENSOR, 448.0, 0, 0)))),
            (inv, "codes", dict(row=R(nv._COut(None, BASE, BASE, None)), cfg=R(rs)))):
        assert _norm(lib, **kw) == want, (word, nv.nvfp4_last_error())
        assert word in nv.nvfp4_last_error(), (word, nv.nvfp4_last_error())
    assert _norm(lib, rows=0) == nv.NVFP4_OK


def _back(lib, dy=BASE, h=2 * BASE, dh=None, dtype=BF, w=3 * BASE, wdtype=BF, rstd=4 * BASE,
          rows=4, cols=64, dx=5 * BASE, dw=6 * BASE, ws=7 * BASE, size=1 << 20):
    return lib.nvfp4_add_rmsnorm_backward(dy, h, dh, dtype, w, wdtype, rstd, rows, cols, dx, dw,
                                          ws, size, None)


def test_norm_backward_refusals(lib):
    inv, uns = nv.NVFP4_ERR_INVALID, nv.NVFP4_ERR_UNSUPPORTED
    need = nv.nvfp4_add_rmsnorm_backward_workspace_size(4, 64)
    assert need == 4 * 4 * 64
    for want, word, kw in (
            (inv, "in_dtype", dict(dtype=2)), (uns, "MAX_COLS", dict(cols=40000)),
            (inv, "non-NULL", dict(dy=None)), (inv, "non-NULL", dict(rstd=None)),
            (inv, "aligned", dict(dw=6 * BASE + 2)), (inv, "overlaps", dict(dx=BASE + 4)),
            (inv, "workspace", dict(ws=None)), (inv, "16-byte", dict(ws=7 * BASE + 8)),
            (inv, str(need), dict(size=need - 1))):
        assert _back(lib, **kw) == want, word
        assert word in nv.nvfp4_last_error(), nv.nvfp4_last_error()
    assert lib.nvfp4_add_rmsnorm_backward_workspace_size(4, 64, None) == inv


def test_gemm_bias_act_refusals(lib):
    inv, uns = nv.NVFP4_ERR_INVALID, nv.NVFP4_ERR_UNSUPPORTED
    op = nv._COperand(256, 256, 256, nv.NVFP4_ROW_SCALED, 448.0)

    def call(epi, k=64, od=nv.NVFP4_OUT_BF16, d=BASE, ws=1 << 12, size=1 << 20, m=4, n=4):
        return lib.nvfp4_gemm_bias_act(R(op), R(op), m, n, k, epi, d, od, ws, size, None)
    good = nv._CEpilogue(None, FP, 0, None, None)
    for want, word, args in (
            (inv, "epilogue", dict(epi=None)),
            (inv, "activation", dict(epi=R(nv._CEpilogue(None, FP, 4, None, None)))),
            (inv, "bias_dtype", dict(epi=R(nv._CEpilogue(BASE, 3, 0, None, None)))),
            (inv, "residual overlaps", dict(epi=R(nv._CEpilogue(None, FP, 0, BASE + 2, None)))),
            (inv, "z overlaps", dict(epi=R(nv._CEpilogue(None, FP, 0, None, BASE)))),
            (inv, "aligned", dict(epi=R(good), d=BASE + 1)),
            (inv, "aligned", dict(epi=R(nv._CEpilogue(BASE + 2, FP, 0, None, None)))),
            (uns, "multiple of 32", dict(epi=R(good), k=48)),
            (inv, "out_dtype", dict(epi=R(good), od=9)), (inv, "d is NULL", dict(epi=R(good), d=None)),
            (inv, "workspace", dict(epi=R(good), m=300, ws=None)),
            (inv, "workspace", dict(epi=R(good), m=300, size=16))):
        assert call(**args) == want, word
        assert word in nv.nvfp4_last_error(), nv.nvfp4_last_error()
    assert call(R(good), m=0) == nv.NVFP4_OK


def test_bias_act_backward_refusals(lib):
    inv = nv.NVFP4_ERR_INVALID

    def call(dd=BASE, z=2 * BASE, dtype=BF, act=1, rows=4, cols=64, dz=3 * BASE, db=4 * BASE,
             ws=7 * BASE, size=1 << 24):
        return lib.nvfp4_bias_act_backward(dd, z, dtype, act, rows, cols, dz, db, None, None, ws,
                                           size, None)
    need = nv.nvfp4_bias_act_backward_workspace_size(4, 64)
    for word, kw in (("dtype", dict(dtype=5)), ("activation", dict(act=9)),
                     ("rows and cols", dict(cols=-2)), ("non-NULL", dict(dz=None)),
                     ("z is NULL", dict(z=None)), ("overlaps", dict(dz=BASE + 2)),
                     ("aligned", dict(db=BASE + 1)), ("workspace", dict(ws=None)),
                     (str(need), dict(size=need - 1))):
        assert call(**kw) == inv, word
        assert word in nv.nvfp4_last_error(), nv.nvfp4_last_error()


def test_clip_refusals(lib):
    inv, uns = nv.NVFP4_ERR_INVALID, nv.NVFP4_ERR_UNSUPPORTED
    T = nv._CTensor

    def call(t, count=1, max_norm=1.0, norm=BASE, ws=2 * BASE, size=1 << 20):
        return lib.nvfp4_clip_grad_norm(t, count, max_norm, norm, ws, size, None)
    for want, word, args, kw in (
            (inv, "count", T(), dict(count=-1)), (uns, "tensors", T(), dict(count=1 << 20)),
            (inv, "max_norm", T(), dict(max_norm=-1.0)),
            (inv, "max_norm", T(), dict(max_norm=float("nan"))),
            (inv, "norm must", T(), dict(norm=None)), (inv, "dtype", T(16, 16, 1, 8), {}),
            (inv, "n out of range", T(16, 16, -1, BF), {}), (inv, "NULL", T(None, 16, 4, BF), {}),
            (inv, "NULL", T(16, None, 4, BF), {}), (inv, "aligned", T(18, 18, 4, FP), {}),
            (inv, "overlaps", T(BASE, BASE + 8, 64, FP), {}),
            (inv, "workspace", T(BASE, BASE, 4, FP), dict(ws=None)),
            (inv, "needed", T(BASE, BASE, 4, FP), dict(size=64))):
        assert call(R(args), **kw) == want, word
        assert word in nv.nvfp4_last_error(), (word, nv.nvfp4_last_error())
    assert lib.nvfp4_clip_grad_norm(None, 1, 1.0, BASE, 2 * BASE, 1 << 20, None) == inv


def test_binding_refusals(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="weight"):
        nv.nvfp4_add_rmsnorm(x, w[:32], 1e-5, y=x)
    with pytest.raises(ValueError, match="contiguous 2-D"):
        nv.nvfp4_add_rmsnorm(x[:, ::2], w, 1e-5, y=x)
    with pytest.raises(ValueError, match="residual"):
        nv.nvfp4_add_rmsnorm(x, w, 1e-5, residual=x.float(), y=x)
    with pytest.raises(TypeError):
        nv.nvfp4_add_rmsnorm(x.half(), w, 1e-5, y=x.half())
    with pytest.raises(ValueError, match="scale"):
        nv.nvfp4_add_rmsnorm(x, w, 1e-5, fp8=nv.Fp8Out(x.view(torch.uint8)[:, :64].contiguous(),
                                                       torch.zeros(3)))
    with pytest.raises(ValueError, match="cfg"):
        nv.nvfp4_add_rmsnorm(x, w, 1e-5, row=nv.Out(w, w, w))
    with pytest.raises(ValueError, match="row"):
        nv.nvfp4_add_rmsnorm(x, w, 1e-5, cfg=nv.Config(nv.NVFP4_ROW_SCALED, 448.0, 0, 0),
                             row=nv.Out(torch.zeros(4, 31, dtype=torch.uint8),
                                        torch.zeros(4, 4, dtype=torch.uint8), torch.zeros(4)))
    with pytest.raises(ValueError, match="dbias"):
        nv.nvfp4_bias_act_backward(x, x, 1, x, dbias=torch.zeros(4))
    with pytest.raises(ValueError, match="dy"):
        nv.nvfp4_add_rmsnorm_backward(x[:2], x, w, torch.zeros(4), x)
    with pytest.raises(ValueError, match="out"):
        nv.nvfp4_clip_grad_norm([w], 1.0, torch.zeros(1), out=[])
    with pytest.raises(ValueError, match="out must"):
        nv.nvfp4_clip_grad_norm([w], 1.0, torch.zeros(1), out=[w.float()])
    op = nv.Operand(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8),
                    torch.zeros(4), nv.NVFP4_ROW_SCALED, 448.0)
    with pytest.raises(ValueError, match="shapes"):
        nv.nvfp4_gemm_bias_act(op, op, torch.zeros(4, 5))
    with pytest.raises(ValueError, match="bias"):
        nv.nvfp4_gemm_bias_act(op, op, torch.zeros(4, 4), bias=torch.zeros(5))


def _on_host():
    """Each layer operator with arguments that are right but for where they lie."""
    x, w, f = torch.zeros(4, 64), torch.ones(64), torch.zeros(4)
    op = nv.Operand(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8),
                    f, nv.NVFP4_ROW_SCALED, 448.0)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    return {
        "norm": lambda: nv.nvfp4_add_rmsnorm(x, w, 1e-5, y=x),
        "norm codes": lambda: nv.nvfp4_add_rmsnorm(
            x, w, 1e-5, fp8=nv.Fp8Out(torch.zeros(4, 64, dtype=torch.uint8), f)),
        "norm rows": lambda: nv.nvfp4_add_rmsnorm(
            x, w, 1e-5, row=nv.Out(op.codes, op.scales, f),
            cfg=nv.Config(nv.NVFP4_ROW_SCALED, 448.0, 0, 0)),
        "norm backward": lambda: nv.nvfp4_add_rmsnorm_backward(x, x, w, f, x, dweight=w),
        "product": lambda: nv.nvfp4_gemm_bias_act(op, op, torch.zeros(4, 4), workspace=ws),
        "activation backward": lambda: nv.nvfp4_bias_act_backward(x, x, 1, x, dbias=w),
        "gradient norm": lambda: nv.nvfp4_grad_norm([w], torch.zeros(1), workspace=ws),
        "clipping": lambda: nv.nvfp4_clip_grad_norm([w], 1.0, torch.zeros(1), out=[w.clone()],
                                                    workspace=ws),
    }


@pytest.mark.parametrize("name", ["norm", "norm codes", "norm rows", "norm backward", "product",
                                  "activation backward", "gradient norm", "clipping"])
def test_host_tensors_are_refused(lib, name):
    """Their addresses would reach the kernels as device memory."""
    with pytest.raises(ValueError, match="on the GPU"):
        _on_host()[name]()


def test_operand_sizes_are_checked(lib):
    """The kernels read codes [lines][k/2], scales [lines][k/16] and an amax per line."""
    def op(codes=(8, 32), scales=(8, 4), amax=(8,), mode=nv.NVFP4_ROW_SCALED, dtype=torch.float32):
        return nv.Operand(torch.zeros(codes, dtype=torch.uint8),
                          torch.zeros(scales, dtype=torch.uint8), torch.zeros(amax, dtype=dtype),
                          mode, 448.0)
    good, d = op(), torch.zeros(8, 8)
    wide = op(codes=(8, 64))
    wide.codes = wide.codes[:, :32]  # rows further apart than the kernel steps
    for bad in (op(scales=(8, 3)), op(scales=(4, 4)), op(amax=(7,)), op(dtype=torch.float64),
                op(amax=(0,), mode=nv.NVFP4_PER_TENSOR), wide):
        for pair, name in (((bad, good), "a"), ((good, bad), "b")):
            with pytest.raises(ValueError, match=name):
                nv.nvfp4_gemm_bias_act(*pair, d)
    with pytest.raises(ValueError, match="on the GPU"):
        nv.nvfp4_gemm_bias_act(good, op(amax=(1,), mode=nv.NVFP4_PER_TENSOR), d)
