"""Refusals of the gated block's operators: argument checks that run before any CUDA call (no
GPU needed), and the binding's own checks."""
import ctypes

import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv

R = ctypes.byref
BF, FP = nv.NVFP4_IN_BF16, nv.NVFP4_IN_FP32
BASE = 1 << 20
INV, UNS = nv.NVFP4_ERR_INVALID, nv.NVFP4_ERR_UNSUPPORTED
GOOD = nv._CMask(0.1, 1, 2, None)


@pytest.fixture(scope="module")
def lib():
    from nvfp4_precision_quantization_gb300 import build
    build.build()
    return nv.load_library()


def _refused(call, cases):
    for want, word, kw in cases:
        assert call(**kw) == want, (word, nv.nvfp4_last_error())
        assert word in nv.nvfp4_last_error(), (word, nv.nvfp4_last_error())


BAD_MASKS = [(INV, "mask->p", dict(mask=R(nv._CMask(p, 1, 2, None))))
             for p in (-0.1, 1.5, float("nan"))] + \
            [(INV, "offset_add", dict(mask=R(nv._CMask(0.1, 1, 2, BASE + 4))))]


def test_layernorm_refusals(lib):
    row = nv._COut(5 * BASE, 6 * BASE, 7 * BASE, None)
    rs = nv.Config(nv.NVFP4_ROW_SCALED, 448.0, 0, 0)

    def call(x=BASE, residual=None, dtype=BF, mask=None, weight=2 * BASE, bias=None, wdtype=BF,
             rows=4, cols=64, eps=1e-5, h=None, y=3 * BASE, mean=None, rstd=None, fp8=None,
             cfg=None, row=None):
        return lib.nvfp4_add_layernorm(x, residual, dtype, mask, weight, bias, wdtype, rows, cols,
                                       eps, h, y, mean, rstd, fp8, cfg, row, None)
    _refused(call, BAD_MASKS + [
        (INV, "in_dtype", dict(dtype=7)), (INV, "weight_dtype", dict(wdtype=-1)),
        (INV, "rows and cols", dict(rows=-1)), (UNS, "MAX_COLS", dict(cols=32769)),
        (INV, "weight is NULL", dict(weight=None)), (INV, "x is NULL", dict(x=None)),
        (INV, "eps", dict(eps=-1.0)), (INV, "eps", dict(eps=float("nan"))),
        (INV, "residual", dict(h=4 * BASE)), (INV, "no output", dict(y=None)),
        (INV, "aligned", dict(x=BASE + 1)), (INV, "aligned", dict(bias=BASE + 1)),
        (INV, "aligned", dict(mean=BASE + 2)),
        (INV, "h overlaps y", dict(mask=R(GOOD), h=3 * BASE)),
        (INV, "without being it", dict(y=BASE + 2)),
        (UNS, "one call", dict(fp8=R(nv._CFp8Out(BASE, BASE, 0)), row=R(row), cfg=R(rs))),
        (INV, "cfg is NULL", dict(row=R(row))),
        (UNS, "16x16", dict(row=R(row), cfg=R(nv.Config(nv.NVFP4_PER_TENSOR, 448.0, 0, 1)))),
        (UNS, "amax_in", dict(row=R(row), cfg=R(nv.Config(nv.NVFP4_PER_TENSOR, 448.0, 0, 0))))])
    assert call(rows=0) == nv.NVFP4_OK


def test_layernorm_backward_refusals(lib):
    need = nv.nvfp4_add_layernorm_backward_workspace_size(4, 64)
    assert need == 2 * 4 * 4 * 64

    def call(dy=BASE, h=2 * BASE, dh=None, dtype=BF, mask=None, w=3 * BASE, wdtype=BF,
             mean=4 * BASE, rstd=5 * BASE, rows=4, cols=64, dx=6 * BASE, dr=None, dw=7 * BASE,
             db=8 * BASE, ws=9 * BASE, size=1 << 20):
        return lib.nvfp4_add_layernorm_backward(dy, h, dh, dtype, mask, w, wdtype, mean, rstd,
                                                rows, cols, dx, dr, dw, db, ws, size, None)
    _refused(call, BAD_MASKS + [
        (INV, "in_dtype", dict(dtype=2)), (UNS, "MAX_COLS", dict(cols=40000)),
        (INV, "non-NULL", dict(dy=None)), (INV, "non-NULL", dict(mean=None)),
        (INV, "aligned", dict(db=6 * BASE + 2)), (INV, "overlaps", dict(dx=BASE + 4)),
        (INV, "dresidual", dict(dr=10 * BASE)),
        (INV, "dx overlaps dresidual", dict(mask=R(GOOD), dr=6 * BASE)),
        (INV, "overlaps", dict(mask=R(GOOD), dr=2 * BASE + 8)),
        (INV, "workspace", dict(ws=None)), (INV, "16-byte", dict(ws=7 * BASE + 8)),
        (INV, str(need), dict(dw=None, size=need - 1))])
    assert lib.nvfp4_add_layernorm_backward_workspace_size(4, 64, None) == INV


def test_dropout_refusals(lib):
    def call(x=BASE, residual=None, dtype=BF, n=64, mask=R(GOOD), y=2 * BASE):
        return lib.nvfp4_dropout(x, residual, dtype, n, mask, y, None)
    _refused(call, BAD_MASKS + [
        (INV, "dtype", dict(dtype=3)), (INV, "n must", dict(n=-1)), (INV, "n must", dict(n=1 << 48)),
        (INV, "mask is NULL", dict(mask=None)), (INV, "non-NULL", dict(x=None)),
        (INV, "non-NULL", dict(y=None)), (INV, "aligned", dict(dtype=FP, x=BASE + 2)),
        (INV, "overlaps", dict(y=BASE + 2)), (INV, "overlaps", dict(residual=2 * BASE + 16))])


def test_gated_product_refusals(lib):
    op = nv._COperand(256, 256, 256, nv.NVFP4_ROW_SCALED, 448.0)

    def call(epi=R(nv._CGatedEpilogue(None, FP, 0, None, None, None)), k=64,
             od=nv.NVFP4_OUT_BF16, d=BASE, ws=1 << 12, size=1 << 30, m=4, n=4, a=R(op)):
        return lib.nvfp4_gemm_gated(a, R(op), m, n, k, epi, d, od, ws, size, None)

    def epi(bias=None, bd=FP, act=0, gu=None, ra=None, ca=None):
        return R(nv._CGatedEpilogue(bias, bd, act, gu, ra, ca))
    _refused(call, [
        (INV, "epilogue", dict(epi=None)), (INV, "activation", dict(epi=epi(act=4))),
        (INV, "bias_dtype", dict(epi=epi(bias=BASE, bd=3))),
        (INV, "gu overlaps", dict(epi=epi(gu=BASE + 2))), (INV, "aligned", dict(d=BASE + 1)),
        (INV, "aligned", dict(epi=epi(bias=BASE + 2))), (INV, "aligned", dict(epi=epi(ra=BASE + 2))),
        (INV, "aligned", dict(epi=epi(ca=BASE + 1))), (INV, "2^31", dict(n=1 << 30)),
        (INV, "rows and cols", dict(m=-1)), (UNS, "multiple of 32", dict(k=48)),
        (INV, "out_dtype", dict(od=9)), (INV, "d is NULL", dict(d=None)),
        (INV, "a or b", dict(a=None)), (INV, "workspace", dict(m=300, ws=None)),
        (INV, "workspace", dict(m=300, ws=(1 << 12) + 16)), (INV, "workspace", dict(m=300, size=16)),
        (INV, "workspace", dict(m=5000, n=5000, size=16))])
    assert call(m=0) == nv.NVFP4_OK
    assert lib.nvfp4_gemm_gated_workspace_size(4, 4, 64, None) == INV


def test_small_workspaces_name_their_size(lib):
    """The refusal states the bytes that are needed, as the call's own size function gives them."""
    m, n, k = 300, 512, 4096
    op = R(nv._COperand(256, 256, 256, nv.NVFP4_ROW_SCALED, 448.0))
    epi = R(nv._CEpilogue(None, FP, 0, None, None))
    gated = R(nv._CGatedEpilogue(None, FP, 0, None, None, None))
    for name, need, call in (
            ("nvfp4_gemm_workspace_size", nv.nvfp4_gemm_workspace_size(m, n, k),
             lambda size: lib.nvfp4_gemm(op, op, m, n, k, BASE, 0, 1 << 12, size, None)),
            ("nvfp4_grouped_gemm_workspace_size", nv.nvfp4_grouped_gemm_workspace_size(m, n, k, 2),
             lambda size: lib.nvfp4_grouped_gemm(op, op, BASE, 2, m, n, k, BASE, 0, 1 << 12, size, None)),
            ("nvfp4_gemm_bias_act_workspace_size", nv.nvfp4_gemm_bias_act_workspace_size(m, n, k),
             lambda size: lib.nvfp4_gemm_bias_act(op, op, m, n, k, epi, BASE, 0, 1 << 12, size, None)),
            ("nvfp4_gemm_gated_workspace_size", nv.nvfp4_gemm_gated_workspace_size(m, n, k),
             lambda size: lib.nvfp4_gemm_gated(op, op, m, n, k, gated, BASE, 0, 1 << 12, size, None))):
        assert call(need - 1) == INV
        said = nv.nvfp4_last_error()
        assert f"{need} needed ({name})" in said and str(need - 1) in said, said


def test_gated_backward_refusals(lib):
    def call(dd=BASE, gu=2 * BASE, dtype=BF, act=1, rows=4, cols=64, dgu=3 * BASE, db=4 * BASE,
             ws=7 * BASE, size=1 << 24):
        return lib.nvfp4_gated_backward(dd, gu, dtype, act, rows, cols, dgu, db, None, None, ws,
                                        size, None)
    need = nv.nvfp4_gated_backward_workspace_size(4, 64)
    _refused(call, [
        (INV, "dtype", dict(dtype=5)), (INV, "activation", dict(act=9)),
        (INV, "rows and cols", dict(cols=-2)), (INV, "2^31", dict(rows=0, cols=1 << 30)),
        (INV, "non-NULL", dict(dgu=None)), (INV, "non-NULL", dict(gu=None)),
        (INV, "overlaps dd", dict(dgu=BASE)), (INV, "without being it", dict(dgu=2 * BASE + 4)),
        (INV, "aligned", dict(db=BASE + 1)), (INV, "workspace", dict(ws=None)),
        (INV, str(need), dict(size=need - 1))])


def test_binding_refusals(lib):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    s, mask = torch.zeros(4), nv.Mask(0.1, 1, 2)
    op = nv.Operand(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 4, dtype=torch.uint8),
                    torch.zeros(8), nv.NVFP4_ROW_SCALED, 448.0)
    a = nv.Operand(op.codes[:4], op.scales[:4], op.amax[:4], nv.NVFP4_ROW_SCALED, 448.0)
    d = torch.zeros(4, 4)
    for word, f in (
            ("on the GPU", lambda: nv.nvfp4_add_layernorm(x, w, 1e-5, y=x)),
            ("weight", lambda: nv.nvfp4_add_layernorm(x, w[:3], 1e-5, y=x)),
            ("bias must have", lambda: nv.nvfp4_add_layernorm(x, w, 1e-5, bias=w.float(), y=x)),
            ("mean", lambda: nv.nvfp4_add_layernorm(x, w, 1e-5, y=x, mean=s[:2])),
            ("offset_add", lambda: nv.nvfp4_dropout(x, nv.Mask(0.1, 1, 2, offset_add=s), x)),
            ("on the GPU", lambda: nv.nvfp4_dropout(x, mask, x)),
            ("residual", lambda: nv.nvfp4_dropout(x, mask, x, residual=x.float())),
            ("contiguous", lambda: nv.nvfp4_dropout(x.t(), mask, x)),
            ("dresidual", lambda: nv.nvfp4_add_layernorm_backward(x, x, w, s, s, x, mask=mask,
                                                                  dresidual=s)),
            ("on the GPU", lambda: nv.nvfp4_add_layernorm_backward(x, x, w, s, s, x)),
            ("twice", lambda: nv.nvfp4_gemm_gated(a, a, d)),
            ("bias", lambda: nv.nvfp4_gemm_gated(a, op, d, bias=torch.zeros(4))),
            ("gu", lambda: nv.nvfp4_gemm_gated(a, op, d, gu=d)),
            ("col_amax", lambda: nv.nvfp4_gemm_gated(a, op, d, col_amax=torch.zeros(8))),
            ("on the GPU", lambda: nv.nvfp4_gemm_gated(a, op, d)),
            ("gu", lambda: nv.nvfp4_gated_backward(d, d, 0, d)),
            ("on the GPU", lambda: nv.nvfp4_gated_backward(d, torch.zeros(4, 8), 0,
                                                           torch.zeros(4, 8)))):
        with pytest.raises(ValueError, match=word):
            f()
