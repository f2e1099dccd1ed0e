"""The gated block's operators on matrices of more than 2^31 elements: rows whose offsets pass 32 bits
come out as the same rows do in a small call, and column sums take all rows.  Inputs are small
integers where sums run over rows or columns, so that FP32 sums are exact whatever their order.
"""
import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv
from test_gpu_gated import _integer_operands

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _room(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip("not enough memory")


def _integers(rows, cols, low, high, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(low, high + 1, (rows, cols), generator=g, device=DEV, dtype=torch.int8).bfloat16()


def _column_sums(f, rows, cols, step=4096):
    total = torch.zeros(cols, dtype=torch.float64, device=DEV)
    for r in range(0, rows, step):
        total += f(slice(r, min(rows, r + step))).sum(0)
    return total


def test_gated_product():
    _room(40)
    m, n, k, last = 90000, 12296, 64, 3000
    a, b = _integer_operands(m, n, k, 1)
    d = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    gu = torch.empty(m, 2 * n, dtype=torch.bfloat16, device=DEV)
    ra, ca = torch.empty(m, device=DEV), torch.empty(n, device=DEV)
    nv.nvfp4_gemm_gated(a, b, d, act=nv.NVFP4_ACT_RELU, gu=gu, row_amax=ra, col_amax=ca)
    end = nv.Operand(a.codes[-last:].contiguous(), a.scales[-last:].contiguous(), a.amax[-last:], a.mode, a.bound)
    e, gv = torch.empty(last, n, dtype=d.dtype, device=DEV), torch.empty(last, 2 * n, dtype=d.dtype, device=DEV)
    nv.nvfp4_gemm_gated(end, b, e, act=nv.NVFP4_ACT_RELU, gu=gv)
    assert torch.equal(d[-last:], e) and torch.equal(gu[-last:], gv)
    assert torch.equal(ra, d.abs().amax(dim=1).float()) and torch.equal(ca, d.abs().amax(dim=0).float())


def test_gated_backward():
    _room(60)
    rows, cols, last = 90000, 12296, 3000
    dd, gu = _integers(rows, cols, -2, 2, 2), _integers(rows, 2 * cols, -3, 3, 3)
    dgu, db = torch.empty_like(gu), torch.empty(2 * cols, device=DEV)
    ra, ca = torch.empty(rows, device=DEV), torch.empty(2 * cols, device=DEV)
    nv.nvfp4_gated_backward(dd, gu, nv.NVFP4_ACT_NONE, dgu, dbias=db, row_amax=ra, col_amax=ca)
    assert torch.equal(dgu[-last:, :cols], dd[-last:] * gu[-last:, cols:])
    assert torch.equal(dgu[-last:, cols:], dd[-last:] * gu[-last:, :cols])
    assert torch.equal(ra, dgu.abs().amax(dim=1).float()) and torch.equal(ca, dgu.abs().amax(dim=0).float())
    assert torch.equal(db.double(), _column_sums(lambda s: dgu[s].double(), rows, 2 * cols))


@pytest.mark.parametrize("cols", [8192, 8191])
def test_layernorm_and_its_backward(cols):
    _room(60)
    rows, last = 270000, 9000
    x, r = _integers(rows, cols, -3, 3, 4), _integers(rows, cols, -2, 2, 5)
    w, b = torch.ones(cols, device=DEV), torch.zeros(cols, device=DEV)
    h, y = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    nv.nvfp4_add_layernorm(x, w, 1e-5, bias=b, residual=r, h=h, y=y, mean=mean, rstd=rstd)
    ends = [torch.empty_like(t[-last:]) for t in (h, y, mean, rstd)]
    xe, re = x[-last:].clone(), r[-last:].clone()  # (their starts are aligned as the whole tensors' are)
    nv.nvfp4_add_layernorm(xe, w, 1e-5, bias=b, residual=re, h=ends[0], y=ends[1], mean=ends[2], rstd=ends[3])
    for got, want in zip((h, y, mean, rstd), ends):
        assert torch.equal(got[-last:], want)
    del y
    # sums over 270000 rows of |dy| <= 2 times |h| <= 5: below 2^24
    mean.zero_()
    rstd.fill_(1.0)
    dw, db, dx = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV), torch.empty_like(x)
    nv.nvfp4_add_layernorm_backward(r, h, w, mean, rstd, dx, dweight=dw, dbias=db)
    dxe = torch.empty_like(xe)
    nv.nvfp4_add_layernorm_backward(re, ends[0], w, mean[:last], rstd[:last], dxe)
    assert torch.equal(dx[-last:], dxe)
    assert torch.equal(dw.double(), _column_sums(lambda s: r[s].double() * h[s].double(), rows, cols))
    assert torch.equal(db.double(), _column_sums(lambda s: r[s].double(), rows, cols))
