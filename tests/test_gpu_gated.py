"""The gated product of NVFP4 operands, and the backward pass of its activation and product, on
the GPU against the FP64 definitions.

Tolerances.  The halves: as in test_gpu_bias_act, t = (k 2^-23 + 2^-20) sum|terms| each, and 2^-23
of |z| for the bias.  d = act(g) u: 1.13 t_g |u| + t_u |act(g)| + 1.13 t_g t_u, the activation's own
2^-20 (1 + |g|) |u|, and 2^-23 |d| for the product.  Storing rounds once.  The maxima are exactly
those of d (of dgu) as the call stored it.
"""
import os
import subprocess
import sys

import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv
import workloads
from block_reference import gated_backward, operand_values
from layer_reference import ACTS, act, at_offset, guarded, half_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda"
RS, PT = nv.NVFP4_ROW_SCALED, nv.NVFP4_PER_TENSOR
DTYPES = [torch.bfloat16, torch.float32]


def _operands(m, n, k, seed, modes=(RS, RS), bounds=(448.0, 448.0), scale_offset=0):
    """Two operands, their FP64 product [m][2n] and the sums of its terms' magnitudes; the values
    are scaled so that the product stays within about 4."""
    dev = []
    for i, lines in enumerate((m, 2 * n)):
        c, s, a = workloads.nvfp4_operand(lines, k, seed + i, modes[i] == RS)
        dev.append(nv.Operand(c.to(DEV), at_offset(s.to(DEV), scale_offset),
                              (a * (0.1 / a.max())).to(DEV), modes[i], bounds[i]))

    def product():
        x, w = (operand_values(o.codes, o.scales, o.amax, o.bound) for o in dev)
        return x @ w.t(), x.abs() @ w.abs().t()
    z, _ = product()
    dev[1].amax = (dev[1].amax * (4.0 / z.abs().max().clamp(min=1e-6))).float()
    return (dev, *product())


def _check(m, n, k, dtype, name, bias=None, keep=True, maxima=True, seed=0, modes=(RS, RS),
           bounds=(448.0, 448.0), offset=0, scale_offset=0):
    (a, b), z, mag = _operands(m, n, k, seed, modes, bounds, scale_offset)
    tol = (k * 2.0 ** -23 + 2.0 ** -20) * mag
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    bv = torch.randn(2 * n, generator=g, device=DEV).to(bias) if bias is not None else None
    if bv is not None:
        z = z + bv.double()
        tol = tol + 2.0 ** -23 * z.abs()
    d, ok_d = guarded((m, n), dtype, offset=offset)
    gu, ok_gu = guarded((m, 2 * n), dtype, offset=offset)
    ra, ok_r = guarded((m,), torch.float32)
    ca, ok_c = guarded((n,), torch.float32)
    nv.nvfp4_gemm_gated(a, b, d, bias=bv, act=ACTS[name], gu=gu if keep else None,
                        row_amax=ra if maxima else None, col_amax=ca if maxima else None)
    torch.cuda.synchronize()
    zg, zu, tg, tu = z[:, :n], z[:, n:], tol[:, :n], tol[:, n:]
    want, half = act(zg, name) * zu, half_ulp(dtype)
    t = 1.13 * tg * zu.abs() + tu * act(zg, name).abs() + 1.13 * tg * tu + 2.0 ** -23 * want.abs()
    if name in ("gelu", "silu"):
        t = t + 2.0 ** -20 * (1 + zg.abs()) * (zu.abs() + tu)
    assert bool(((d.double() - want).abs() <= t * (1 + half) + half * want.abs()).all())
    if keep:
        assert bool(((gu.double() - z).abs() <= tol * (1 + half) + half * z.abs()).all())
    if maxima:
        assert torch.equal(ra, d.abs().amax(dim=1).float())
        assert torch.equal(ca, d.abs().amax(dim=0).float())
    for ok in (ok_d, ok_gu, ok_r, ok_c):
        ok()
    return d


# one token to several tiles, odd sizes on both axes, K tails of a K tile
SIZES = [(1, 256, 256), (1, 1, 32), (1, 4097, 512), (2, 100, 96), (7, 300, 320), (8, 512, 1024),
         (16, 1000, 544), (17, 129, 64), (31, 64, 800), (33, 640, 256), (64, 255, 288),
         (65, 384, 512), (100, 77, 96), (128, 256, 128), (129, 257, 160), (200, 520, 992),
         (300, 500, 320), (257, 128, 256), (385, 6000, 64), (450, 5000, 96), (1000, 2561, 160),
         (700, 1300, 2080)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_product(m, n, k, dtype):
    name = list(ACTS)[(m + n + k // 32) % 4]
    _check(m, n, k, dtype, name, torch.float32, seed=m + n + k)
    _check(m, n, k, dtype, "silu", None, False, False, m + n + k + 1, (PT, RS), (256.0, 448.0))


# what goes to the pairs of SMs: long sums of more than 64 rows, at the borders of their tiles (256
# rows, 128 columns, 256 values) and below them; and many tiles, whose rows need not be aligned
@pytest.mark.parametrize("m,n,k", [(65, 8, 1056), (100, 136, 1120), (129, 128, 4096), (256, 128, 1280),
                                   (257, 264, 2080), (300, 1000, 1312), (513, 72, 1056),
                                   (2500, 2561, 96), (5200, 1001, 64), (2600, 2500, 288)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_pairs_of_sms(m, n, k, dtype):
    name = list(ACTS)[(m + n + k // 32) % 4]
    _check(m, n, k, dtype, name, torch.float32, seed=m + n)
    _check(m, n, k, dtype, "silu", None, False, False, m + n + 1, (RS, PT), (448.0, 256.0))
    if m < 600:
        _check(m, n, k, dtype, "gelu", torch.bfloat16, False, True, m + 2, (PT, PT), scale_offset=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_many_tiles_of_unaligned_rows(offset, dtype):
    _check(2600, 2512, 96, dtype, "silu", torch.float32, seed=3, offset=offset, scale_offset=1)


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("bias", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("keep,maxima", [(False, True), (True, False)])
@pytest.mark.parametrize("m,n", [(1, 272), (5, 272), (40, 272), (150, 272), (700, 6000)])
def test_epilogue_combinations(m, n, name, bias, keep, maxima):
    _check(m, n, 160, torch.bfloat16, name, bias, keep, maxima, 3 * m)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n", [(1, 264), (9, 264), (140, 264), (640, 5000)])
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_unaligned_outputs_and_scales(m, n, offset, dtype):
    _check(m, n, 128, dtype, "silu", torch.float32, seed=m, offset=offset, scale_offset=offset)


@pytest.mark.parametrize("m,n", [(1, 5000), (40, 20000), (1, 40000), (129, 10100)])
def test_tiles_cut_along_k(m, n):
    """More tiles than SMs with a rest that is cut along K, beside whole tiles."""
    _check(m, n, 2080, torch.bfloat16, "gelu", torch.float32, seed=m)


@pytest.mark.parametrize("m,n", [(1, 320), (20, 320), (130, 320), (450, 5000)])
def test_long_k(m, n):
    _check(m, n, 8192 + 96, torch.float32, "none", torch.float32, seed=5)


def _integer_operands(m, n, k, seed):
    """Row-scaled operands whose values are E2M1 values times 1 or 2: every product is a multiple of 1/4 of
    at most 144."""
    dev = []
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    for lines in (m, 2 * n):
        codes = torch.randint(0, 256, (lines, k // 2), generator=g, device=DEV).to(torch.uint8)
        twice = torch.randint(0, 2, (lines, k // 16), generator=g, device=DEV)
        scales = torch.where(twice == 1, 0x40, 0x38).to(torch.uint8)  # E4M3 2 and 1
        dev.append(nv.Operand(codes, scales, torch.full((lines,), 448.0 * 6, device=DEV), RS, 448.0))
    return dev


@pytest.mark.parametrize("m,n,k", [(1, 320, 8288), (20, 320, 8288), (64, 257, 8288), (130, 320, 8288),
                                   (450, 1000, 8288), (300, 1001, 4128), (700, 2000, 2080),
                                   (1, 5000, 8192), (3, 20000, 2080), (257, 264, 16416)])
@pytest.mark.parametrize("keep", [False, True])
def test_long_sums_are_exact(m, n, k, keep):
    """Sums of products that are multiples of 1/4 are exact in FP32 while they stay below 2^22 (the largest
    possible sum of 16416 terms is 2.4 million), and alpha and beta are 1 (448 * 6 times its rounded
    reciprocal rounds to 1): a lost or doubled value, scale or block of a sum shows.  d = g u rounds once."""
    f = torch.tensor(448.0 * 6)
    assert float(f * (1.0 / f)) == 1.0
    a, b = _integer_operands(m, n, k, m + n)
    d = torch.empty(m, n, device=DEV)
    gu = torch.empty(m, 2 * n, device=DEV) if keep else None
    nv.nvfp4_gemm_gated(a, b, d, act=nv.NVFP4_ACT_NONE, gu=gu)
    z = operand_values(a.codes, a.scales, a.amax, 448.0) @ operand_values(b.codes, b.scales, b.amax,
                                                                          448.0).t()
    z = (4.0 * z).round() / 4.0  # operand_values' FP64 factor amax / (bound * 6) is 1 or next to it
    assert torch.equal(d, (z[:, :n] * z[:, n:]).float())
    if keep:
        assert torch.equal(gu.double(), z)


@pytest.mark.parametrize("m,n", [(3, 384), (150, 384), (900, 5000), (2600, 2501)])
def test_halves_are_the_product_with_either_weight(m, n):
    """gu is nvfp4_gemm with the stacked weights, within both sums' rounding, and repeatable."""
    (a, b), _, mag = _operands(m, n, 2048, 6)
    both, gu = (torch.empty(m, 2 * n, device=DEV) for _ in range(2))
    d, e = torch.empty(m, n, device=DEV), torch.empty(m, n, device=DEV)
    ra, rb = torch.empty(m, device=DEV), torch.empty(m, device=DEV)
    nv.nvfp4_gemm(a, b, both)
    nv.nvfp4_gemm_gated(a, b, d, gu=gu, row_amax=ra)
    assert bool(((both.double() - gu.double()).abs() <= 2 * 2048 * 2.0 ** -23 * mag).all())
    for _ in range(3):
        nv.nvfp4_gemm_gated(a, b, e, row_amax=rb)
        assert torch.equal(d, e) and torch.equal(ra, rb)


def test_maxima_are_the_quantizes_own():
    """Given to the quantization of d, they change no byte."""
    (a, b), _, _ = _operands(160, 512, 512, 2)
    d = torch.empty(160, 512, dtype=torch.bfloat16, device=DEV)
    ra, ca = torch.empty(160, device=DEV), torch.empty(512, device=DEV)
    nv.nvfp4_gemm_gated(a, b, d, row_amax=ra, col_amax=ca)
    cfg = nv.Config(RS, 448.0, 0, 0)
    outs = []
    for given in (False, True):
        row, col = nv.alloc_out(160, 512, 160), nv.alloc_out(512, 160, 512)
        if given:
            row.amax_in, col.amax_in = ra, ca
        nv.nvfp4_quantize_both(d, cfg, row, col)
        outs.append((row, col))
    torch.cuda.synchronize()
    for one, two in zip(*outs):
        for f in ("codes", "scales", "amax"):
            assert torch.equal(getattr(one, f), getattr(two, f))


def test_a_bad_line_stays_in_its_row_and_column():
    """An infinite amax spoils its own line's products alone; maxima skip the NaN it makes."""
    (a, b), _, _ = _operands(20, 200, 256, 8)
    d, e = torch.empty(20, 200, device=DEV), torch.empty(20, 200, device=DEV)
    ca = torch.empty(200, device=DEV)
    nv.nvfp4_gemm_gated(a, b, d)
    b.amax[7] = float("nan")  # column 7's gate
    nv.nvfp4_gemm_gated(a, b, e, col_amax=ca)
    assert bool(e[:, 7].isnan().all()) and float(ca[7]) == 0.0
    keep = torch.arange(200, device=DEV) != 7
    assert torch.equal(d[:, keep], e[:, keep])
    assert torch.equal(ca[keep], e[:, keep].abs().amax(dim=0))


def test_empty_sum_and_empty_outputs():
    bias = torch.randn(80, device=DEV)
    empty = lambda lines: nv.Operand(torch.empty(lines, 0, dtype=torch.uint8, device=DEV),  # noqa: E731
                                     torch.empty(lines, 0, dtype=torch.uint8, device=DEV),
                                     torch.ones(lines, device=DEV), RS, 448.0)
    d, gu = torch.empty(3, 40, device=DEV), torch.empty(3, 80, device=DEV)
    ra, ca = torch.full((3,), 9.0, device=DEV), torch.full((40,), 9.0, device=DEV)
    nv.nvfp4_gemm_gated(empty(3), empty(80), d, bias=bias, act=nv.NVFP4_ACT_RELU, gu=gu,
                        row_amax=ra, col_amax=ca)
    want = bias[:40].clamp(min=0) * bias[40:]
    assert torch.equal(gu, bias.expand(3, 80)) and torch.equal(d, want.expand(3, 40))
    assert torch.equal(ca, want.abs()) and torch.equal(ra, want.abs().amax().expand(3))
    (a, b), _, _ = _operands(4, 40, 64, 1)
    none = nv.Operand(a.codes[:0], a.scales[:0], a.amax[:0], RS, 448.0)
    ca.fill_(5.0)
    nv.nvfp4_gemm_gated(none, b, torch.empty(0, 40, device=DEV), col_amax=ca)
    assert float(ca.abs().max()) == 0.0
    nothing = nv.Operand(b.codes[:0], b.scales[:0], b.amax[:0], RS, 448.0)
    ra = torch.full((4,), 5.0, device=DEV)
    nv.nvfp4_gemm_gated(a, nothing, torch.empty(4, 0, device=DEV), row_amax=ra)
    assert float(ra.abs().max()) == 0.0


def test_empty_sum_of_the_most_rows():
    """A row count whose last step past the end leaves 32 bits: the rows' maxima are cleared and
    raised, and nothing in front of them or behind them is touched."""
    m, pad = (1 << 31) - 8192, 1 << 16
    bias = torch.tensor([1.5, -2.0], device=DEV)
    none = torch.empty(m, 0, dtype=torch.uint8, device=DEV)
    a = nv.Operand(none, none, torch.ones(1, device=DEV), PT, 448.0)
    b = nv.Operand(none[:2], none[:2], torch.ones(1, device=DEV), PT, 448.0)
    buf = torch.full((m + 2 * pad,), 9.0, device=DEV)
    d = torch.empty(m, 1, dtype=torch.bfloat16, device=DEV)
    nv.nvfp4_gemm_gated(a, b, d, bias=bias, act=nv.NVFP4_ACT_RELU, row_amax=buf[pad:pad + m])
    torch.cuda.synchronize()
    assert bool((buf[:pad] == 9.0).all()) and bool((buf[pad + m:] == 9.0).all())
    assert bool((buf[pad:pad + m] == 3.0).all()) and bool((d == -3.0).all())


@pytest.mark.parametrize("m,n", [(2, 512), (140, 512), (1500, 3000)])
def test_workspace_stream_and_graph(m, n):
    """A given workspace of the stated size, on another stream, and captured."""
    (a, b), _, _ = _operands(m, n, 1024, 9)
    d, e = (torch.empty(m, n, device=DEV) for _ in range(2))
    ra, rb, cb = torch.empty(m, device=DEV), torch.empty(m, device=DEV), torch.empty(n, device=DEV)
    nv.nvfp4_gemm_gated(a, b, d, row_amax=ra)
    ws, ok = guarded((max(nv.nvfp4_gemm_gated_workspace_size(m, n, 1024), 256),), torch.uint8)
    ws.random_(0, 256)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(2):  # what one call leaves in the workspace does not matter to the next
        e.zero_()
        torch.cuda.synchronize()
        nv.nvfp4_gemm_gated(a, b, e, row_amax=rb, col_amax=cb, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(d, e) and torch.equal(ra, rb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        nv.nvfp4_gemm_gated(a, b, e, row_amax=rb, col_amax=cb, workspace=ws)
    for _ in range(3):
        e.zero_()
        rb.fill_(1e9)
        cb.fill_(1e9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, e) and torch.equal(ra, rb)
        assert torch.equal(cb, e.abs().amax(dim=0))
    ok()


def test_two_calls_at_once():
    """Calls on two streams with a workspace each, many rows and few, again and again."""
    cases = [(1500, 3000, 1056), (7, 9000, 2048)]
    ops = [_operands(m, n, k, 11)[0] for m, n, k in cases]
    want = [torch.empty(m, n, device=DEV) for m, n, _ in cases]
    for (a, b), d in zip(ops, want):
        nv.nvfp4_gemm_gated(a, b, d)
    got = [torch.empty_like(d) for d in want for _ in range(2)]
    maxima = [torch.empty(d.shape[0], device=DEV) for d in got]
    ws = [torch.empty(nv.nvfp4_gemm_gated_workspace_size(*cases[i // 2]), dtype=torch.uint8, device=DEV)
          for i in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(4):
            a, b = ops[i // 2]
            nv.nvfp4_gemm_gated(a, b, got[i], row_amax=maxima[i], workspace=ws[i], stream=streams[i % 2])
    torch.cuda.synchronize()
    for i in range(4):
        assert torch.equal(got[i], want[i // 2])
        assert torch.equal(maxima[i], got[i].abs().amax(dim=1))
    assert nv.nvfp4_device_status() == 0


FIRST_CALLS = """
import threading, torch, test_gpu_gated as t
nv = t.nv
m, sizes = 300, [(640, 1056), (1001, 1056)]  # aligned rows of d, and not
ops = [t._operands(m, n, k, 4)[0] for n, k in sizes]
got = [torch.empty(m, sizes[i % 2][0], device="cuda") for i in range(8)]
ws = [torch.empty(nv.nvfp4_gemm_gated_workspace_size(m, *sizes[i % 2]), dtype=torch.uint8, device="cuda")
      for i in range(8)]
streams = [torch.cuda.Stream() for _ in range(8)]
torch.cuda.synchronize()
start, errors = threading.Barrier(8), []
def call(i):
    try:
        torch.cuda.set_device(0)
        start.wait()
        nv.nvfp4_gemm_gated(*ops[i % 2], got[i], workspace=ws[i], stream=streams[i])
    except Exception as e:
        errors.append(e)
threads = [threading.Thread(target=call, args=(i,)) for i in range(8)]
[x.start() for x in threads]
[x.join() for x in threads]
torch.cuda.synchronize()
assert not errors, errors
for i, d in enumerate(got):
    want = torch.empty_like(d)
    nv.nvfp4_gemm_gated(*ops[i % 2], want)
    assert torch.equal(d, want)
print("same")
"""


def test_first_calls_of_several_threads():
    """Eight threads make a process's first gated products at once."""
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": path}, cwd=os.path.dirname(here))
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


# ---------------------------------------------------------------- backward

BACK = [(1, 1), (1, 4096), (3, 16), (5, 17), (40, 64), (1000, 8), (129, 100), (300, 512),
        (77, 513), (64, 5000), (2000, 1024), (5, 28672), (700, 2056), (0, 8), (8, 0),
        (3000, 1001), (999, 515), (1200, 2050)]


def _back_inputs(rows, cols, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    gu = (3 * torch.randn(rows, 2 * cols, generator=g, device=DEV)).to(dtype)
    return torch.randn(rows, cols, generator=g, device=DEV).to(dtype), gu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", BACK)
def test_backward(rows, cols, dtype):
    """dg, du: act and act' are within 2^-20 (1 + |g|) of values below 1.13 (1 + |g|), two more
    products 2^-23; dbias: sums of `rows` terms, at most rows / CTAs + 80 additions a chain."""
    dd, gu = _back_inputs(rows, cols, dtype, rows + cols)
    names = list(ACTS) if rows < 700 else [list(ACTS)[(rows + cols) % 4]]
    half = half_ulp(dtype)
    for name in names:
        dgu, ok_d = guarded((rows, 2 * cols), dtype)
        db, ok_b = guarded((2 * cols,), torch.float32)
        ra, ok_r = guarded((rows,), torch.float32)
        ca, ok_c = guarded((2 * cols,), torch.float32)
        nv.nvfp4_gated_backward(dd, gu, ACTS[name], dgu, dbias=db, row_amax=ra, col_amax=ca)
        torch.cuda.synchronize()
        want = gated_backward(dd, gu, name)
        g, u = gu[:, :cols].double().abs(), gu[:, cols:].double().abs()
        own = 2.0 ** -20 * (1 + g) * dd.double().abs()
        tol = torch.cat([own * u, own], dim=1) + 2.0 ** -22 * want.abs()
        assert bool(((dgu.double() - want).abs() <= tol * (1 + half) + half * want.abs() + 1e-37).all())
        tol_b = tol.sum(0) + (rows + 100) * 2.0 ** -24 * want.abs().sum(0)
        assert bool(((db.double() - want.sum(0)).abs() <= tol_b + 1e-37).all())
        if rows and cols:
            assert torch.equal(ra, dgu.abs().amax(dim=1).float())
            assert torch.equal(ca, dgu.abs().amax(dim=0).float())
        else:
            assert not bool(ra.any()) and not bool(ca.any()) and not bool(db.any())
        for ok in (ok_d, ok_b, ok_r, ok_c):
            ok()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_backward_unaligned_and_alone(dtype, offset):
    """Any start gives the same bits, and so does a call without sums and maxima, in place."""
    dd, gu = _back_inputs(70, 1008, dtype, 3)
    want, dgu = torch.empty_like(gu), torch.empty_like(gu)
    nv.nvfp4_gated_backward(dd, gu, nv.NVFP4_ACT_GELU, want, dbias=torch.empty(2016, device=DEV))
    got, ok = guarded((70, 2016), dtype, offset=offset)
    nv.nvfp4_gated_backward(at_offset(dd, offset), at_offset(gu, offset), nv.NVFP4_ACT_GELU, got)
    assert torch.equal(got, want)
    ok()
    dgu.copy_(gu)
    nv.nvfp4_gated_backward(dd, dgu, nv.NVFP4_ACT_GELU, dgu)
    assert torch.equal(dgu, want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,offset", [(3000, 1001, 0), (999, 515, 0), (1200, 2050, 0), (500, 3001, 1),
                                              (40, 33, 0), (2000, 1008, 3), (7, 5000, 2)])
def test_backward_in_place_of_unaligned_rows(rows, cols, offset, dtype):
    """dgu over gu where rows share 16-byte units with their neighbours, again and again: the same bits
    as out of place, and nothing beside it changes."""
    dd, gu = _back_inputs(rows, cols, dtype, 4)
    dd = at_offset(dd, offset)
    want = torch.empty_like(gu)
    db, dc, ra = torch.empty(2 * cols, device=DEV), torch.empty(2 * cols, device=DEV), torch.empty(rows, device=DEV)
    nv.nvfp4_gated_backward(dd, gu, nv.NVFP4_ACT_SILU, want, dbias=db)
    got, ok = guarded((rows, 2 * cols), dtype, offset=offset)
    for _ in range(4):
        got.copy_(gu)
        nv.nvfp4_gated_backward(dd, got, nv.NVFP4_ACT_SILU, got, dbias=dc, row_amax=ra)
        assert torch.equal(got, want) and torch.equal(db, dc)
        assert torch.equal(ra, want.abs().amax(dim=1).float())
    ok()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(3000, 1001), (999, 515), (16000, 64), (2000, 1024), (777, 2056),
                                       (9001, 24), (5, 5000)])
def test_backward_sums_of_small_integers_are_exact(rows, cols, dtype):
    """g = dd u and u's gradient dd g of small integers (no activation): every partial sum is an integer
    below 2^24, so dbias is exact whatever the order of its additions."""
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    dd = torch.randint(-2, 3, (rows, cols), generator=g, device=DEV).to(dtype)
    gu = torch.randint(-3, 4, (rows, 2 * cols), generator=g, device=DEV).to(dtype)
    dgu, db = torch.empty_like(gu), torch.empty(2 * cols, device=DEV)
    nv.nvfp4_gated_backward(dd, gu, nv.NVFP4_ACT_NONE, dgu, dbias=db)
    want = torch.cat([dd.double() * gu[:, cols:].double(), dd.double() * gu[:, :cols].double()], dim=1)
    assert torch.equal(dgu.double(), want) and torch.equal(db.double(), want.sum(0))


@pytest.mark.parametrize("name", ["relu", "gelu", "silu", "none"])
def test_backward_at_the_ends(name):
    """Gates far out: act' is 0 or 1, act is 0 or g, and nothing overflows on the way."""
    big = torch.tensor([-3e38, -1e30, -1e4, -100.0, -65.0, -0.0, 0.0, 65.0, 100.0, 1e4, 1e30],
                       device=DEV)
    gu = torch.cat([big, torch.full_like(big, 2.0)])[None].contiguous()
    dd, dgu = torch.ones(1, big.numel(), device=DEV), torch.empty_like(gu)
    nv.nvfp4_gated_backward(dd, gu, ACTS[name], dgu)
    n = big.numel()
    if name == "none":
        assert bool((dgu[0, :n] == 2).all()) and torch.equal(dgu[0, n:], big)
        return
    far = big.abs() >= 65
    slope, value = dgu[0, :n] / 2, dgu[0, n:]
    assert torch.equal(slope[far], (big[far] > 0).float())
    # silu(-65) is -65 e^-65, about -4e-27
    assert bool((value[far & (big < 0)].abs() <= 1e-26).all())
    assert torch.equal(value[far & (big > 0)], big[far & (big > 0)])


def test_backward_against_differences():
    """The halves' gradients are the slopes of sum(dd act(g) u) in FP64 (tanh and exp of torch),
    by central differences of 2^-12: third derivatives below 4 leave 2^-23, FP64 nothing."""
    from layer_reference import act
    dd, gu = _back_inputs(4, 40, torch.float32, 12)
    for name in ("gelu", "silu", "none"):
        dgu = torch.empty_like(gu)
        nv.nvfp4_gated_backward(dd, gu, ACTS[name], dgu)
        e, x = 2.0 ** -12, gu.double()

        def loss(g, u):
            return dd.double() * act(g, name) * u
        g, u = x[:, :40], x[:, 40:]
        slope = torch.cat([(loss(g + e, u) - loss(g - e, u)) / (2 * e),
                           (loss(g, u + e) - loss(g, u - e)) / (2 * e)], dim=1)
        mag = dd.double().abs().repeat(1, 2) * (1 + x.abs().amax())
        assert bool(((dgu.double() - slope).abs() <= 2.0 ** -19 * mag * (1 + x.abs().amax())).all())
