"""Dropout from a counter-based generator on the GPU: the mask is that of the definition (numpy),
element for element, wherever a call starts and whatever its type; the sum is within 2^-23 of
|x factor| + |r| before it is rounded once."""
import numpy as np
import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv
from block_reference import drop, keep_mask, threshold
from layer_reference import at_offset, guarded, half_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float32]


def _kept(n, mask, dtype=torch.float32):
    """The mask as the kernel has it: a vector of ones goes through it."""
    y = torch.empty(n, dtype=dtype, device=DEV)
    nv.nvfp4_dropout(torch.ones(n, dtype=dtype, device=DEV), mask, y)
    return (y != 0).cpu().numpy(), y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 7, 16, 17, 511, 512, 513, 4096, 100003, 5000000])
@pytest.mark.parametrize("p,seed,offset", [(0.1, 0, 0), (0.5, (1 << 64) - 1, (1 << 64) - 1),
                                           (0.9, 0x123456789ABCDEF0, 1 << 33)])
def test_mask_is_the_definitions(n, dtype, p, seed, offset):
    keep, y = _kept(n, nv.Mask(p, seed, offset), dtype)
    assert np.array_equal(keep, keep_mask(n, p, seed, offset))
    factor = torch.tensor(65536.0 / (65536 - threshold(p))).to(dtype)
    assert bool((y[y != 0] == factor.item()).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,offset", [((1, 1), 0), ((333, 1001), 0), ((64, 4096), 0),
                                          ((5, 777), 1), ((100, 1000), 3), ((7, 512), 8), ((0, 5), 0)])
def test_values(shape, offset, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(shape[1])
    x, r = (at_offset(torch.randn(shape, generator=g, device=DEV).to(dtype), offset) for _ in range(2))
    for residual, p in ((None, 0.25), (r, 0.1), (r, 0.0), (None, 0.0), (r, 1.0)):
        y, ok = guarded(shape, dtype, offset=offset)
        nv.nvfp4_dropout(x, nv.Mask(p, 3, 4), y, residual=residual)
        torch.cuda.synchronize()
        want = drop(x, p, 3, 4)
        mag = want.abs()
        if residual is not None:
            want, mag = want + r.double(), mag + r.double().abs()
        half = half_ulp(dtype)
        assert bool(((y.double() - want).abs() <= 2.0 ** -23 * (1 + half) * mag + half * want.abs()).all())
        ok()
        if residual is None and p > 0:
            assert bool(((y == 0) | (want != 0)).all() and ((y != 0) | (want == 0) | (x == 0)).all())
    z = x.clone()
    nv.nvfp4_dropout(z, nv.Mask(0.1, 3, 4), z, residual=r)
    y = torch.empty_like(x)
    nv.nvfp4_dropout(x, nv.Mask(0.1, 3, 4), y, residual=r)
    assert torch.equal(y, z)
    z = r.clone()
    nv.nvfp4_dropout(x, nv.Mask(0.1, 3, 4), z, residual=z)
    assert torch.equal(y, z)


@pytest.mark.parametrize("bits", [32, 35])
def test_elements_past_32_bits(bits):
    """4.3 and 34.4 billion elements: the last ones have the bits of their own index, whose
    blocks' upper counter word is 0 and 1."""
    n = (1 << bits) + 4099
    if torch.cuda.mem_get_info()[0] < 2 * n + (8 << 30):
        pytest.skip("not enough memory")
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    nv.nvfp4_dropout(x, nv.Mask(0.5, 11, 12), x)
    first = (1 << bits) - 37
    got = (x[first:] != 0).cpu().numpy()
    assert np.array_equal(got, keep_mask(n - first, 0.5, 11, 12, first))
    assert not np.array_equal(got[37:], (x[:4099] != 0).cpu().numpy())


def test_shares_and_independence():
    """Of n draws the share dropped is within 5 standard deviations of the rounded p; masks of
    other seeds or offsets agree with it no more often than chance."""
    n, p = 1 << 22, 0.3
    q = threshold(p) / 65536.0
    base = _kept(n, nv.Mask(p, 1, 1))[0]
    five = 5 * (q * (1 - q) / n) ** 0.5
    assert abs((1 - base.mean()) - q) <= five
    same = q * q + (1 - q) * (1 - q)
    for seed, offset in ((2, 1), (1, 2), (1 + (1 << 32), 1), (1, 1 + (1 << 32))):
        other = _kept(n, nv.Mask(p, seed, offset))[0]
        assert abs((base == other).mean() - same) <= 5 * (same * (1 - same) / n) ** 0.5
    for lag in (1, 2, 8, 16, 512):
        assert abs((base[lag:] == base[:-lag]).mean() - same) <= 6 * (same * (1 - same) / n) ** 0.5


def test_edges_of_p():
    n = 100000
    assert _kept(n, nv.Mask(0.0, 1, 1))[0].all()
    assert _kept(n, nv.Mask(2.0 ** -18, 1, 1))[0].all()  # rounds to no element
    assert not _kept(n, nv.Mask(1.0, 1, 1))[0].any()
    assert not _kept(n, nv.Mask(1.0 - 2.0 ** -20, 1, 1))[0].any()
    for p in (2.0 ** -16, 1.0 - 2.0 ** -16):
        assert np.array_equal(_kept(1 << 20, nv.Mask(p, 5, 6))[0], keep_mask(1 << 20, p, 5, 6))


def test_dropped_values_do_not_matter():
    x = torch.full((4096,), float("nan"), device=DEV)
    x[::3] = float("inf")
    y = torch.empty_like(x)
    nv.nvfp4_dropout(x, nv.Mask(0.5, 2, 3), y)
    keep = torch.from_numpy(keep_mask(4096, 0.5, 2, 3)).to(DEV)
    assert bool((y[~keep] == 0).all()) and not bool(y[keep].isfinite().any())


def test_captured_call_counts_on():
    """offset_add is read when the kernel runs: each replay of a graph has another mask."""
    x, y = torch.ones(10000, device=DEV), torch.empty(10000, device=DEV)
    count = torch.zeros(1, dtype=torch.int64, device=DEV)
    mask = nv.Mask(0.4, 21, 100, offset_add=count)
    nv.nvfp4_dropout(x, mask, y)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        nv.nvfp4_dropout(x, mask, y)
        count.add_(1)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal((y != 0).cpu().numpy(), keep_mask(10000, 0.4, 21, 100 + i))
