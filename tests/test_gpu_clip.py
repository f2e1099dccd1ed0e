"""Global gradient norm and clipping on the GPU against FP64.

Tolerance: a thread's FP32 sum takes 32 squares in four chains (2^-20 of the sum), the
rest is FP64; the square root halves it, the store rounds once: 2^-20 relative for the
norm.  A scaled value adds the coefficient's division and one product: 2^-19, and the
rounding to its type."""
import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv
from layer_reference import at_offset, guarded, half_ulp

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _list(sizes, seed, std=0.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ts = []
    for i, n in enumerate(sizes):
        t = std * torch.randn(n, generator=g, device=DEV)
        ts.append(t.to(torch.bfloat16 if i % 3 else torch.float32))
    return ts


def _norm(ts):
    return sum(float(t.double().square().sum()) for t in ts) ** 0.5


LISTS = [[1], [5], [0], [0, 7, 0], [16384], [16385, 3, 32768], [1, 2, 3, 5, 8, 13, 21],
         [100_003, 17, 4096, 250_000], [64] * 700, [3_000_001], []]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{sum(s)}")
@pytest.mark.parametrize("part", [0.25, 4.0])
def test_clip(sizes, part):
    ts = _list(sizes, len(sizes) + sum(sizes))
    want = _norm(ts)
    max_norm = want * part if want else 1.0
    outs, checks = zip(*[guarded(t.shape, t.dtype) for t in ts]) if ts else ((), ())
    norm, ok = guarded((1,), torch.float32)
    nv.nvfp4_clip_grad_norm(ts, max_norm, norm, out=list(outs))
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= 2.0 ** -20 * want
    coef = min(1.0, max_norm / (want + 1e-6))
    for t, o, check in zip(ts, outs, checks):
        e = t.double() * coef
        assert bool(((o.double() - e).abs() <= (2.0 ** -19 + half_ulp(t.dtype)) * e.abs()).all())
        if part > 1:
            assert torch.equal(o, t)
        check()
    ok()
    only = torch.empty(1, device=DEV)
    nv.nvfp4_grad_norm(ts, only)
    assert torch.equal(only, norm)


def test_in_place_is_the_same():
    ts = _list([70_001, 12, 40_000], 5)
    outs = [torch.empty_like(t) for t in ts]
    norm, norm2 = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    nv.nvfp4_clip_grad_norm(ts, 1.0, norm, out=outs)
    kept = [t.clone() for t in ts]
    nv.nvfp4_clip_grad_norm(ts, 1e9, norm2)  # nothing to clip: untouched
    assert all(torch.equal(a, b) for a, b in zip(ts, kept)) and torch.equal(norm, norm2)
    nv.nvfp4_clip_grad_norm(ts, 1.0, norm2)
    assert all(torch.equal(a, b) for a, b in zip(ts, outs)) and torch.equal(norm, norm2)


def test_unaligned_tensors_and_views():
    ts = _list([5000, 30_000, 1111], 6)
    outs = [torch.empty_like(t) for t in ts]
    norm, norm2 = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    nv.nvfp4_clip_grad_norm(ts, 1.0, norm, out=outs)
    for offset in (1, 4, 8):
        moved = [at_offset(t, offset) for t in ts]
        into = [guarded(t.shape, t.dtype, offset=offset) for t in ts]
        nv.nvfp4_clip_grad_norm(moved, 1.0, norm2, out=[o for o, _ in into])
        assert torch.equal(norm, norm2)
        for o, (p, ok) in zip(outs, into):
            assert torch.equal(o, p)
            ok()


def test_non_finite():
    for bad, norm_is, out_is in ((float("inf"), float("inf"), 0.0), (float("nan"),) * 3):
        ts = _list([1000, 50], 7)
        ts[0][17] = bad
        norm = torch.empty(1, device=DEV)
        nv.nvfp4_clip_grad_norm(ts, 1.0, norm)
        assert str(float(norm)) == str(norm_is)
        assert str(float(ts[1][3].abs())) == str(out_is)
    # zero gradients stay zero
    ts = [torch.zeros(100, device=DEV)]
    nv.nvfp4_clip_grad_norm(ts, 0.5, norm)
    assert float(norm) == 0.0 and float(ts[0].abs().max()) == 0.0
    # max_norm 0 clears everything
    ts = _list([100], 8)
    nv.nvfp4_clip_grad_norm(ts, 0.0, norm)
    assert float(ts[0].abs().max()) == 0.0


def test_repeatable_and_captured():
    """The same bits every time, also from a captured graph."""
    ts = _list([400_000, 33, 90_000], 9)
    outs, outs2 = ([torch.empty_like(t) for t in ts] for _ in range(2))
    norm, norm2 = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    ws = torch.empty(nv.nvfp4_clip_grad_norm_workspace_size(), dtype=torch.uint8, device=DEV)
    nv.nvfp4_clip_grad_norm(ts, 1.0, norm, out=outs, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_clip_grad_norm(ts, 1.0, norm2, out=outs2, workspace=ws)
    for _ in range(3):
        norm2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, norm2)
        assert all(torch.equal(a, b) for a, b in zip(outs, outs2))
