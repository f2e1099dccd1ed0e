"""Calls in a row on one stream: the first launch of a call starts only when everything
before it is done.

A kernel launched with a programmatic dependency may start while the kernel before it still
runs, and the encode kernel loads x before it waits.  So the first launch of a call has to be
an ordinary one: between two calls the captured graph must hold full edges only.  (The graphs
are captured to be read; the values are checked apart.)
"""
import ctypes as C

import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROWS, COLS = 32, 512
RS, PT = nv.NVFP4_ROW_SCALED, nv.NVFP4_PER_TENSOR
PROGRAMMATIC = 1  # CU_GRAPH_DEPENDENCY_TYPE_PROGRAMMATIC


class _EdgeData(C.Structure):
    _fields_ = [("from_port", C.c_ubyte), ("to_port", C.c_ubyte), ("type", C.c_ubyte),
                ("reserved", C.c_ubyte * 5)]


def _edge_types(*calls):
    """The dependency types of the chain of launches that the calls make on one stream."""
    cu = C.CDLL("libcuda.so.1")
    s, graph = torch.cuda.Stream(), C.c_void_p()
    torch.cuda.synchronize()
    stream = C.c_void_p(s.cuda_stream)
    assert cu.cuStreamBeginCapture_v2(stream, C.c_int(2)) == 0  # relaxed
    try:
        for call in calls:
            call(s)
    finally:
        rc = cu.cuStreamEndCapture(stream, C.byref(graph))
    assert rc == 0
    nodes, edges = C.c_size_t(0), C.c_size_t(0)
    assert cu.cuGraphGetNodes(graph, None, C.byref(nodes)) == 0
    assert cu.cuGraphGetEdges_v2(graph, None, None, None, C.byref(edges)) == 0
    n = edges.value
    assert n == nodes.value - 1  # a chain
    a, b, data = (C.c_void_p * n)(), (C.c_void_p * n)(), (_EdgeData * n)()
    assert n == 0 or cu.cuGraphGetEdges_v2(graph, a, b, data, C.byref(edges)) == 0
    assert cu.cuGraphDestroy(graph) == 0
    after = {a[i]: (b[i], data[i].type) for i in range(n)}
    node = next(iter(set(a) - set(b)), None)
    types = []
    while node in after:
        node, t = after[node]
        types.append(t)
    return types


def _out(lines, n, rs):
    """An output whose amax is given in place."""
    o = nv.alloc_out(lines, n, lines if rs else 1)
    o.amax.fill_(3.0)
    o.amax_in = o.amax
    return o


def _quantizes(x):
    """Every quantize whose first launch is its encode: the amax is given in place."""
    rows, cols = x.shape
    rs, fos, pt = (nv.Config(RS, 448.0, 0, 0), nv.Config(RS, 448.0, 1, 0),
                   nv.Config(PT, 448.0, 0, 0))
    r, c = _out(rows, cols, True), _out(cols, rows, True)
    r1, c1 = _out(rows, cols, False), _out(cols, rows, False)
    ws = torch.empty(rows * cols, device=DEV)
    pt2d = nv.Config(PT, 448.0, 0, 1)
    return {
        "rowwise": lambda s: nv.nvfp4_quantize_rowwise(x, rs, r, stream=s),
        "columnwise": lambda s: nv.nvfp4_quantize_columnwise(x, rs, c, stream=s),
        "both": lambda s: nv.nvfp4_quantize_both(x, rs, r, c, stream=s),
        "both four-over-six": lambda s: nv.nvfp4_quantize_both(x, fos, r, c, stream=s),
        "per tensor": lambda s: nv.nvfp4_quantize_both(x, pt, r1, c1, stream=s),
        "transform": lambda s: nv.nvfp4_quantize_columnwise_rht(x, 0x6D2B, rs, c, stream=s),
        "transform both": lambda s: nv.nvfp4_quantize_both_rht(x, 0x6D2B, rs, r, c, stream=s),
        "transform 16x16": lambda s: nv.nvfp4_quantize_columnwise_rht(x, 0x6D2B, pt2d, c1,
                                                                      workspace=ws, stream=s),
    }, (r, c, r1, c1)


def _producers(dtype):
    """Backward passes that launch no joining kernel, and what they write."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    z, dd = (torch.randn(ROWS, COLS, generator=g, device=DEV).to(dtype) for _ in range(2))
    w, rstd = torch.ones(COLS, device=DEV), torch.rand(ROWS, generator=g, device=DEV) + 0.5
    dz, dx = torch.empty_like(z), torch.empty_like(z)
    return {
        "activation": (dz, lambda s: nv.nvfp4_bias_act_backward(dd, z, nv.NVFP4_ACT_GELU, dz,
                                                                stream=s)),
        "norm": (dx, lambda s: nv.nvfp4_add_rmsnorm_backward(dd, z, w, rstd, dx, stream=s)),
    }


@pytest.mark.parametrize("producer", ["activation", "norm"])
def test_full_edges_between_calls(producer):
    x, make = _producers(torch.bfloat16)[producer]
    calls, _ = _quantizes(x)
    make(None)
    for call in calls.values():  # loads the kernels
        call(None)
    before = len(_edge_types(make))
    inside = 0
    for name, call in calls.items():
        types = _edge_types(make, call)
        assert types[before] != PROGRAMMATIC, name
        inside += PROGRAMMATIC in types[before + 1:]
    assert inside  # the four-over-six call's second pass: such edges are seen where they are


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("producer", ["activation", "norm"])
def test_quantize_takes_what_the_call_before_wrote(producer, dtype):
    """Few rows, so that the next kernel would find idle SMs, against a pass with a wait
    between the calls."""
    x, make = _producers(dtype)[producer]
    calls, outs = _quantizes(x)
    for name, call in calls.items():
        make(None)
        torch.cuda.synchronize()
        for o in outs:
            o.codes.zero_()
        call(None)
        torch.cuda.synchronize()
        want = [(o.codes.clone(), o.scales.clone()) for o in outs]
        for _ in range(20):
            x.zero_()
            for o in outs:
                o.codes.zero_()
            torch.cuda.synchronize()
            make(None)
            call(None)
            torch.cuda.synchronize()
            for o, (codes, scales) in zip(outs, want):
                assert torch.equal(o.codes, codes) and torch.equal(o.scales, scales), name
