"""The gated block's operators together: the block of examples/gated_block.py."""
import os
import sys

import pytest
import torch

import nvfp4_precision_quantization_gb300 as nv
from block_reference import drop

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
pytestmark = pytest.mark.gpu


def _cosine(u, v):
    return float((u.double() * v.double()).sum() / u.double().norm() / v.double().norm())


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("tokens,width,hidden", [(128, 256, 512), (1024, 512, 2560)])
def test_gradients_point_with_the_unquantized_block(tokens, width, hidden, p):
    """NVFP4 keeps about three significant bits a value: gradients through four quantized
    products agree in direction with the FP64 block's (noise of 10 to 20 % a product, of random
    sign: a cosine above 0.9).  A wrong or shifted mask alone would take 20 % of the energy."""
    import gated_block
    block = gated_block.GatedBlock(width, hidden, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x, r, t = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3))
    mask = nv.Mask(p, 5, 6) if p else None
    out, saved = block.forward(x, r, mask)
    dout = (out.float() - t.float()).bfloat16()
    dx, dr = block.backward(dout, saved)
    params = {k: v.double().requires_grad_() for k, v in block.params.items()}
    xd, rd = x.double().requires_grad_(), r.double().requires_grad_()
    keep = drop(torch.ones_like(xd), p, 5, 6).detach() if p else torch.ones_like(xd)
    h = rd + xd * keep
    c = h - h.mean(1, keepdim=True)
    y = c * (c.square().mean(1, keepdim=True) + block.eps).rsqrt() * params["norm"] + params["shift"]
    gate, up = (y @ params["w1"].t()).chunk(2, dim=1)
    ref = (torch.nn.functional.silu(gate) * up) @ params["w2"].t() + params["b2"] + h
    ref.backward(dout.double())
    assert _cosine(out, ref.detach()) > 0.98
    assert _cosine(dr, rd.grad) > 0.9 and _cosine(dx, xd.grad) > 0.9
    if p:
        assert bool((dx[keep == 0] == 0).all())
    for k in params:
        assert _cosine(block.grads[k], params[k].grad) > 0.9, k


def test_training_runs_and_one_token_decodes():
    import gated_block
    block = gated_block.GatedBlock(256, 768, seed=5)
    losses = gated_block.train(block, tokens=128, steps=3)
    assert all(v == v and v < 1e3 for v in losses)
    x = torch.randn(96, 256, device="cuda").bfloat16()
    whole, _ = block.forward(x, torch.zeros_like(x))
    many = block.decode(x, torch.zeros_like(x))
    assert torch.equal(whole, many)
    one = block.decode(x[40:41].contiguous(), torch.zeros_like(x[:1]))
    # sums in another order, so a code may flip: BF16 steps of the larger terms
    assert float((whole[40] - one[0]).abs().max()) <= 2.0 ** -6 * float(whole[40].abs().max())


def test_training_step_in_a_graph():
    """Forward and backward captured once; offset_add gives each replay another mask, the same
    as calls made one by one."""
    import gated_block
    block = gated_block.GatedBlock(256, 512, seed=7)
    x, r, d = (torch.randn(64, 256, device="cuda").bfloat16() for _ in range(3))
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    mask = nv.Mask(0.3, 9, 100, offset_add=count)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):  # loads the kernels
        out, saved = block.forward(x, r, mask)
        block.backward(d, saved)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, saved = block.forward(x, r, mask)
        dx, dr = block.backward(d, saved)
        count.add_(1)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, dx, dr, block.grads["w1"])]
        one, saved = block.forward(x, r, nv.Mask(0.3, 9, 100 + i))
        ex, er = block.backward(d, saved)
        for a, b in zip(got, (one, ex, er, block.grads["w1"])):
            assert torch.equal(a, b)


def test_columns_alone_are_those_of_both_directions():
    """The weight gradient's operand, quantized without the rows that nothing reads."""
    import gated_block
    y = torch.randn(192, 320, device="cuda").bfloat16()
    one, two = gated_block._columns(y), gated_block._both(y)[1]
    for f in ("codes", "scales", "amax"):
        assert torch.equal(getattr(one, f), getattr(two, f))
