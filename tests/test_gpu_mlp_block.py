"""The layer operators together: the MLP block of examples/mlp_block.py."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
pytestmark = pytest.mark.gpu


def test_gradients_point_with_the_unquantized_block():
    """NVFP4 keeps about three significant bits a value: gradients through four quantized
    products agree in direction with the FP64 block's (noise of 10 to 20 % a product, of
    random sign: a cosine above 0.9), and the loss falls when trained."""
    import mlp_block
    block = mlp_block.MlpBlock(256, 1024, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x, r, t = (torch.randn(128, 256, generator=g, device="cuda").bfloat16() for _ in range(3))
    out, saved = block.forward(x, r)
    dout = (out.float() - t.float()).bfloat16()
    dx = block.backward(dout, saved)
    p = {k: v.double().requires_grad_() for k, v in block.params.items()}
    xd = x.double().requires_grad_()
    h = xd + r.double()
    y = h * p["norm"] * (h.square().mean(1, keepdim=True) + block.eps).rsqrt()
    a = torch.nn.functional.gelu(y @ p["w1"].t() + p["b1"], approximate="tanh")
    ref = a @ p["w2"].t() + p["b2"] + h
    ref.backward(dout.double())

    def cosine(u, v):
        return float((u.double() * v.double()).sum() / u.double().norm() / v.double().norm())
    assert cosine(out, ref.detach()) > 0.98
    assert cosine(dx, xd.grad) > 0.9
    for k in p:
        assert cosine(block.grads[k], p[k].grad) > 0.9, k


def test_training_lowers_the_loss_and_one_token_decodes():
    import mlp_block
    block = mlp_block.MlpBlock(256, 512, seed=5)
    losses = mlp_block.train(block, tokens=128, steps=12)
    assert losses[-1] < 0.9 * losses[0] and all(b < 1.05 * a for a, b in zip(losses, losses[1:]))
    x = torch.randn(96, 256, device="cuda").bfloat16()
    whole, _ = block.forward(x, torch.zeros_like(x))
    one, _ = block.forward(x[40:41].contiguous(), torch.zeros_like(x[:1]))
    # the same codes, sums in another order: BF16 steps of the larger terms
    assert float((whole[40] - one[0]).abs().max()) <= 2.0 ** -6 * float(whole[40].abs().max())
