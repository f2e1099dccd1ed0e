"""A pre-norm MLP block trained and served in NVFP4, on the library's kernels alone.

    h = x + residual                      nvfp4_add_rmsnorm (NVFP4 rows of the norm's y)
    z = norm(h) W1^T + b1                 nvfp4_gemm_bias_act, z kept for the backward
    out = gelu(z) W2^T + b2 + h           nvfp4_quantize_both, nvfp4_gemm_bias_act

and back: nvfp4_bias_act_backward gives dz with the maxima its quantization takes,
nvfp4_gemm the data and weight gradients, nvfp4_add_rmsnorm_backward the stream's gradient,
nvfp4_clip_grad_norm the gradients of a step.  Torch holds memory, draws the data and
applies the weight update.

    python examples/mlp_block.py          # trains a small block, then decodes one token
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_precision_quantization_gb300 as nv  # noqa: E402

BOUND = 448.0
CFG = nv.Config(nv.NVFP4_ROW_SCALED, BOUND, 0, 0)


def _operand(o: nv.Out) -> nv.Operand:
    return o.as_operand(nv.NVFP4_ROW_SCALED, BOUND)


def _both(t: torch.Tensor, row_amax=None, col_amax=None):
    """Row- and columnwise NVFP4 of t [rows][cols], with given maxima where there are any."""
    rows, cols = t.shape
    row, col = nv.alloc_out(rows, cols, rows, t.device), nv.alloc_out(cols, rows, cols, t.device)
    row.amax_in, col.amax_in = row_amax, col_amax
    nv.nvfp4_quantize_both(t, CFG, row, col)
    return row, col


class MlpBlock:
    """Weights in FP32; their NVFP4 forms are made again after every update."""

    def __init__(self, width: int, hidden: int, eps: float = 1e-5, device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std
        self.eps, self.device = eps, device
        self.params = {
            "norm": torch.ones(width, device=device),
            "w1": normal(hidden, width, std=width ** -0.5), "b1": torch.zeros(hidden, device=device),
            "w2": normal(width, hidden, std=hidden ** -0.5), "b2": torch.zeros(width, device=device),
        }
        self.grads = {k: torch.empty_like(v) for k, v in self.params.items()}
        self.norm = torch.empty(1, device=device)
        self.quantize_weights()

    def quantize_weights(self) -> None:
        self.w1, self.w1_t = _both(self.params["w1"])
        self.w2, self.w2_t = _both(self.params["w2"])

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """out [tokens][width] (BF16) and what the backward needs."""
        p, (m, width) = self.params, x.shape
        hidden = p["w1"].shape[0]
        h, y, act = torch.empty_like(x), torch.empty_like(x), x.new_empty(m, hidden)
        z, out = torch.empty_like(act), torch.empty_like(x)
        rstd = torch.empty(m, device=x.device)
        y_rows = nv.alloc_out(m, width, m, x.device)
        nv.nvfp4_add_rmsnorm(x, p["norm"], self.eps, residual=residual, h=h, y=y, rstd=rstd,
                             row=y_rows, cfg=CFG)
        nv.nvfp4_gemm_bias_act(_operand(y_rows), _operand(self.w1), act, bias=p["b1"],
                               act=nv.NVFP4_ACT_GELU, z=z)
        a_rows = nv.alloc_out(m, hidden, m, x.device)
        nv.nvfp4_quantize_rowwise(act, CFG, a_rows)
        nv.nvfp4_gemm_bias_act(_operand(a_rows), _operand(self.w2), out, bias=p["b2"], residual=h)
        return out, (h, y, rstd, z, act)

    def backward(self, dout: torch.Tensor, saved) -> torch.Tensor:
        """Fills self.grads; returns the gradient of x and of residual."""
        h, y, rstd, z, act = saved
        p, g, (m, width), dev = self.params, self.grads, dout.shape, dout.device
        hidden = act.shape[1]

        def columns(t):
            col = nv.alloc_out(t.shape[1], t.shape[0], t.shape[1], dev)
            nv.nvfp4_quantize_columnwise(t, CFG, col)
            return _operand(col)

        def linear(dd, z, kind, name, x_cols, w_t, d_in):
            """dz of one linear layer, its bias and weight gradients, its input's gradient."""
            rows, cols = dd.shape
            dz = torch.empty_like(dd)
            ra, ca = torch.empty(rows, device=dev), torch.empty(cols, device=dev)
            nv.nvfp4_bias_act_backward(dd, z, kind, dz, dbias=g["b" + name], row_amax=ra, col_amax=ca)
            row, col = _both(dz, ra, ca)
            nv.nvfp4_gemm(_operand(col), x_cols, g["w" + name])
            nv.nvfp4_gemm(_operand(row), _operand(w_t), d_in)
            return d_in
        dact = linear(dout, None, nv.NVFP4_ACT_NONE, "2", columns(act), self.w2_t,
                      torch.empty_like(act))
        dy = linear(dact, z, nv.NVFP4_ACT_GELU, "1", columns(y), self.w1_t, torch.empty_like(y))
        dx = torch.empty_like(h)
        nv.nvfp4_add_rmsnorm_backward(dy, h, p["norm"], rstd, dx, dweight=g["norm"], dh=dout)
        return dx

    def step(self, rate: float, max_norm: float) -> torch.Tensor:
        """Clip the gradients by their global norm, descend, quantize the new weights; returns
        the norm before clipping."""
        nv.nvfp4_clip_grad_norm(list(self.grads.values()), max_norm, self.norm)
        for k, v in self.params.items():
            v.sub_(self.grads[k], alpha=rate)
        self.quantize_weights()
        return self.norm


def train(block: MlpBlock, tokens: int, steps: int, rate: float = 0.5, seed: int = 1):
    """Fit the block to a fixed random map; returns the losses."""
    width = block.params["norm"].numel()
    g = torch.Generator(device=block.device)
    g.manual_seed(seed)
    x, r, t = (torch.randn(tokens, width, generator=g, device=block.device).bfloat16()
               for _ in range(3))
    losses = []
    for _ in range(steps):
        out, saved = block.forward(x, r)
        diff = out.float() - t.float()
        losses.append(0.5 * diff.square().mean())
        # the mean over tokens of each token's squared error: gradients of order one
        block.backward((diff / tokens).bfloat16(), saved)
        block.step(rate, max_norm=1.0)
    return [float(v) for v in losses]


if __name__ == "__main__":
    block = MlpBlock(512, 2048)
    losses = train(block, tokens=256, steps=20)
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    token = torch.randn(1, 512, device="cuda").bfloat16()
    out, _ = block.forward(token, torch.zeros_like(token))
    print("one decoded token, first values:", [round(float(v), 3) for v in out[0, :4]])
