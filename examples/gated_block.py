"""A pre-norm gated feed-forward block trained and served in NVFP4, on the library's kernels.

    h = residual + drop(x)                 nvfp4_add_layernorm (NVFP4 rows of the norm's y)
    a = silu(norm(h) Wg^T) * norm(h) Wu^T  nvfp4_gemm_gated, [g | u] kept for the backward, the
                                           maxima of a for its quantization
    out = a W2^T + b2 + h                  nvfp4_quantize_both, nvfp4_gemm_bias_act

and back: nvfp4_bias_act_backward and nvfp4_gated_backward give the products' gradients with the
maxima that their quantization takes, nvfp4_gemm the data and weight gradients (gate and up
projection in one product each), nvfp4_add_layernorm_backward the gradients of x (through the
dropout mask, made again from its seed) and of the residual.  Torch holds memory, draws the data
and applies the weight update.

    python examples/gated_block.py        # a few training steps, then one decoded token
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
    return _operand(row), _operand(col)


def _columns(t: torch.Tensor):
    """Columnwise NVFP4 alone, for a weight gradient."""
    rows, cols = t.shape
    col = nv.alloc_out(cols, rows, cols, t.device)
    nv.nvfp4_quantize_columnwise(t, CFG, col)
    return _operand(col)


class GatedBlock:
    """Weights in FP32; their NVFP4 forms are made again after every update."""

    def __init__(self, width: int, hidden: int, eps: float = 1e-5, device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std
        self.eps = eps
        self.params = {
            "norm": torch.ones(width, device=device), "shift": torch.zeros(width, device=device),
            "w1": normal(2 * hidden, width, std=width ** -0.5),  # the gate's lines, then up's
            "w2": normal(width, hidden, std=hidden ** -0.5), "b2": torch.zeros(width, device=device),
        }
        self.grads = {k: torch.empty_like(v) for k, v in self.params.items()}
        self.norm = torch.empty(1, device=device)
        self.quantize_weights()

    def quantize_weights(self) -> None:
        self.w1, self.w1_t = _both(self.params["w1"])
        self.w2, self.w2_t = _both(self.params["w2"])

    def forward(self, x: torch.Tensor, residual: torch.Tensor, mask=None):
        """out [tokens][width] (BF16) and what the backward needs; mask: an nv.Mask in training."""
        p, dev, (m, width) = self.params, x.device, x.shape
        hidden = p["w2"].shape[1]
        h, y, out = (torch.empty_like(x) for _ in range(3))
        mean, rstd = torch.empty(m, device=dev), torch.empty(m, device=dev)
        rows = nv.alloc_out(m, width, m, dev)
        nv.nvfp4_add_layernorm(x, p["norm"], self.eps, bias=p["shift"], residual=residual, mask=mask,
                               h=h, y=y, mean=mean, rstd=rstd, row=rows, cfg=CFG)
        a, gu = x.new_empty(m, hidden), x.new_empty(m, 2 * hidden)
        ra, ca = torch.empty(m, device=dev), torch.empty(hidden, device=dev)
        nv.nvfp4_gemm_gated(_operand(rows), self.w1, a, act=nv.NVFP4_ACT_SILU, gu=gu, row_amax=ra,
                            col_amax=ca)
        a_rows, a_cols = _both(a, ra, ca)
        nv.nvfp4_gemm_bias_act(a_rows, self.w2, out, bias=p["b2"], residual=h)
        return out, (h, y, mean, rstd, gu, a_cols, mask)

    def decode(self, x: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        """The forward pass alone: nothing kept, no column direction."""
        p, dev, (m, width) = self.params, x.device, x.shape
        hidden = p["w2"].shape[1]
        h, out, rows = torch.empty_like(x), torch.empty_like(x), nv.alloc_out(m, width, m, dev)
        nv.nvfp4_add_layernorm(x, p["norm"], self.eps, bias=p["shift"], residual=residual, h=h,
                               row=rows, cfg=CFG)
        a, a_rows = x.new_empty(m, hidden), nv.alloc_out(m, hidden, m, dev)
        a_rows.amax_in = torch.empty(m, device=dev)
        nv.nvfp4_gemm_gated(_operand(rows), self.w1, a, act=nv.NVFP4_ACT_SILU,
                            row_amax=a_rows.amax_in)
        nv.nvfp4_quantize_rowwise(a, CFG, a_rows)
        nv.nvfp4_gemm_bias_act(_operand(a_rows), self.w2, out, bias=p["b2"], residual=h)
        return out

    def backward(self, dout: torch.Tensor, saved):
        """Fills self.grads; returns the gradients of x and of residual."""
        h, y, mean, rstd, gu, a_cols, mask = saved
        p, g, (m, width), dev = self.params, self.grads, dout.shape, dout.device
        hidden = p["w2"].shape[1]
        dz, ra, ca = torch.empty_like(dout), torch.empty(m, device=dev), torch.empty(width, device=dev)
        nv.nvfp4_bias_act_backward(dout, None, nv.NVFP4_ACT_NONE, dz, dbias=g["b2"], row_amax=ra,
                                   col_amax=ca)
        row, col = _both(dz, ra, ca)
        nv.nvfp4_gemm(col, a_cols, g["w2"])
        da = dout.new_empty(m, hidden)
        nv.nvfp4_gemm(row, self.w2_t, da)
        ca = torch.empty(2 * hidden, device=dev)
        nv.nvfp4_gated_backward(da, gu, nv.NVFP4_ACT_SILU, gu, row_amax=ra, col_amax=ca)
        row, col = _both(gu, ra, ca)
        nv.nvfp4_gemm(col, _columns(y), g["w1"])
        dy = torch.empty_like(y)
        nv.nvfp4_gemm(row, self.w1_t, dy)
        dx, dr = torch.empty_like(h), torch.empty_like(h) if mask is not None else None
        nv.nvfp4_add_layernorm_backward(dy, h, p["norm"], mean, rstd, dx, dweight=g["norm"],
                                        dbias=g["shift"], dh=dout, mask=mask, dresidual=dr)
        return dx, dr if mask is not None else dx

    def step(self, rate: float, max_norm: float) -> torch.Tensor:
        """Clip the gradients by their global norm, descend, quantize the new weights; returns
        the norm before clipping."""
        nv.nvfp4_clip_grad_norm(list(self.grads.values()), max_norm, self.norm)
        for k, v in self.params.items():
            v.sub_(self.grads[k], alpha=rate)
        self.quantize_weights()
        return self.norm


def train(block: GatedBlock, tokens: int, steps: int, p: float = 0.1, rate: float = 0.2,
          seed: int = 1):
    """Fit the block to a fixed random map, with dropout; returns the losses."""
    width = block.params["norm"].numel()
    g = torch.Generator(device=block.norm.device)
    g.manual_seed(seed)
    x, r, t = (torch.randn(tokens, width, generator=g, device=block.norm.device).bfloat16()
               for _ in range(3))
    losses = []
    for i in range(steps):
        out, saved = block.forward(x, r, nv.Mask(p, seed, i))
        diff = out.float() - t.float()
        losses.append(0.5 * diff.square().mean())
        block.backward((diff / tokens).bfloat16(), saved)
        block.step(rate, max_norm=1.0)
    return [float(v) for v in losses]


if __name__ == "__main__":
    block = GatedBlock(512, 1536)
    losses = train(block, tokens=256, steps=10)
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    token = torch.randn(1, 512, device="cuda").bfloat16()
    out = block.decode(token, torch.zeros_like(token))
    print("one decoded token, first values:", [round(float(v), 3) for v in out[0, :4]])
