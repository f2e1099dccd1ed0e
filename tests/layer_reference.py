"""The layer operators' definitions in FP64 (torch), for the GPU tests."""
from __future__ import annotations

import math

import torch

C, A = math.sqrt(2.0 / math.pi), 0.044715
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(C * (z + A * z ** 3)))
    return z / (1 + torch.exp(-z)) if name == "silu" else z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        t = torch.tanh(C * (z + A * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C * (1 + 3 * A * z * z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def norm(x, residual, weight, eps):
    h = x.double() + (residual.double() if residual is not None else 0.0)
    rstd = (h.square().mean(dim=1) + eps).rsqrt()
    return h, rstd, h * weight.double() * rstd[:, None]


def norm_backward(dy, h, weight, rstd, dh):
    dy, h, rstd = dy.double(), h.double(), rstd.double()[:, None]
    n, g = h * rstd, dy * weight.double()
    dx = rstd * (g - n * (g * n).mean(dim=1, keepdim=True))
    return dx + (dh.double() if dh is not None else 0.0), (dy * n).sum(dim=0)


def half_ulp(dtype):
    """Unit roundoff of a stored value: 2^-p for a significand of p bits (8 and 24)."""
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def guarded(shape, dtype, device="cuda", offset=0, pad=64):
    """A tensor of `shape` inside a larger buffer of canary bytes, `offset` elements past
    a 256-byte boundary, and a check that nothing around it was written."""
    n = math.prod(shape)
    size = torch.empty((), dtype=dtype).element_size()
    buf = torch.full(((n + offset + 2 * pad) * size + 512,), 0xA5, dtype=torch.uint8,
                     device=device)
    first = (-buf.data_ptr()) % 256 + pad * 4 + offset * size
    first += (-first) % size
    t = buf[first:first + n * size].view(dtype).view(shape)

    def check():
        assert bool((buf[:first] == 0xA5).all()), "written before the buffer"
        assert bool((buf[first + n * size:] == 0xA5).all()), "written past the buffer"
    return t, check


def at_offset(t, offset):
    """A contiguous copy of t that starts `offset` elements past an aligned address."""
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device=t.device)
    v = buf[offset:].view(t.shape)
    v.copy_(t)
    return v
