"""FP64 definitions of the gated block's operators (torch), and the dropout mask in numpy, for
the tests."""
from __future__ import annotations

import numpy as np
import torch

from layer_reference import act, act_slope

PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)


def philox4x32(counter, key, rounds=10):
    """The words of the blocks whose counters are the columns of `counter` [4][n] (uint64 values
    below 2^32), under the key (two 32-bit words)."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(PHILOX_M[0]), c[2] * np.uint64(PHILOX_M[1])
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(v + w) & 0xFFFFFFFF for v, w in zip(k, PHILOX_W)]
    return c


def threshold(p):
    return int(np.floor(np.float64(np.float32(p)) * 65536.0 + 0.5))


def keep_mask(n, p, seed, offset, first=0):
    """Which of the elements first .. first + n - 1 are kept, as numpy booleans."""
    block = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)  # eight elements each
    low = np.uint64(0xFFFFFFFF)
    offset &= (1 << 64) - 1
    words = philox4x32((block & low, block >> np.uint64(32),
                        np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)),
                       (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    halves = [h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))]
    kept = np.stack([h >= np.uint64(threshold(p)) for h in halves], axis=1).reshape(-1)
    return kept[first % 8:first % 8 + n]


def drop(x, p, seed, offset):
    """x in FP64 through the mask."""
    x = x.double()
    if threshold(p) == 0:
        return x
    keep = torch.from_numpy(keep_mask(x.numel(), p, seed, offset)).to(x.device).view(x.shape)
    factor = 65536.0 / (65536 - threshold(p)) if threshold(p) < 65536 else 0.0
    return torch.where(keep, x * factor, torch.zeros_like(x))


def layernorm(x, residual, weight, bias, eps, mask=None):
    h = x.double() if mask is None else drop(x, *mask)
    if residual is not None:
        h = h + residual.double()
    mean = h.mean(dim=1)
    c = h - mean[:, None]
    rstd = (c.square().mean(dim=1) + eps).rsqrt()
    y = c * rstd[:, None] * weight.double()
    return h, mean, rstd, y + (bias.double() if bias is not None else 0.0)


def layernorm_backward(dy, h, weight, mean, rstd, dh, mask=None):
    """dx, dresidual, dweight, dbias."""
    dy, s = dy.double(), rstd.double()[:, None]
    n, g = (h.double() - mean.double()[:, None]) * s, dy * weight.double()
    d = s * (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True))
    if dh is not None:
        d = d + dh.double()
    return drop(d, *mask) if mask is not None else d, d, (dy * n).sum(dim=0), dy.sum(dim=0)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def operand_values(codes, scales, amax, bound):
    """The FP64 values of an NVFP4 operand: code * decode(scale) * amax / (bound * 6)."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], dim=2).flatten(1)
    sf = scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=1)
    return v * sf * (amax.double().reshape(-1, 1) / (bound * 6.0))


def gated_backward(dd, gu, name):
    n = dd.shape[1]
    dd, g, u = dd.double(), gu[:, :n].double(), gu[:, n:].double()
    return torch.cat([dd * u * act_slope(g, name), dd * act(g, name)], dim=1)
