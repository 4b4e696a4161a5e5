"""Plain implementations in 64 bits of the operators around the products: norm, routing, 8-bit checkpoints and
low-rank adapters (torch on the CPU; no code of the library)."""
from __future__ import annotations

import math

import torch


# ------------------------------------------------------------------ norm
def rms_norm(x, residual, weight, eps):
    """(s, y) of rows x."""
    s = x.double() if residual is None else x.double() + residual.double()
    q = (s.pow(2).mean(1, keepdim=True) + eps) ** -0.5
    w = 1.0 if weight is None else weight.double()
    return s, s * q * w


def rms_norm_backward(dy, s, weight, eps, ds):
    """(dx, dweight, magnitudes of the terms of each)."""
    dy, s = dy.double(), s.double()
    q = (s.pow(2).mean(1, keepdim=True) + eps) ** -0.5
    n = s * q
    g = dy if weight is None else dy * weight.double()
    dx = q * (g - n * (g * n).mean(1, keepdim=True))
    mag = q * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if ds is not None:
        dx, mag = dx + ds.double(), mag + ds.double().abs()
    return dx, (dy * n).sum(0), mag, (dy * n).abs().sum(0)


def unpack_words(words, K):
    """Scales [T, K/128] that UE8M0 words [ceil(K/512), T] stand for."""
    w = words.long() & 0xffffffff
    e = torch.stack([(w >> (8 * j)) & 255 for j in range(4)], 1)            # [words, 4, T]
    e = e.reshape(-1, w.shape[1])[:K // 128].t()
    return torch.where(e == 255, torch.full((), math.nan, dtype=torch.float64), torch.exp2(e.double() - 127))


def e4m3_values(codes, scales):
    """Values of codes [T, K] with scales [T, K/128]."""
    v = codes.view(torch.float8_e4m3fn).double()
    return (v.reshape(v.shape[0], -1, 128) * scales.double()[..., None]).reshape(v.shape)
