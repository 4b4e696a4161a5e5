"""Plain CPU forms, in 64 bits, of the products with a fused epilogue and of their gradients."""
from __future__ import annotations

import math

import numpy as np
import torch
from scipy.special import erf, expit

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0)
    if name == "silu":
        return z * expit(z)
    if name == "gelu":
        return 0.5 * z * (1 + erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = expit(z)
        return s * (1 + z * expit(-z))
    if name == "gelu":
        return 0.5 * (1 + erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def values(p):
    """A [rows, K] and B [G, N, K] of a generated problem (tests/gen.py) in 64 bits, scales applied."""
    def of(t):
        return (t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t).double().numpy()
    a, b = of(p.A), of(p.B)
    K = a.shape[-1]
    if not p.bf16:
        sfa, sfb = np.moveaxis(p.sfa.numpy(), -2, -1), p.sfb.numpy()        # [.., rows, K/128], [.., N/128, K/128]
        if p.ue8m0:                                                         # four exponents a word
            def unpack(w):
                e = (w.view(np.uint32)[..., None] >> np.array([0, 8, 16, 24], np.uint32)) & 255
                return np.ldexp(1.0, e.astype(np.int64) - 127).reshape(*w.shape[:-1], -1)[..., :K // 128]
            sfa, sfb = unpack(np.ascontiguousarray(sfa)), unpack(sfb)
        a = a * np.repeat(sfa.astype(np.float64), 128, -1)
        b = b * np.repeat(np.repeat(sfb.astype(np.float64), 128, -2)[..., :b.shape[-2], :], 128, -1)
    return a.reshape(-1, K), b.reshape(-1, *b.shape[-2:])


def expert_of_rows(p):
    """Expert of each flat row, -1 where none computes it."""
    if p.kind == "dense":
        return np.zeros(p.A.shape[0], np.int64)
    if p.kind == "contiguous":
        m = p.m_indices.numpy().astype(np.int64)
        return np.where((m >= 0) & (m < p.B.shape[0]), m, -1)
    G, M = p.A.shape[:2]
    r = np.arange(M)[None, :]
    return np.where(r < p.masked_m.numpy()[:, None], np.arange(G)[:, None], -1).reshape(-1)


def forward(p, bias, name, residual):
    """(Z, D, computed rows): bias [G, N] and residual [rows, N] may be None."""
    a, b = values(p)
    g = expert_of_rows(p)
    z = np.zeros((a.shape[0], b.shape[1]))
    for e in range(b.shape[0]):
        rows = np.nonzero(g == e)[0]
        if len(rows):
            z[rows] = a[rows] @ b[e].T + (0 if bias is None else bias[e])
    d = act(z, name) + (0 if residual is None else residual)
    return z, d, g >= 0
