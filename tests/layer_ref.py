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


# ------------------------------------------------------------------ routing
def scores(logits, score):
    """p of rows of logits; a row of nothing but -inf has zeros."""
    l = logits.double()
    if score == "sigmoid":
        return torch.sigmoid(l)
    p = torch.softmax(l, 1)
    return torch.where((l == -math.inf).all(1, keepdim=True), torch.zeros_like(p), p)


def route(logits, bias, k, score, groups=1, topk_groups=1, group_best=1, renormalise=True, scale=1.0):
    """(ids, weights) token by token, by sorting (value, lowest index) pairs."""
    T, E = logits.shape
    p = scores(logits, score)
    v = p if bias is None else p + bias.double()
    ids, weights = torch.full((T, k), -1, dtype=torch.int32), torch.zeros((T, k), dtype=torch.float64)
    size = E // groups
    for t in range(T):
        row = []                                     # (-value, expert) of the available ones
        for e in range(E):
            x = float(v[t, e])
            if float(logits[t, e]) == -math.inf or x == -math.inf:
                continue
            row.append((1e300 if math.isnan(x) else -x, e))
        if groups > 1:
            worth = []
            for g in range(groups):
                mine = sorted(r for r in row if r[1] // size == g)[:group_best]
                if mine:
                    worth.append((sum(r[0] for r in mine), g))
            keep = {g for _, g in sorted(worth)[:topk_groups]}
            row = [r for r in row if r[1] // size in keep]
        for j, (_, e) in enumerate(sorted(row)[:k]):
            ids[t, j], weights[t, j] = e, p[t, e]
    if renormalise:
        total = weights.sum(1, keepdim=True)
        weights = torch.where(total == 0, torch.zeros_like(weights), weights / total)
    return ids, scale * weights


def route_backward(logits, ids, d_weights, score, renormalise, scale):
    """(d_logits, magnitude of its terms)."""
    l = logits.double()
    T, E = l.shape
    p = scores(logits, score)
    out, mag = torch.zeros_like(p), torch.zeros_like(p)
    for t in range(T):
        mine = [(int(e), scale * float(d)) for e, d in zip(ids[t], d_weights[t]) if 0 <= int(e) < E]
        total = sum(float(p[t, e]) for e, _ in mine)
        mean = sum(d * float(p[t, e]) for e, d in mine) / total if renormalise and total else 0.0
        size = sum(abs(d) * float(p[t, e]) for e, d in mine) / total if renormalise and total else 0.0
        dp, dm = torch.zeros(E, dtype=torch.float64), torch.zeros(E, dtype=torch.float64)
        for e, d in mine:
            if renormalise and not total:
                continue
            dp[e] += (d - mean) / total if renormalise else d
            dm[e] += (abs(d) + size) / total if renormalise else abs(d)
        if score == "sigmoid":
            slope = p[t] * torch.sigmoid(-l[t])
            out[t], mag[t] = dp * slope, dm * slope
        else:
            out[t] = p[t] * (dp - (dp * p[t]).sum())
            mag[t] = p[t] * (dm + (0 if renormalise else (dm * p[t]).sum()))
            if renormalise:                          # the sum is zero: only the chosen get a gradient
                out[t] = p[t] * dp
    return out, mag


# ------------------------------------------------------------------ 8-bit checkpoints
def keep(x, m_indices=None):
    """(values x 2^-e [M,N] before the code's rounding, exponent bytes [M,ceil(N/128)]) of BF16 rows."""
    M, N = x.shape
    x = x.double()
    if m_indices is not None:
        x = torch.where((m_indices >= 0)[:, None], x, torch.zeros_like(x))
    B = -(-N // 128)
    e = torch.empty((M, B), dtype=torch.uint8)
    v = torch.empty_like(x)
    for t in range(M):
        for b in range(B):
            block = x[t, 128 * b:128 * b + 128]
            top = float(block.abs().max())
            if not bool(torch.isfinite(block).all()):
                e[t, b], v[t, 128 * b:128 * b + 128] = 255, math.nan
                continue
            k = 0 if top == 0 else -126
            while top > 448 * 2.0 ** k:
                k += 1
            block = block * 2.0 ** -k
            if k == 120:                     # 256 2^120 is past BF16's largest number
                block = block.clamp(-240, 240)
            e[t, b], v[t, 128 * b:128 * b + 128] = k + 127, block
    return v, e


def kept_values(codes, scales):
    """Values of codes [M,N] (uint8) with exponent bytes."""
    s = torch.where(scales == 255, torch.full((), math.nan, dtype=torch.float64), torch.exp2(scales.double() - 127))
    v = codes.view(torch.float8_e4m3fn).double()
    return v * s.repeat_interleave(128, 1)[:, :v.shape[1]]


def activation(z, name):
    """(activation, slope) of 64-bit z."""
    if name == "relu":
        return torch.relu(z), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        phi = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(u * (z + 0.044715 * z ** 3))
        return z * s, s + z * s * (1 - s) * u * (1 + 0.134145 * z * z)
    return z, torch.ones_like(z)


# ------------------------------------------------------------------ low-rank adapters
def lora(a, b, down, up, adapter, scale, bias):
    """(Z, magnitudes of the shared product's and of the adapters' terms)."""
    a = a.double()
    z, base = a @ b.double().t(), a.abs() @ b.double().abs().t()
    low = torch.zeros_like(z)
    for i in range(down.shape[0]):
        r = torch.nonzero(adapter == i)[:, 0]
        if not len(r):
            continue
        s = 1.0 if scale is None else float(scale[i])
        z[r] += s * (a[r] @ down[i].double().t()) @ up[i].double().t()
        low[r] += abs(s) * (a[r].abs() @ down[i].double().abs().t()) @ up[i].double().abs().t()
    if bias is not None:
        z, base = z + bias.double(), base + bias.double().abs()
    return z, base, low
