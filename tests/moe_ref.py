"""Plain CPU implementations of the token sorting, dispatch and combine operators, in 64 bits where
they compute (numpy; no code of the library)."""
from __future__ import annotations

import numpy as np
import torch

ALIGN = 128


def sorted_rows(T, k, G):
    n = T * k
    return (n + min(n, G) * (ALIGN - 1) + ALIGN - 1) // ALIGN * ALIGN


def sort_contiguous(ids, G, rows):
    """(pos, m_indices, ks) by walking the assignments expert by expert."""
    T, k = ids.shape
    pos = np.full(T * k, -1, np.int32)
    m = np.full(rows, -2, np.int32)
    ks = np.zeros(G, np.int32)
    at = 0
    flat = ids.reshape(-1)
    for g in range(G):
        mine = np.nonzero(flat == g)[0]
        seg = (len(mine) + ALIGN - 1) // ALIGN * ALIGN
        for r, i in enumerate(mine):
            if at + r < rows:
                pos[i] = at + r
        m[at:at + len(mine)] = g
        m[at + len(mine):at + seg] = -1
        ks[g] = max(0, min(seg, rows - at))
        at += seg
    return pos.reshape(T, k), m, ks


def sort_masked(ids, G, m_max):
    T, k = ids.shape
    pos = np.full(T * k, -1, np.int32)
    count = np.zeros(G, np.int64)
    for i, e in enumerate(ids.reshape(-1)):
        if 0 <= e < G:
            if count[e] < m_max:
                pos[i] = e * m_max + count[e]
            count[e] += 1
    return pos.reshape(T, k), np.minimum(count, m_max).astype(np.int32)


def quantise(x, ue8m0=False):
    """x float32 [rows, H]: (E4M3 codes uint8, scales float32 [rows, H/128], exponents or None)."""
    b = x.astype(np.float32).reshape(x.shape[0], -1, 128)
    with np.errstate(all="ignore"):
        amax = np.abs(b).max(-1)                       # numpy's max keeps a NaN
        s = (amax / np.float32(448)).astype(np.float32)
        s = np.where(s < np.float32(2.0 ** -126), np.float32(2.0 ** -126), s)
        s = np.where(amax == 0, np.float32(1), s).astype(np.float32)
        e = None
        if ue8m0:
            m, ex = np.frexp(s.astype(np.float64))
            ex = np.where(m == 0.5, ex - 1, ex)
            e = np.where(np.isfinite(s), ex + 127, 255).astype(np.int64)
            s = np.where(np.isfinite(s), np.ldexp(1.0, np.where(np.isfinite(s), ex, 0)), np.nan).astype(np.float32)
        q = (b / s[..., None]).astype(np.float32)
        q = np.clip(q, np.float32(-448), np.float32(448))
    codes = torch.from_numpy(q.reshape(x.shape)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes, s, e


def combine(rows, pos, weights, residual):
    """(Y, sum of the absolute terms) in 64 bits; rows of dropped assignments are never touched."""
    T, k = pos.shape
    y = np.zeros((T, rows.shape[1])) if residual is None else residual.astype(np.float64).copy()
    mag = np.abs(y)
    for t in range(T):
        for j in range(k):
            r = pos[t, j]
            if 0 <= r < rows.shape[0]:
                v = (1.0 if weights is None else float(weights[t, j])) * rows[r].astype(np.float64)
                y[t] += v
                mag[t] += np.abs(v)
    return y, mag


def combine_backward(dy, rows, pos, weights):
    """({row: gradient}, d_weights, sum of the absolute products) in 64 bits."""
    T, k = pos.shape
    d_rows, dw, mag = {}, np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = int(pos[t, j])
            if 0 <= r < rows.shape[0]:
                d_rows[r] = (1.0 if weights is None else float(weights[t, j])) * dy[t].astype(np.float64)
                p = dy[t].astype(np.float64) * rows[r].astype(np.float64)
                dw[t, j], mag[t, j] = p.sum(), np.abs(p).sum()
    return d_rows, dw, mag
