"""Plain NumPy float64 forms of the serving operators: adapters beside a packed layer, head
norms with the position rotation, rows of the 4-bit cache, attention over cached keys and
values. Each follows its definition step by step, one token and head at a time, and shares
no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from .gptq_oracle import dequantize_packed

F16_MAX = 65504.0


# ---------------------------------------------------------------- adapters
def adapter_linear(X, words, scales, zeros, bits, group_size, A, B, ids, alpha=None):
    """Y[t] = X[t] W_hat^T + alpha[a] B[a] (A[a] X[t]) with a = ids[t], nothing when negative."""
    X = np.asarray(X, dtype=np.float64)
    W = dequantize_packed(words, scales, zeros, bits, X.shape[1], group_size, None)
    Y = X @ W.T
    for t, a in enumerate(ids):
        if a >= 0:
            w = 1.0 if alpha is None else float(alpha[a])
            Y[t] += w * (np.asarray(B[a], np.float64) @ (np.asarray(A[a], np.float64) @ X[t]))
    return Y


# ---------------------------------------------------------------- norm and rotation
def norm_rope(x, positions=None, cos=None, sin=None, w=None, eps=1e-6, interleaved=False):
    """x (T, heads, D): the RMS norm of each head (w None: none), then each pair turned."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    if cos is None:
        return y
    half = cos.shape[1]
    out = y.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c = np.asarray(cos, np.float64)[positions, i][:, None]
        s = np.asarray(sin, np.float64)[positions, i][:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


# ---------------------------------------------------------------- the cache
def quantize_row(x):
    """(codes, scale, low) of one row: low and scale rounded to float16, true division, ties
    to even, each step in float32 as the cache's format defines it."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any():
        return np.zeros(x.shape, np.int64), np.float16(np.nan), np.float16(0)
    x = np.clip(x, -F16_MAX, F16_MAX)
    lo, hi = np.float32(x.min()), np.float32(x.max())
    scale = np.float16(np.float32(hi - lo) / np.float32(15))
    low = np.float16(lo)
    if scale == 0:
        return np.zeros(x.shape, np.int64), scale, low
    quotient = (x.astype(np.float32) - np.float32(low)) / np.float32(scale)     # both float32
    codes = np.clip(np.rint(quotient), 0, 15).astype(np.int64)
    return codes, scale, low


def block_bytes(page_size, dim):
    return page_size * (dim + 8)


def write_slot(pool, page_size, dim, slot, head, k_row, v_row):
    """Store one token's K and V rows of one head in pool (pages, heads, bytes) uint8."""
    page, at = divmod(int(slot), page_size)
    block = pool[page, head]
    for kv, row in enumerate((k_row, v_row)):
        codes, scale, low = quantize_row(row)
        start = (kv * page_size + at) * (dim // 2)
        block[start:start + dim // 2] = (codes[0::2] | (codes[1::2] << 4)).astype(np.uint8)
        n = page_size * dim + 8 * at + 4 * kv
        block[n:n + 4] = np.array([scale, low], dtype=np.float16).view(np.uint8)


def read_slot(pool, page_size, dim, slot, head):
    """(k, v) float64 of one token and head."""
    page, at = divmod(int(slot), page_size)
    block, out = pool[page, head], []
    for kv in range(2):
        start = (kv * page_size + at) * (dim // 2)
        b = block[start:start + dim // 2]
        codes = np.stack([b & 15, b >> 4], axis=-1).reshape(-1).astype(np.float64)
        n = page_size * dim + 8 * at + 4 * kv
        scale, low = block[n:n + 4].copy().view(np.float16).astype(np.float64)
        out.append(codes * scale + low)
    return out


def read_sequence(pool, page_size, dim, pages, n, head):
    """K and V (n, D) float64 of the first n tokens of a sequence whose pages are `pages`."""
    rows = [read_slot(pool, page_size, dim, int(pages[j // page_size]) * page_size + j % page_size, head)
            for j in range(n)]
    if not rows:
        return np.zeros((0, dim)), np.zeros((0, dim))
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def attention(q, k, v, first, sm_scale, causal=True, window=0):
    """q (n, D) at positions first, first + 1, ... over k, v (len, D): (o, lse). A query that
    sees no key gets zeros and -inf."""
    o, lse = np.zeros(q.shape), np.full(q.shape[0], -np.inf)
    for i in range(q.shape[0]):
        pos = first + i
        seen = np.arange(k.shape[0])
        if causal:
            seen = seen[seen <= pos]
        if window > 0:
            seen = seen[seen > pos - window]
        if seen.size == 0:
            continue
        z = sm_scale * (k[seen] @ q[i])
        m = z.max()
        e = np.exp(z - m)
        o[i] = (e @ v[seen]) / e.sum()
        lse[i] = m + np.log(e.sum())
    return o, lse
