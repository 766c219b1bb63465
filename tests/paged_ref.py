"""Paged-cache operators in float64, from their definitions, key by key."""
import math

import numpy as np
import torch


def rope_freqs(dim, base, factor=1.0, orig=0, fast=32.0, slow=1.0):
    i = np.arange(dim // 2)
    f = base ** (-2.0 * i / max(dim, 1))
    if orig > 0:
        def at(turns):
            return dim * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), dim - 1)
        w = np.clip((i - low) / max(high - low, 1e-3), 0, 1)
        f = f / factor * w + f * (1 - w)
    return f


def rotate(x, pos, freqs, halves):
    """x [T, heads, D] float64, pos [T]: (rotated values, |a| + |b| of each value's pair)."""
    dim = 2 * len(freqs)
    y, mag = x.clone(), x.abs().clone()
    if dim == 0:
        return y, mag
    ang = torch.from_numpy(np.outer(np.asarray(pos, dtype=np.float64), freqs))[:, None]
    c, s = ang.cos(), ang.sin()
    D = x.shape[-1]
    ia = torch.arange(dim // 2) + D - dim if halves else 2 * torch.arange(dim // 2) + D - dim
    ib = ia + (dim // 2 if halves else 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def attention(q, k, v, scale):
    """q [G, D], k and v [n, D] float64: (output, sum of p |v|, logit error scale, n)."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64)
        return z, z, 0.0
    s = q @ k.T * scale
    p = torch.softmax(s, dim=-1)
    eps = float((q.abs() @ k.abs().T * abs(scale)).max()) * q.shape[1] * 2.0 ** -23
    return p @ v, p @ v.abs(), eps


def gather(cache, table_row, h, keys, P):
    """Rows of the given positions of one sequence, [n, D] float64."""
    keys = torch.as_tensor(keys, dtype=torch.long)
    pages = torch.as_tensor(table_row, dtype=torch.long)[keys // P]
    return cache[pages, h, keys % P].double()


def block_keys(p, P, idx_row, local, max_pages):
    """Positions a token attends: its list's pages (in list order) and the local ones."""
    last = p // P
    f = max(last + 1 - local, 0)
    keys = []
    for j in idx_row:
        j = int(j)
        if 0 <= j < f:
            keys += list(range(j * P, min((j + 1) * P - 1, p) + 1))
    return keys + list(range(f * P, p + 1))


def attn_bound(ref, mag, eps, n):
    """Largest |out - ref| of a bf16 output: half a bf16 step of the value (eps /
    2 = 2^-8), weights rounded to bf16 (2^-8 of sum p |v|), logits off by eps
    (weight and sum: twice), fp32 sums of n terms (truncating adds: 2^-23)."""
    e = (2.0 ** -8 + 2 * eps + (n + 8) * 2.0 ** -23) * mag
    return 2.0 ** -8 * (ref.abs() + e) + e + 1e-30
