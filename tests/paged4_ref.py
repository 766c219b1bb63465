"""The 4-bit paged cache in float64, from its definitions."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(byte):
    byte = np.asarray(byte).astype(np.int64)
    e, m = (byte >> 3) & 15, byte & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((byte & 127) == 127, np.nan, v)
    return np.where(byte & 128, -v, v)


_GRID = e4m3_value(np.arange(127))  # 0 .. 448, ascending


def _nearest(grid, x):
    """Index of the value nearest x (x >= 0), ties to the even index, the last for
    what lies past it."""
    x = np.minimum(x, grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def quantise(z):
    """float64 rows [..., D] -> (codes [..., D / 2], scales [..., D / 16]) uint8."""
    z = np.asarray(z, np.float64)
    b = z.reshape(z.shape[:-1] + (-1, 16))
    a = np.abs(b)
    bad = np.isnan(a).any(axis=-1)
    top = np.where(bad, 0.0, np.nan_to_num(a, nan=0.0, posinf=np.inf).max(axis=-1))
    s = _nearest(_GRID, np.maximum(np.minimum(top / 6, 1e30), 2.0 ** -9)).astype(np.uint8)
    with np.errstate(invalid="ignore"):
        code = _nearest(E2M1, np.nan_to_num(np.minimum(a, 1e30) / _GRID[s][..., None], nan=0.0))
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(b)).astype(np.uint8).reshape(z.shape)
    s = np.where(bad, 127, s).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def values(codes, scales):
    """(codes, scales) uint8 -> float64 rows."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[:-1] + (-1,))
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    return v * np.repeat(e4m3_value(scales), 16, axis=-1)


def rows(cache, table_row, h, n, P):
    """Slots 0 .. n - 1 of one sequence and KV head, and which of them are in a page."""
    codes, scales = cache
    j = np.arange(n)
    page = np.asarray(table_row)[j // P]
    ok = (page >= 0) & (page < codes.shape[0])
    page = np.where(ok, page, 0)
    return torch.from_numpy(values(codes[page, h, j % P], scales[page, h, j % P])), torch.from_numpy(ok)


def attention(q, k, v, ok, scale):
    """q [G, D], k and v [n, D], ok [n]: output, lse, logits, error of a logit, sum p |v|."""
    k, v = k[ok], v[ok]
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], q.shape[1], dtype=torch.float64)
        return z, torch.full((q.shape[0],), -np.inf, dtype=torch.float64), None, 0.0, z
    s = q @ k.T * scale
    p = torch.softmax(s, dim=-1)
    mag = float((q.abs() @ k.abs().T * abs(scale)).nan_to_num(0.0).max())
    # fp32 sums of D exact products, two to four partial sums, in any order and
    # truncating (2^-23 each); the query's fp16 form (2^-24), the scale's rounding
    eps = mag * (q.shape[1] + 8) * 2.0 ** -23
    return p @ v, torch.logsumexp(s, dim=-1), s, eps, p @ v.abs()


def out_bound(ref, mag, eps, n, vmax):
    """Largest |out - ref| of a bf16 output: half a step (2^-8 of the value), weights
    rounded to fp16 (2^-11), or lost below 2^-25 of a sum that is at least 2^6
    (n 2^-31 max |v|), logits off by eps (weight and sum: twice), the exponential
    (2^-21), fp32 sums of n terms and their merges."""
    e = (2.0 ** -11 + 2 * eps + 2.0 ** -21 + (n + 64) * 2.0 ** -23) * mag + n * 2.0 ** -31 * vmax
    return 2.0 ** -8 * (ref.abs() + e) + e + 1e-30


def lse_bound(lse, eps, n):
    return eps + (n + 64) * 2.0 ** -23 + 2.0 ** -20 + lse.abs() * 2.0 ** -22


def evict(length, newest, budget, recent, weight, born):
    """Per row: which slots stay, and the source of every slot of the new order."""
    n = int(length)
    keep = min(n, budget)
    order = []
    for j in range(n):
        w = weight[j]
        safe = int(born[j]) > int(newest) - recent
        order.append((not safe, 0.0 if safe else (-np.inf if np.isnan(w) else -w - 0.0), 0 if safe or np.isnan(w) else 1, j))
    kept = sorted(x[3] for x in sorted(order)[:keep])
    src = list(range(keep))
    movers = [j for j in kept if j >= keep]
    for j, m in zip([j for j in range(keep) if j not in set(kept)], movers):
        src[j] = m
    return src
