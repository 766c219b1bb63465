"""Bounds of the 4-bit cache's attention over long sequences that a lost step of a warp
shows through: sums are bounded as the kernels form them, roundings of single
weights in quadrature."""
import torch


def depth(n):
    """Additions that a term of a sum over n slots passes, at most: a lane (few columns) adds 4
    weights of 32 slots in 2 additions, of every 6th or 8th such group; a thread (many
    columns) 64 in 18, then one more a half tile; then lanes, warps, parts of CTAs."""
    return n / 64 + 64


def lse_bound(lse, eps, n):
    """eps: a logit's error (paged4_ref.attention).  Positive terms: the sum is off by depth
    2^-24 of itself; the exponential and the subtraction of a reference up to 20 away 2^-19; the
    sum with the reference and the change of base 2^-22 of the result."""
    return eps + depth(n) * 2.0 ** -24 + 2.0 ** -19 + lse.abs() * 2.0 ** -22


def row_bound(o, spread, eps, n):
    """Bound of the norm of a row's error.  spread: sqrt(sum_j p_j^2 v_j^2) per value.  The
    output's bf16: 2^-8 of it.  Weights are off independently of one another, by 2^-11 (fp16), 2 eps
    and 2^-19 at most: in quadrature that times the spread; 8 times it leaves room.  The
    product's partial sums, walks of 4 spreads at most, are rounded (or truncated: 2^-23) n / 16
    times; the sum they are divided by as in lse_bound."""
    w = 8 * (2.0 ** -11 + 2 * eps + 2.0 ** -19) + 4 * n / 16 * 2.0 ** -23
    return (2.0 ** -8 + depth(n) * 2.0 ** -24) * o.norm(dim=-1) + w * spread.norm(dim=-1) + 1e-30


def attention(q, k, v, seen, scale):
    """float64: q [R, D], k and v [n, D], seen [R, n]: outputs, log-sums, spreads, a logit's error."""
    s = (q @ k.T) * scale
    mag = float(((q.abs() @ k.abs().T) * abs(scale)).masked_fill(~seen, 0.0).max())
    s = s.masked_fill(~seen, -torch.inf)
    lse = torch.logsumexp(s, dim=-1)
    p = torch.where(seen, torch.exp(s - lse[:, None]), 0.0)
    # (as paged4_ref.attention: fp32 sums of D products in any order, the query's fp16 form, the scale)
    return p @ v, lse, (p.square() @ v.square()).sqrt(), mag * (q.shape[1] + 8) * 2.0 ** -23, p
