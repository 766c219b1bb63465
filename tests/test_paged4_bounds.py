"""The bounds of tests/paged4_bounds.py on the CPU: a computation with the kernels'
roundings keeps them, one that loses 32 slots of the longest sequences does not."""
import pytest
import torch

import paged4_bounds as pb


@pytest.mark.parametrize("n", [300, 20000, 40000, 65536])
@pytest.mark.parametrize("D", [64, 128])
def test_a_lost_group_shows(n, D):
    g = torch.Generator().manual_seed(n + D)
    R = 8
    k, v = (torch.randn(n, D, generator=g, dtype=torch.float64).to(torch.float8_e4m3fn).double() for _ in range(2))
    q = torch.randn(R, D, generator=g, dtype=torch.float64).bfloat16().double()
    scale = D ** -0.5
    o, lse, spread, eps, _ = pb.attention(q, k, v, torch.ones(R, n, dtype=torch.bool), scale)

    def kernel(keep):
        """fp32 logits, weights to a reference 6 below the largest, fp16 for their product, bf16 results."""
        s = (q.float() @ k[keep].float().T) * torch.tensor(scale * 1.4426950408889634).float()
        ref = s.amax(dim=-1, keepdim=True) - 6
        w = torch.exp2(s - ref)
        total = w.double().sum(dim=-1).float()
        out = (w.half().double() @ v[keep]).float() / total[:, None]
        return out.bfloat16().double(), ((ref[:, 0] + total.log2()) * 0.6931471805599453).double()

    every = torch.ones(n, dtype=torch.bool)
    out, got = kernel(every)
    assert ((out - o).norm(dim=-1) <= pb.row_bound(o, spread, eps, n)).all()
    assert ((got - lse).abs() <= pb.lse_bound(lse, eps, n)).all()
    for first in (0, n // 2 // 32 * 32, (n - 33) // 32 * 32):
        lost = every.clone()
        lost[first:first + 32] = False
        out, got = kernel(lost)
        # (rows of one KV head lose the same keys: one that shows it is enough)
        assert ((out - o).norm(dim=-1) > pb.row_bound(o, spread, eps, n)).any(), first
        assert ((got - lse).abs() > pb.lse_bound(lse, eps, n)).all(), first
