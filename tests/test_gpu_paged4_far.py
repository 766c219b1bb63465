"""The 4-bit cache where numbers are far from ordinary ones: logits past 2^24."""
import numpy as np
import pytest
import torch

import paged4_ref as r4
from test_gpu_paged4 import Case, step

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("G", [8, 16, 32])
def test_logits_where_a_step_of_fp32_is_not_small(G):
    """Keys of two kinds, whose logits (in powers of two) are m 2^e and up to 32 more, first
    the lower ones.  The steps of fp32 at 2^24 .. 2^28 are 2 .. 16: a reference 6 below the
    first kind is rounded, and so is what it is compared with, so a weight may come out as
    2^16, past fp16, where the comparison is not that of the weight itself.  A logit is off
    by a few steps, so which kind prevails is open; but outputs lie between the two kinds'
    values, 1 and 2, and the log-sum is the larger logit to 2^-20 of it (16 steps)."""
    n, Hkv = 512, 2
    rows = [((1 + m / 8) * 2.0 ** e, d) for e in range(24, 28) for m in range(8) for d in (8.0, 12.0, 16.0, 20.0, 24.0, 32.0)]
    lens = [n] * len(rows)
    c = Case(1, lens, D=128, P=64, Hkv=Hkv, G=G)
    kc, ks = np.zeros((2, 64), np.uint8), np.full((2, 8), 0x38, np.uint8)   # scales of 1
    kc[:, 0], kc[1, 8] = 2, 2                                               # value 0, and of the second kind value 16: 1
    vc, vs = np.array([[0x22] * 64, [0x44] * 64], np.uint8), ks
    assert r4.values(kc, ks).sum(axis=1).tolist() == [1, 2] and (r4.values(vc, vs) == [[1.0], [2.0]]).all()
    for b in range(c.B):
        for j in range(n // 64):
            page, kind = c.table[b, j], int(64 * j >= n // 2)
            c.K[0][page], c.K[1][page] = kc[kind], ks[kind]
            c.V[0][page], c.V[1][page] = vc[kind], vs[kind]
    c.tokens(*step(lens))
    first, more = torch.tensor(rows, dtype=torch.float64).T[..., None]
    q = torch.zeros(c.T, c.H, 128)
    q[:, :, 0], q[:, :, 16] = first, more
    c.q, c.scale = q.bfloat16(), float(np.float32(np.log(2)))
    c.upload()
    out, lse = c.attn()
    out, lse = out.double().cpu(), lse.double().cpu()
    bad = ~(torch.isfinite(out) & (out >= 1) & (out <= 2)).flatten(1).all(dim=1)
    assert not bad.any(), [rows[i] for i in bad.nonzero()[:, 0]]
    want = np.log(2) * (first + more) + np.log(n // 2)
    assert ((lse - want).abs() <= 2.0 ** -20 * want).all()
