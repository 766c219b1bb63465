"""The 4-bit cache where numbers are far from ordinary ones: logits past 2^24,
infinite queries, rotations at far positions; and slots that a call is given twice."""
import numpy as np
import pytest
import torch

import paged4_ref as r4
import turns
from indexer_selected_sparse_score_gb300 import binding as sb
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


@pytest.mark.parametrize("G", [8, 16, 32])
def test_infinite_queries(G):
    """All logits -inf: a row of zeros, and nothing gathered; one of +inf: NaN; -inf beside
    finite ones: those alone."""
    lens = [150, 150, 150]
    c = Case(12, lens, D=128, P=64, Hkv=1, G=G).tokens(*step(lens))
    for b in range(3):
        for j in range(150):
            codes = c.K[0][c.table[b, j // 64], 0, j % 64]
            codes[0] = (codes[0] & 0xF0) | (0 if b == 2 and j % 2 else 2)  # value 0 is positive, or zero in every other slot
            c.K[1][c.table[b, j // 64], 0, j % 64, 0] = 0x38
    c.q[0, :, 0], c.q[1, :, 0] = -torch.inf, torch.inf
    c.q[2, :, 0] = -3e38                                     # (-inf times zero is NaN; this is not)
    c.q[2, :, 1:] = c.q[2, :, 1:] * 1e30
    c.upload()
    out, lse = c.attn()
    assert (out[0] == 0).all() and (lse[0] == -torch.inf).all()
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert torch.isfinite(out[2]).all() and torch.isfinite(lse[2]).all()
    w = torch.ones(3, 1, c.max_pages * 64, device=DEV)
    sb.sa_paged4_weights(c.pa, c.d["q"], lse, w, c.ws)
    assert (w[0] == 1).all() and w[1, 0, :150].isnan().all() and (w[1, 0, 150:] == 1).all()


def _turned(a, b, ang):
    return a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)


def _bf16(x):
    return torch.from_numpy(np.asarray(x)).float().bfloat16().double().numpy()


@pytest.mark.parametrize("far,halves", [(2 ** 31 - 1, True), (-2 ** 31, False), (-(2 ** 30) - 7, True)])
def test_append_at_far_positions(far, halves):
    """Keys whose code depends on the last bits of the angle: one value, rotated, lies so near
    the middle of two bf16 neighbours to either side of a code's border that an angle from
    a frequency over 2 pi as a double (2^-56.5 of a turn off a position for a frequency of
    1, 2^-22.8 in radians at 2^31) gives another code.  Base 2^32 and 64 rotated values:
    frequencies 2^-i, exact.  What the call promises, 2^-39 + |r| 2^-61, is below 2^-29.9;
    values within 2^-29 of a rounding's border, by way of fp32 too, are left out."""
    D, dim, each = 128, 64, 800000
    pos = far - np.sign(far) * 977 * np.arange(48)
    ang = turns.angles(pos, 2.0 ** -np.arange(dim // 2.0))
    double = [int(p) * int(2.0 ** 64 / (2 * np.pi)) % (1 << 64) / 2.0 ** 64 * 2 * np.pi for p in pos]
    r = np.random.RandomState(abs(far) % 1000 + halves)
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])  # for a scale of 1
    rows = []
    for i in range(len(pos)):
        a, b = (_bf16(r.choice([-1, 1], each) * 2.0 ** r.uniform(-m, 2, each)) for m in (2, 12))
        y, z, e = _turned(a, b, ang[i, 0])[0], _turned(a, b, double[i])[0], 2.0 ** -29 * (np.abs(a) + np.abs(b))
        # (a border is a bf16 value, and a tie: of two neighbours, the codes differ where it is one)
        lo, hi = np.sort(np.abs([_bf16(y), _bf16(z)]), axis=0)
        rows += [(i, a[j], b[j]) for j in np.nonzero((lo < hi) & (hi < 5.5) & (_bf16(y - e) == _bf16(y + e)))[0]
                 if np.isin(borders, [lo[j], hi[j]]).any()]
    n = len(rows)
    at = np.array([x[0] for x in rows])
    # pair 0 is the one above; pair 7's first value becomes 6, so that the scale of both's block is 1
    first, step_, second = D - dim, (1 if halves else 2), (dim // 2 if halves else 1)
    k = torch.zeros(n, 1, D, dtype=torch.float64)
    k[:, 0, first], k[:, 0, first + second] = torch.tensor([x[1:] for x in rows], dtype=torch.float64).T
    k[:, 0, first + 7 * step_] = torch.from_numpy(6 * np.cos(ang[at, 7])).bfloat16()
    k[:, 0, first + 7 * step_ + second] = torch.from_numpy(-6 * np.sin(ang[at, 7])).bfloat16()

    def quantised(angle):
        x = k.clone().numpy()
        for i in (0, 7):
            u = first + i * step_
            x[:, 0, u], x[:, 0, u + second] = _turned(k[:, 0, u].numpy(), k[:, 0, u + second].numpy(), angle[:, i])
        return r4.quantise(_bf16(x))
    codes, scales = quantised(ang[at])
    other, _ = quantised(np.where(np.arange(dim // 2) == 0, np.array(double)[at][:, None], ang[at]))
    block = slice(first // 2, first // 2 + 8)
    tells = (codes != other)[:, 0, block].any(axis=1)
    assert (scales[:, 0, first // 16] == 0x38).all() and tells.any()
    c = Case(9, [n], D, 64, 1, 1).tokens([0] * n, range(n)).upload()
    rope = sb.RopeArgs(dim, 2.0 ** 32, 1.0, 0, 32.0, 1.0)
    k = k.bfloat16().to(DEV)
    sb.sa_paged4_append(c.pa, k, k, c.ws, rope=rope, halves=halves,
                        rope_pos=torch.from_numpy(pos[at].astype(np.int32)).to(DEV))
    assert sb.sa_check_device_status(c.ws) == sb.SA_OK
    page, slot = c.table[0, np.arange(n) // 64], np.arange(n) % 64
    assert np.array_equal(c.d["Ks"].cpu().numpy()[page, 0, slot][:, first // 16], scales[:, 0, first // 16])
    # (value 0 is the one that was looked at; its pair's other value and pair 7's small one may lie at a border)
    got = c.d["K"].cpu().numpy()[page, 0, slot][:, first // 2] & 15
    assert np.array_equal(got, codes[:, 0, first // 2] & 15), (got != codes[:, 0, first // 2] & 15).sum()


def test_a_slot_given_twice():
    """Codes (in units of eight) and scales are one token's or the other's, perhaps of both in
    one row; nothing else is written."""
    n, D, P = 300, 128, 64
    c = Case(11, [n], D, P, 2, 1).tokens([0] * (2 * n), list(range(n)) * 2).upload()
    k, v = (torch.from_numpy(c.r.standard_normal((2 * n, 2, D)) * 4.0 ** np.repeat([0, 1], n)[:, None, None]).bfloat16()
            for _ in range(2))
    before = [c.d[x].cpu().numpy().copy() for x in ("K", "Ks", "V", "Vs")]
    sb.sa_paged4_append(c.pa, k.to(DEV), v.to(DEV), c.ws)
    assert sb.sa_check_device_status(c.ws) == sb.SA_OK
    page, slot = c.table[0, np.arange(n) // P], np.arange(n) % P
    for i, (x, name) in enumerate(((k, "K"), (k, "Ks"), (v, "V"), (v, "Vs"))):
        want = r4.quantise(x.double().numpy())[i % 2]
        got = c.d[name].cpu().numpy()
        rows = got[page, :, slot]
        unit = (lambda y: y.reshape(n, 2, -1, 4)) if i % 2 == 0 else (lambda y: y[..., None])
        one, other = (unit(rows) == unit(want[:n])).all(axis=-1), (unit(rows) == unit(want[n:])).all(axis=-1)
        assert (one | other).all()
        got[page, :, slot] = before[i][page, :, slot]
        assert np.array_equal(got, before[i])
