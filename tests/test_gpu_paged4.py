"""The 4-bit paged cache on the GPU against float64 definitions
(tests/paged4_ref.py) at the sizes and masks where it can go wrong."""
import numpy as np
import pytest
import torch

import paged4_ref as r4
import paged_ref as ref
from indexer_selected_sparse_score_gb300 import binding as sb

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    """A 4-bit cache on the CPU and the GPU: sequences of given lengths, their pages
    shuffled; every slot past a sequence's last one, and every page that no
    sequence names, holds NaN scales and arbitrary codes."""

    def __init__(self, seed, lens, D=128, P=64, Hkv=2, G=8, extra=3, k_gain=1.0, v_gain=1.0, spread=1.0):
        r = np.random.RandomState(seed)
        self.r = r
        self.B, self.D, self.P, self.Hkv, self.G, self.H = len(lens), D, P, Hkv, G, Hkv * G
        self.lens = list(lens)
        need = [(n + P - 1) // P for n in lens]
        self.max_pages = max(max(need), 1) + 1
        self.total = sum(need) + extra
        perm = r.permutation(self.total)
        self.table = np.full((self.B, self.max_pages), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.k_gain, self.v_gain, self.scale = k_gain, v_gain, float(np.float32(D ** -0.5))
        shape = (self.total, Hkv, P, D)
        self.K = list(r4.quantise(r.standard_normal(shape) * spread))
        self.V = list(r4.quantise(r.standard_normal(shape)))
        used = np.zeros((self.total, P), bool)
        for b, n in enumerate(need):
            for j in range(n):
                used[self.table[b, j], :max(0, min(P, lens[b] - j * P))] = True
        for c in (self.K, self.V):
            c[0].transpose(0, 2, 1, 3)[~used] = 0xA7
            c[1].transpose(0, 2, 1, 3)[~used] = 0x7F

    def tokens(self, seq, pos, spread=1.0):
        self.seq, self.pos, self.T = np.array(seq, np.int32), np.array(pos, np.int32), len(seq)
        self.q = torch.from_numpy(self.r.standard_normal((self.T, self.H, self.D)) * spread).bfloat16()
        return self

    def upload(self):
        def dev(x):
            return (x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))).to(DEV)
        self.d = {n: dev(getattr(self, n)) for n in ("seq", "pos", "table", "q")}
        self.d.update(K=dev(self.K[0]), Ks=dev(self.K[1]), V=dev(self.V[0]), Vs=dev(self.V[1]))
        self.pa = sb.paged4_args(self.d["seq"], self.d["pos"], self.d["table"], self.H, self.Hkv, self.D, self.P, self.total,
                                 self.d["K"], self.d["V"], self.d["Ks"], self.d["Vs"], self.scale, self.k_gain,
                                 self.v_gain)
        self.ws = sb.new_paged4_workspace(self.pa)
        return self

    def valid(self, t):
        return 0 <= self.seq[t] < self.B and 0 <= self.pos[t] < self.max_pages * self.P

    def attn(self, expect=sb.SA_OK):
        out = torch.full((self.T, self.H, self.D), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((self.T, self.H), 7.0, device=DEV)
        sb.sa_paged4_attn(self.pa, self.d["q"], out, self.ws, lse=lse)
        assert sb.sa_check_device_status(self.ws) == expect
        return out, lse

    def rows(self, b, h, n):
        k, ok = r4.rows(self.K, self.table[b], h, n, self.P)
        v, _ = r4.rows(self.V, self.table[b], h, n, self.P)
        return k * self.k_gain, v * self.v_gain, ok

    def check_attn(self, out, lse):
        out, lse = out.cpu().double(), lse.cpu().double()
        seen = {}
        for t in range(self.T):
            if not self.valid(t):
                assert (out[t] == 7).all() and (lse[t] == 7).all()
                continue
            b, n = int(self.seq[t]), int(self.pos[t]) + 1
            for h in range(self.Hkv):
                if (b, h) not in seen:
                    top = 1 + max(int(p) for s, p, u in zip(self.seq, self.pos, range(self.T)) if s == b and self.valid(u))
                    seen[b, h] = self.rows(b, h, top)
                k, v, ok = (x[:n] for x in seen[b, h])
                sl = slice(h * self.G, (h + 1) * self.G)
                o, l, s, eps, mag = r4.attention(self.q[t, sl].double(), k, v, ok, self.scale)
                got, got_l = out[t, sl], lse[t, sl]
                assert torch.equal(got.isnan(), o.isnan()), (t, h)
                assert torch.equal(got_l.isnan(), l.isnan()), (t, h)
                vmax = float(v[ok].abs().nan_to_num(0.0).max()) if ok.any() else 0.0
                bound = r4.out_bound(o, mag, eps, n, vmax)
                bad = ((got - o).abs() > bound) & ~o.isnan()
                assert not bad.any(), (t, h, float(((got - o).abs() / bound)[bad].max()))
                if ok.any():
                    fine = torch.isfinite(l)
                    assert ((got_l - l).abs()[fine] <= r4.lse_bound(l, eps, n)[fine]).all(), (t, h, got_l, l)
                else:
                    assert (got_l == -np.inf).all() and (got == 0).all()


def step(lens):
    return list(range(len(lens))), [n - 1 for n in lens]


# lengths of one slot, ends inside and at the border of a page, a tile and 16 slots
LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1024, 1537]


@pytest.mark.parametrize("D,P,Hkv,G", [(128, 64, 2, 8), (128, 16, 1, 4), (64, 32, 2, 8), (64, 128, 1, 1), (128, 128, 2, 16),
                                       (64, 16, 2, 16), (128, 32, 3, 5), (128, 64, 1, 12), (64, 64, 4, 3), (128, 64, 1, 64),
                                       (64, 16, 1, 24), (128, 16, 2, 17), (128, 128, 1, 128)])
def test_decode(D, P, Hkv, G):
    c = Case(1, LENS, D, P, Hkv, G).tokens(*step(LENS)).upload()
    c.check_attn(*c.attn())


@pytest.mark.parametrize("lens", [[1], [40000], [5, 30000, 1], [17] * 70 + [3000]])
@pytest.mark.parametrize("G", [2, 8, 16, 40])
def test_decode_lengths(lens, G):
    c = Case(2, lens, G=G, Hkv=1 if len(lens) > 10 else 2).tokens(*step(lens)).upload()
    c.check_attn(*c.attn())


@pytest.mark.parametrize("D,P,Hkv,G,new", [(128, 64, 2, 4, 4), (128, 16, 2, 8, 3), (64, 32, 1, 1, 7), (128, 128, 1, 5, 40),
                                           (64, 64, 2, 16, 33), (128, 64, 1, 64, 5), (128, 32, 2, 3, 130), (64, 16, 2, 8, 70)])
def test_several_tokens_of_a_sequence(D, P, Hkv, G, new):
    lens = [new, new + 1, 300, 129 + new]
    seq = np.repeat(range(4), new).tolist()
    pos = np.concatenate([np.arange(n - new, n) for n in lens]).tolist()
    c = Case(3, lens, D, P, Hkv, G).tokens(seq, pos).upload()
    c.check_attn(*c.attn())


def test_tokens_in_any_order():
    lens = [200, 77, 513]
    r = np.random.RandomState(4)
    tok = [(b, p) for b, n in enumerate(lens) for p in r.choice(n, 25, replace=False)]
    r.shuffle(tok)
    tok = tok[:20] + [tok[5], tok[5]] + tok[20:]  # the same token twice
    for G in (1, 4, 8, 32):
        c = Case(5, lens, G=G, Hkv=1).tokens([t[0] for t in tok], [t[1] for t in tok]).upload()
        c.check_attn(*c.attn())


def test_gains_scales_and_spread():
    c = Case(6, [300, 40], k_gain=0.25, v_gain=8.0, spread=6.0).tokens([0, 1], [299, 39], spread=3.0)
    c.scale = -0.05
    c.upload()
    c.check_attn(*c.attn())
    c.scale = 0.0
    c.upload()
    c.check_attn(*c.attn())


def test_queries_of_any_magnitude():
    c = Case(7, [300] * 6, G=4).tokens(range(6), [299] * 6)
    f = torch.tensor([1e-30, 1e-8, 1.0, 1e3, 1e20, 0.0])
    c.q = (c.q.float() * f[:, None, None]).bfloat16()
    c.upload()
    c.check_attn(*c.attn())


def test_rising_logits():
    # every later tile's logits pass the reference
    lens = [2000]
    for G in (8, 64):
        c = Case(8, lens, G=G, Hkv=1)
        c.tokens([0], [1999])
        c.q = torch.ones_like(c.q)
        k = np.repeat((np.arange(2000) // 16 * 0.4)[:, None], 128, axis=1) * 0.1
        codes, scales = r4.quantise(k)
        for j in range(2000):
            c.K[0][c.table[0, j // 64], 0, j % 64] = codes[j]
            c.K[1][c.table[0, j // 64], 0, j % 64] = scales[j]
        c.scale = 1.0
        c.upload()
        c.check_attn(*c.attn())


def test_lost_pages_and_skipped_tokens():
    lens = [700, 260, 64, 500]
    for G in (4, 32):
        c = Case(9, lens, G=G, P=32)
        c.table[0, [0, 5, 21]] = [-1, c.total, 1 << 30]
        c.table[2, :] = -3                                   # a row without keys
        c.tokens([0, 1, -1, 4, 2, 3, 3, 1], [699, 259, 5, 5, 63, -1, c.max_pages * 32, 100]).upload()
        c.check_attn(*c.attn(expect=sb.SA_ERR_DEVICE_DATA))
        assert sb.sa_check_device_status(c.ws) == sb.SA_OK


@pytest.mark.parametrize("G", [2, 8, 33])
def test_nan_rows_stay_in_their_rows(G):
    # a NaN key and a NaN block of values: the tokens before them do not see them
    lens = [150, 150]
    c = Case(10, lens, G=G, Hkv=1, P=64)
    seq, pos = [0] * 12 + [1] * 12, list(range(138, 150)) * 2
    c.tokens(seq, pos)
    c.V[1][c.table[0, 145 // 64], 0, 145 % 64, 3] = 0x7F
    c.V[1][c.table[0, 140 // 64], 0, 140 % 64, 5] = 0xFF
    c.K[1][c.table[1, 143 // 64], 0, 143 % 64, 0] = 0x7F
    c.upload()
    out, lse = c.attn()
    c.check_attn(out, lse)
    out = out.cpu()
    assert not out[:2].isnan().any() and out[7, :, 48:64].isnan().all() and not out[7, :, :48].isnan().any()
    assert out[17:].isnan().all() and not out[12:17].isnan().any()


def test_no_tokens_and_no_lse():
    c = Case(11, [40]).tokens([], [])
    c.q = torch.zeros(0, c.H, c.D, dtype=torch.bfloat16)
    c.upload()
    c.attn()
    c = Case(11, [40]).tokens([0], [39]).upload()
    out = torch.zeros(1, c.H, c.D, dtype=torch.bfloat16, device=DEV)
    sb.sa_paged4_attn(c.pa, c.d["q"], out, c.ws)
    assert torch.equal(out, c.attn()[0])


def test_same_results_again_and_from_a_graph():
    lens = [900, 33, 5000, 2048]
    for G in (8, 16, 48):
        c = Case(12, lens, G=G).tokens(*step(lens)).upload()
        first = c.attn()
        s = torch.cuda.Stream()
        out, lse = (torch.zeros_like(x) for x in first)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            sb.sa_paged4_attn(c.pa, c.d["q"], out, c.ws, lse=lse)
        s.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sb.sa_paged4_attn(c.pa, c.d["q"], out, c.ws, lse=lse)
        # the graph follows what lies in the positions at replay
        c.pos = np.array([n // 2 for n in lens], np.int32)
        c.d["pos"].copy_(torch.from_numpy(c.pos))
        for _ in range(3):
            out.fill_(7)
            g.replay()
        torch.cuda.synchronize()
        c.check_attn(out, lse)


def test_nothing_to_attend():
    """Calls whose every token is skipped leave everything as it was."""
    lens = [100, 200]
    for G, T in ((8, 2), (8, 100), (48, 2), (48, 100)):
        c = Case(13, lens, G=G).tokens([-2 ** 31, 2, 0, 1] * (T // 2), [5, 5, 2 ** 31 - 1, -2 ** 31] * (T // 2)).upload()
        out, lse = c.attn(expect=sb.SA_ERR_DEVICE_DATA)
        assert (out == 7).all() and (lse == 7).all()
        weight = torch.full((c.B, c.Hkv, c.max_pages * c.P), 3.0, device=DEV)
        sb.sa_paged4_weights(c.pa, c.d["q"], lse, weight, c.ws)
        assert sb.sa_check_device_status(c.ws) == sb.SA_ERR_DEVICE_DATA
        assert (weight == 3).all()


# ----------------------------------------------------------------- append ---

def _state(c, ld=None):
    ld = ld or c.max_pages * c.P
    return (torch.full((c.B, c.Hkv, ld), 5.0, device=DEV), torch.full((c.B, c.Hkv, ld), 5, dtype=torch.int32, device=DEV))


def _append(c, k, v, dim, halves, turn=None, records=True, q=True, base=10000.0, **kw):
    rope = sb.RopeArgs(dim, base, 1.0, 0, 32.0, 1.0)
    q_out = torch.full((c.T, c.H, c.D), 7.0, dtype=torch.bfloat16, device=DEV) if q else None
    weight, born = _state(c) if records else (None, None)
    sb.sa_paged4_append(c.pa, k, v, c.ws, q=c.d["q"] if q else None, q_out=q_out, rope=rope, halves=halves,
                        rope_pos=torch.tensor(turn, dtype=torch.int32, device=DEV) if turn is not None else None,
                        weight=weight, born=born, **kw)
    return q_out, weight, born


def _check_append(c, k, v, dim, halves, turn, expect=sb.SA_OK, base=10000.0):
    turn = c.pos if turn is None else np.asarray(turn)
    before = [x.clone() for x in (c.d["K"], c.d["Ks"], c.d["V"], c.d["Vs"])]
    q_out, weight, born = _append(c, k.to(DEV), v.to(DEV), dim, halves, turn, base=base)
    assert sb.sa_check_device_status(c.ws) == expect
    freqs = ref.rope_freqs(dim, base)
    kr, mag = ref.rotate(k.double(), turn, freqs, halves)
    qr, qmag = ref.rotate(c.q.double(), turn, freqs, halves)
    # a rotated value in fp32: the angle to 2^-24 of a half turn, sine and cosine
    # (2 ulp), two products and a sum: 2^-21 of the pair
    err, qerr = 2.0 ** -21 * mag, 2.0 ** -21 * qmag
    if dim:
        err[..., :c.D - dim] = 0
    else:
        err.zero_()
    lo, hi = (kr - err).bfloat16(), (kr + err).bfloat16()
    want = [x.cpu().numpy().copy() for x in before]
    sure = np.zeros(before[1].shape, bool)
    w_want, b_want = _state(c)
    w_want, b_want = w_want.cpu(), b_want.cpu()
    ok = [t for t in range(c.T) if c.valid(t)]
    for t in ok:
        b, p = int(c.seq[t]), int(c.pos[t])
        w_want[b, :, p], b_want[b, :, p] = 0, int(turn[t])
        page = c.table[b, p // c.P]
        if not 0 <= page < c.total:
            continue
        want[0][page, :, p % c.P], want[1][page, :, p % c.P] = r4.quantise(lo[t].double().numpy() / c.k_gain)
        want[2][page, :, p % c.P], want[3][page, :, p % c.P] = r4.quantise(v[t].double().numpy() / c.v_gain)
        same = (lo[t] == hi[t]) | (lo[t].isnan() & hi[t].isnan())
        sure[page, :, p % c.P] = same.reshape(c.Hkv, -1, 16).all(dim=-1).numpy()
    got = [x.cpu().numpy() for x in (c.d["K"], c.d["Ks"], c.d["V"], c.d["Vs"])]
    assert np.array_equal(got[2], want[2]) and np.array_equal(got[3], want[3])
    # keys: blocks whose rotated values round one way only
    touched = np.zeros(before[1].shape, bool)
    for t in ok:
        page = c.table[int(c.seq[t]), int(c.pos[t]) // c.P]
        if 0 <= page < c.total:
            touched[page, :, int(c.pos[t]) % c.P] = True
    # (a value is unsure for 2 err of a step of at least 2^-8 of it: 2^-12 mag / |y|,
    # mag / |y| about 4 on average with values near 0; 16 values a block: 2 %, and as
    # much again for the few blocks here)
    assert sure[touched].mean() > 0.9 if touched.any() else True
    same_s = got[1] == want[1]
    same_c = (got[0] == want[0]).reshape(same_s.shape + (8,)).all(axis=-1)
    assert (same_s & same_c)[sure | ~touched].all()
    # the others: a neighbouring value
    unsure = touched & ~sure
    if unsure.any():
        x, y = r4.values(got[0], got[1]), r4.values(want[0], want[1])
        d = np.abs(x - y).reshape(unsure.shape + (16,))[unsure]
        s = r4.e4m3_value(want[1])[unsure][:, None]
        assert (d <= 2.5 * s).all()
    for t in range(c.T):
        if t in ok:
            e = qerr[t] + 2.0 ** -8 * (qr[t].abs() + qerr[t])
            assert ((q_out[t].cpu().double() - qr[t]).abs() <= e).all()
        else:
            assert (q_out[t] == 7).all()
    assert torch.equal(weight.cpu(), w_want) and torch.equal(born.cpu(), b_want)


@pytest.mark.parametrize("D,P,Hkv,G,dim,halves", [(128, 64, 2, 4, 128, True), (128, 64, 8, 8, 64, False),
                                                  (64, 16, 1, 3, 32, True), (64, 128, 3, 1, 64, True),
                                                  (128, 32, 2, 2, 96, True), (128, 32, 2, 2, 96, False),
                                                  (128, 16, 1, 20, 0, True), (128, 64, 40, 1, 32, False)])
def test_append(D, P, Hkv, G, dim, halves):
    lens = [70, 1, 200]
    seq, pos = [0, 2, 1, 2, 0, 2], [69, 199, 0, 64, 5, 130]
    c = Case(20, lens, D, P, Hkv, G, k_gain=0.5, v_gain=4.0).tokens(seq, pos).upload()
    k = torch.from_numpy(c.r.standard_normal((6, Hkv, D))).bfloat16()
    v = torch.from_numpy(c.r.standard_normal((6, Hkv, D))).bfloat16()
    _check_append(c, k, v, dim, halves, None)
    _check_append(c, k, v, dim, halves, [100069, 0, 2000000000, 7, -3, 64])


@pytest.mark.parametrize("D,dim,halves,far", [(128, 128, True, 0), (128, 64, False, 100000), (64, 64, True, 3)])
def test_append_rounds_keys_as_64_bits_do(D, dim, halves, far):
    """Every code and scale of many rotated keys.  A key is within 2^-40 of its pair's
    magnitude (2^-9 of the rounding's step to bf16, by way of fp32, 2^-15 of fp32's), so of
    a million one in 2^-31 2^20, or none, is expected to be rounded another way; the 64-bit
    angle is exact to 2^-52 of 10^5."""
    n, Hkv = 1000, 8
    c = Case(24, [n], D, 64, Hkv, 1).tokens([0] * n, range(n)).upload()
    k, v = (torch.from_numpy(c.r.standard_normal((n, Hkv, D))).bfloat16() for _ in range(2))
    turn = np.arange(n) * 7 + far
    _append(c, k.to(DEV), v.to(DEV), dim, halves, turn)
    kr, _ = ref.rotate(k.double(), turn, ref.rope_freqs(dim, 10000.0), halves)
    for got, x in zip((("K", "Ks"), ("V", "Vs")), (kr, v.double())):
        codes, scales = r4.quantise(x.float().bfloat16().double().numpy())
        page = c.table[0, np.arange(n) // 64]
        assert np.array_equal(c.d[got[0]].cpu().numpy()[page, :, np.arange(n) % 64], codes)
        assert np.array_equal(c.d[got[1]].cpu().numpy()[page, :, np.arange(n) % 64], scales)


def test_append_a_ragged_prompt():
    lens = [333, 1, 500, 64]
    seq = np.repeat(range(4), lens).tolist()
    pos = np.concatenate([np.arange(n) for n in lens]).tolist()
    c = Case(21, lens, Hkv=2, G=2).tokens(seq, pos).upload()
    k = torch.from_numpy(c.r.standard_normal((c.T, 2, 128))).bfloat16()
    v = torch.from_numpy(c.r.standard_normal((c.T, 2, 128))).bfloat16()
    _check_append(c, k, v, 128, True, None)


def test_append_values_at_borders():
    # every multiple of a quarter step and its bf16 neighbours, over scales of all
    # exponents; zeros, infinities, NaN, values beyond both ends of the scales
    r = np.random.RandomState(22)
    rows = []
    for e in range(-14, 12):
        for m in range(8):
            s = (1 + m / 8) * 2.0 ** e
            mids = np.concatenate([(r4.E2M1[1:] + r4.E2M1[:-1]) / 2, r4.E2M1, [0.125, 4.5]]) * s
            x = torch.from_numpy(mids).bfloat16()
            near = torch.cat([x, (x.view(torch.int16) + 1).view(torch.bfloat16), (x.view(torch.int16) - 1).clamp(min=0).view(
                torch.bfloat16)])
            near = near[torch.from_numpy(r.permutation(len(near)))]
            sign = torch.from_numpy(r.choice([-1.0, 1.0], len(near))).bfloat16()
            rows.append(torch.cat([near * sign, x[:-1], torch.tensor([6 * s, -6 * s, 6.1 * s]).bfloat16()])[:64])
    rows = torch.stack([x if len(x) == 64 else torch.cat([x, torch.zeros(64 - len(x)).bfloat16()]) for x in rows])
    rows = rows.reshape(-1, 1, 64)
    special = torch.zeros(8, 1, 64).bfloat16()
    special[0, 0, 3] = float("inf")
    special[1, 0, 20] = float("nan")
    special[2] = 3e38
    special[3] = -0.0
    special[4] = 1e-38
    special[5, 0, :16] = torch.arange(16) * 2.0 ** -11
    special[6, 0, 5] = -float("inf")
    special[6, 0, 6] = 100.0
    v = torch.cat([rows, special])
    T = len(v)
    c = Case(22, [T], D=64, P=64, Hkv=1, G=1).tokens([0] * T, list(range(T))).upload()
    _check_append(c, v, v.clone(), 0, False, None)


def test_append_slices_skips_and_lost_pages():
    lens = [100, 50]
    c = Case(23, lens, Hkv=2, G=2, P=32)
    c.table[1, 0] = -1
    c.tokens([0, 5, 1, 0, -1, 1], [99, 3, 3, -2, 0, 40]).upload()
    qkv = torch.from_numpy(c.r.standard_normal((6, 10 * 128 + 8))).bfloat16().to(DEV)
    k, v = qkv[:, 512:768].view(6, 2, 128), qkv[:, 768:1024].view(6, 2, 128)
    _check_append(c, k.cpu(), v.cpu(), 64, True, None, expect=sb.SA_ERR_DEVICE_DATA)
    before = c.d["K"].clone()
    _append(c, k, v, 64, True, records=False, q=False)
    assert torch.equal(before, c.d["K"])
    assert sb.sa_check_device_status(c.ws) == sb.SA_ERR_DEVICE_DATA


@pytest.mark.parametrize("D,P", [(128, 64), (64, 16)])
def test_read(D, P):
    lens = [100, 7]
    c = Case(24, lens, D, P, k_gain=0.5, v_gain=4.0).tokens([0, 1, 0, 3, 0], [99, 6, 0, 1, 50])
    c.table[0, 50 // P] = -1 if P == 16 else c.table[0, 50 // P]
    c.upload()
    ko, vo = (torch.full((5, c.Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sb.sa_paged4_read(c.pa, ko, vo, c.ws)
    assert sb.sa_check_device_status(c.ws) == sb.SA_ERR_DEVICE_DATA
    for t in range(5):
        for h in range(c.Hkv):
            page = c.table[c.seq[t], c.pos[t] // P] if t != 3 else -1
            if page < 0:
                assert (ko[t] == 7).all() and (vo[t] == 7).all()
                continue
            for out, cache, gain in ((ko, c.K, 0.5), (vo, c.V, 4.0)):
                want = r4.values(cache[0][page, h, c.pos[t] % P], cache[1][page, h, c.pos[t] % P]) * gain
                assert np.array_equal(out[t, h].cpu().double().numpy(), want)  # (six significant bits)
    k2 = torch.zeros_like(ko)
    sb.sa_paged4_read(c.pa, k2, None, c.ws)
    v2 = torch.full_like(vo, 7.0)
    sb.sa_paged4_read(c.pa, None, v2, c.ws)
    assert torch.equal(k2[0], ko[0]) and torch.equal(v2, vo)


# ---------------------------------------------------------------- weights ---

def _check_weights(c, expect=sb.SA_OK, lse=None):
    if lse is None:
        _, lse = c.attn(expect)
    w0 = torch.rand(c.B, c.Hkv, c.max_pages * c.P + 5, generator=torch.Generator().manual_seed(1))
    w = w0.to(DEV)
    sb.sa_paged4_weights(c.pa, c.d["q"], lse, w, c.ws)
    assert sb.sa_check_device_status(c.ws) == expect
    want, mag = w0.double(), torch.zeros_like(w0, dtype=torch.float64)
    terms = torch.zeros_like(mag)
    l64 = lse.cpu().double()
    for t in range(c.T):
        if not c.valid(t):
            continue
        b, n = int(c.seq[t]), int(c.pos[t]) + 1
        for h in range(c.Hkv):
            k, _, ok = c.rows(b, h, n)
            sl = slice(h * c.G, (h + 1) * c.G)
            _, _, s, eps, _ = r4.attention(c.q[t, sl].double(), k, k, ok, c.scale)
            if s is None:
                continue
            p = torch.exp(s - l64[t, sl, None]).nan_to_num(0.0) if (l64[t, sl] == -np.inf).any() else torch.exp(s - l64[t, sl, None])
            j = torch.arange(n)[ok]
            want[b, h, j] += p.sum(dim=0)
            # logits off by eps, the factors' roundings, the exponential
            mag[b, h, j] += (p * (2 * eps + 2.0 ** -20 + (s.abs() + l64[t, sl, None].abs()) * 2.0 ** -21)).sum(dim=0)
            terms[b, h, j] += c.G
    bound = mag + (terms + 8) * 2.0 ** -23 * want.abs() + 1e-35
    got = w.cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    bad = ((got - want).abs() > bound) & ~want.isnan()
    assert not bad.any(), float(((got - want).abs() / bound)[bad].max())
    assert torch.equal(w.cpu()[..., c.max_pages * c.P:], w0[..., c.max_pages * c.P:])
    return w


@pytest.mark.parametrize("D,P,Hkv,G", [(128, 64, 2, 8), (64, 16, 1, 4), (128, 128, 1, 16), (64, 32, 2, 3), (128, 32, 1, 40),
                                       (128, 64, 1, 128)])
def test_weights_decode(D, P, Hkv, G):
    c = Case(30, LENS, D, P, Hkv, G).tokens(*step(LENS)).upload()
    _check_weights(c)


@pytest.mark.parametrize("D,P,Hkv,G,new", [(128, 64, 2, 4, 4), (64, 32, 1, 1, 7), (128, 128, 1, 5, 40), (64, 64, 2, 16, 33),
                                           (128, 32, 2, 3, 300), (64, 16, 2, 8, 270)])
def test_weights_of_several_tokens(D, P, Hkv, G, new):
    lens = [new, new + 1, 300 + new, 129 + new]
    seq = np.repeat(range(4), new).tolist()
    pos = np.concatenate([np.arange(n - new, n) for n in lens]).tolist()
    c = Case(31, lens, D, P, Hkv, G).tokens(seq, pos).upload()
    w = _check_weights(c)
    assert torch.equal(w, _check_weights(c))  # one order


def test_weights_of_tokens_in_any_order_and_lost_ones():
    lens = [200, 77, 513]
    r = np.random.RandomState(32)
    tok = [(b, p) for b, n in enumerate(lens) for p in r.choice(n, 25, replace=False)] + [(-1, 4), (3, 4), (1, -1), (0, 1 << 20)]
    r.shuffle(tok)
    c = Case(32, lens, G=4, Hkv=2)
    c.table[2, 3] = -1
    c.tokens([t[0] for t in tok], [t[1] for t in tok]).upload()
    _check_weights(c, expect=sb.SA_ERR_DEVICE_DATA)


def test_weights_sum_to_the_heads():
    # what the slots gather in a step is one per query head
    c = Case(33, [900, 31], G=8).tokens([0, 1], [899, 30]).upload()
    _, lse = c.attn()
    w = torch.zeros(2, c.Hkv, c.max_pages * c.P, device=DEV)
    sb.sa_paged4_weights(c.pa, c.d["q"], lse, w, c.ws)
    assert ((w.double().sum(-1) - 8).abs() < 8 * 900 * 2.0 ** -20).all()
    # a row whose lse is -inf adds nothing
    w2 = w.clone()
    sb.sa_paged4_weights(c.pa, c.d["q"], torch.full_like(lse, -float("inf")), w2, c.ws)
    assert torch.equal(w, w2)


def test_weights_nan_key():
    c = Case(34, [40], G=2, Hkv=1).tokens([0, 0], [20, 39])
    c.K[1][c.table[0, 0], 0, 30, 0] = 0x7F
    c.upload()
    lse = torch.full((2, 2), 3.0, device=DEV)
    w = _check_weights(c, lse=lse)
    assert w[0, 0, 30].isnan() and not w[0, 0, :30].isnan().any()


# ------------------------------------------------------------------ evict ---

def _check_evict(c, length, newest, budget, recent, weight, born, expect=sb.SA_OK):
    dev = lambda x, t: torch.tensor(np.asarray(x), dtype=t, device=DEV)  # noqa: E731
    w, bn = dev(weight, torch.float32), dev(born, torch.int32)
    wo, bo = torch.full_like(w, -1.0), torch.full_like(bn, -1)
    lo = torch.full((c.B,), -1, dtype=torch.int32, device=DEV)
    sb.sa_paged4_evict(c.pa, dev(length, torch.int32), dev(newest, torch.int32), budget, recent, w, bn, wo, bo, lo, c.ws)
    assert sb.sa_check_device_status(c.ws) == expect
    caches = [c.K[0].copy(), c.K[1].copy(), c.V[0].copy(), c.V[1].copy()]
    weight, born = w.cpu().numpy(), bn.cpu().numpy()
    w_want, b_want = np.full(weight.shape, -1.0, np.float32), np.full(born.shape, -1, np.int32)
    for b in range(c.B):
        n = int(length[b]) if 0 <= length[b] <= c.max_pages * c.P else 0
        assert int(lo[b]) == min(n, budget)
        for h in range(c.Hkv):
            src = r4.evict(n, newest[b], budget, recent, weight[b, h], born[b, h])
            for j, m in enumerate(src):
                w_want[b, h, j], b_want[b, h, j] = weight[b, h, m], born[b, h, m]
                pd, ps = c.table[b, j // c.P], c.table[b, m // c.P]
                if m != j and 0 <= pd < c.total and 0 <= ps < c.total:
                    for x in caches:
                        x[pd, h, j % c.P] = x[ps, h, m % c.P]
    assert np.array_equal(wo.cpu().numpy(), w_want, equal_nan=True) and np.array_equal(bo.cpu().numpy(), b_want)
    for x, name in zip(caches, ("K", "Ks", "V", "Vs")):
        assert np.array_equal(c.d[name].cpu().numpy(), x), name


def _records(c, r, lens, ties=False):
    ld = c.max_pages * c.P
    w = np.exp(2 * r.standard_normal((c.B, c.Hkv, ld))).astype(np.float32)
    if ties:
        w = np.round(w)  # many equal ones, zeros among them
    born = np.stack([[r.permutation(ld) for _ in range(c.Hkv)] for _ in range(c.B)]).astype(np.int32)
    return w, born


@pytest.mark.parametrize("D,P,Hkv", [(128, 64, 2), (64, 16, 3), (128, 128, 1), (64, 32, 8)])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 10), (100, 100), (257, 0), (3000, 5)])
def test_evict(D, P, Hkv, budget, recent):
    lens = [0, 1, 64, 65, 300, 999, 100, 101]
    r = np.random.RandomState(40)
    for ties in (False, True):
        c = Case(40, lens, D, P, Hkv, 1).tokens([], [])
        c.q = torch.zeros(0, c.H, D, dtype=torch.bfloat16)
        c.upload()
        w, born = _records(c, r, lens, ties)
        _check_evict(c, lens, [n - 1 for n in lens], budget, recent, w, born)


@pytest.mark.parametrize("n,budget", [(20000, 2048), (20000, 15000), (60000, 300), (33333, 33332)])
def test_evict_long(n, budget):
    c = Case(41, [n], P=128, Hkv=1, G=1).tokens([], [])
    c.q = torch.zeros(0, c.H, c.D, dtype=torch.bfloat16)
    c.upload()
    w, born = _records(c, np.random.RandomState(41), [n])
    _check_evict(c, [n], [n - 1], budget, 128, w, born)


@pytest.mark.parametrize("B,Hkv,P,wide", [(40, 4, 64, 0), (10, 4, 128, 0), (5, 4, 32, 0), (19, 8, 16, 0), (1, 1, 64, 0),
                                          (10, 8, 128, 300), (10, 8, 128, 500), (20, 8, 128, 100), (2, 2, 16, 400)])
def test_evict_few_and_many_rows(B, Hkv, P, wide):
    """Rows of one CTA of either size, and of two, four and eight; tables wider than they
    need to be."""
    lens = [1100 + 37 * i % 1500 for i in range(B)]
    r = np.random.RandomState(43)
    for ties in (False, True):
        c = Case(43, lens, 64, P, Hkv, 1)
        c.table = np.concatenate([c.table, np.full((B, wide), -1, np.int32)], axis=1)
        c.max_pages = c.table.shape[1]
        c.tokens([], [])
        c.q = torch.zeros(0, c.H, 64, dtype=torch.bfloat16)
        c.upload()
        w, born = _records(c, r, lens, ties)
        _check_evict(c, lens, [n - 1 for n in lens], 1000, 100, w, born)


@pytest.mark.parametrize("n", [33, 5000, 33000])
def test_evict_from_a_wide_table(n):
    """A table whose rows could be longer than what eight CTAs hold."""
    c = Case(44, [n], 64, P=128, Hkv=1, G=1)
    c.table = np.concatenate([c.table, np.full((1, 3200), -1, np.int32)], axis=1)
    c.max_pages = c.table.shape[1]
    c.tokens([], [])
    c.q = torch.zeros(0, c.H, c.D, dtype=torch.bfloat16)
    c.upload()
    w, born = _records(c, np.random.RandomState(44), [n], ties=True)
    _check_evict(c, [n], [n - 1], max(n // 3, 1), n // 10, w, born)


def test_evict_special_weights_and_lengths():
    lens = [200, 200, 200, 200, 200]
    c = Case(42, lens, P=32, Hkv=2, G=1)
    c.table[3, 1] = -1
    c.tokens([], [])
    c.q = torch.zeros(0, c.H, c.D, dtype=torch.bfloat16)
    c.upload()
    w, born = _records(c, np.random.RandomState(42), lens)
    w[0, 0, 150:160] = np.nan
    w[0, 1, 10:190] = 0.0
    w[0, 1, 20:30] = -0.0
    w[1, 0, 100:] = np.inf
    w[1, 1, :] = 3.0
    w[2, 0, ::2] = 1e-40          # subnormal
    w[2, 1, ::3] = -1.0
    _check_evict(c, [200, 200, 200, 200, c.max_pages * 32 + 1], [199, 250, -5, 199, 3], 50, 20, w, born,
                 expect=sb.SA_ERR_DEVICE_DATA)
    _check_evict_len(c, [-4, 200, 200, 200, 200], w, born)


def _check_evict_len(c, length, w, born):
    dev = lambda x, t: torch.tensor(np.asarray(x), dtype=t, device=DEV)  # noqa: E731
    lo = torch.full((c.B,), -1, dtype=torch.int32, device=DEV)
    wd, bd = dev(w, torch.float32), dev(born, torch.int32)
    sb.sa_paged4_evict(c.pa, dev(length, torch.int32), dev([199] * c.B, torch.int32), 300, 20, wd, bd, torch.zeros_like(wd),
                       torch.zeros_like(bd), lo, c.ws)
    assert sb.sa_check_device_status(c.ws) == sb.SA_ERR_DEVICE_DATA
    assert lo.tolist() == [0, 200, 200, 200, 200]


# --------------------------------------------------------------- together ---

def test_a_loop_that_decodes_within_a_budget():
    """Prompt, weights, eviction, and decode steps whose slots fall behind their
    positions: attention and records against a float64 walk over the same cache."""
    budget, recent, H, Hkv, D, P, B = 96, 16, 8, 2, 128, 32, 3
    r = np.random.RandomState(50)
    lens = [150, 97, 40]
    c = Case(50, [256] * B, D, P, Hkv, H // Hkv).tokens([], [])
    ld = c.max_pages * P
    weight, born = (torch.zeros(B, Hkv, ld, device=DEV), torch.zeros(B, Hkv, ld, dtype=torch.int32, device=DEV))
    rope = sb.RopeArgs(64, 10000.0, 1.0, 0, 32.0, 1.0)
    slots, position = list(lens), list(lens)

    def call(seq, pos, turn):
        c.seq, c.pos, c.T = np.array(seq, np.int32), np.array(pos, np.int32), len(seq)
        x = torch.from_numpy(r.standard_normal((c.T, H + 2 * Hkv, D))).bfloat16().to(DEV)
        d = {k: v for k, v in c.d.items()} if hasattr(c, "d") else None
        c.q = x[:, :H].contiguous().cpu()
        if d is None:
            c.upload()
        else:
            c.d.update(seq=torch.from_numpy(c.seq).to(DEV), pos=torch.from_numpy(c.pos).to(DEV))
            c.pa = sb.paged4_args(c.d["seq"], c.d["pos"], c.d["table"], c.H, Hkv, D, P, c.total, c.d["K"], c.d["V"],
                                  c.d["Ks"], c.d["Vs"], c.scale)
            c.ws = sb.new_paged4_workspace(c.pa)
        q = torch.empty(c.T, H, D, dtype=torch.bfloat16, device=DEV)
        sb.sa_paged4_append(c.pa, x[:, H:H + Hkv], x[:, H + Hkv:], c.ws, q=x[:, :H], q_out=q, rope=rope, halves=True,
                            rope_pos=torch.tensor(turn, dtype=torch.int32, device=DEV), weight=weight, born=born)
        c.q, c.d["q"] = q.cpu(), q
        c.K = [c.d["K"].cpu().numpy(), c.d["Ks"].cpu().numpy()]
        c.V = [c.d["V"].cpu().numpy(), c.d["Vs"].cpu().numpy()]
        out, lse = c.attn()
        c.check_attn(out, lse)
        before = weight.cpu().double()
        sb.sa_paged4_weights(c.pa, q, lse, weight, c.ws)
        gained = (weight.cpu().double() - before).sum(dim=(0, 2))
        assert ((gained - c.T * c.G).abs() < 1e-3 * c.T * c.G).all()

    call(np.repeat(range(B), lens), np.concatenate([np.arange(n) for n in lens]),
         np.concatenate([np.arange(n) for n in lens]))
    for _ in range(4):
        wo, bo = torch.zeros_like(weight), torch.zeros_like(born)
        length = torch.tensor(slots, dtype=torch.int32, device=DEV)
        left = torch.empty_like(length)
        sb.sa_paged4_evict(c.pa, length, torch.tensor(position, dtype=torch.int32, device=DEV) - 1, budget, recent, weight,
                           born, wo, bo, left, c.ws)
        slots = left.tolist()
        weight, born = wo, bo
        for b in range(B):
            assert slots[b] == min(budget, lens[b]) or slots[b] <= budget
            for h in range(Hkv):
                have = set(born[b, h, :slots[b]].tolist())
                assert len(have) == slots[b] and set(range(position[b] - min(recent, position[b]), position[b])) <= have
        call(range(B), slots, position)
        slots, position = [s + 1 for s in slots], [p + 1 for p in position]
    assert slots == [97, 97, 44]


class Step:
    """A decode step over a full cache: append, attention, slot weights, eviction."""

    def __init__(self, seed, G, lens):
        self.c = c = Case(seed, [n + 1 for n in lens], G=G, Hkv=2).tokens(range(len(lens)), lens).upload()
        r = np.random.RandomState(seed)
        dev = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
        self.x = torch.from_numpy(r.standard_normal((c.T, c.H + 2 * c.Hkv, c.D))).bfloat16().to(DEV)
        ld = c.max_pages * c.P
        self.turn = dev(np.array(lens, np.int32) + 1000)
        self.weight = dev(np.exp(r.standard_normal((c.B, c.Hkv, ld))).astype(np.float32))
        self.born = dev(np.tile(np.arange(ld, dtype=np.int32) + 1000, (c.B, c.Hkv, 1)))
        self.length = dev(np.array(lens, np.int32) + 1)
        self.rope = sb.RopeArgs(64, 10000.0, 1.0, 0, 32.0, 1.0)
        self.state = dict(K=c.d["K"], Ks=c.d["Ks"], V=c.d["V"], Vs=c.d["Vs"], weight=self.weight, born=self.born)
        self.out = dict(q=torch.zeros(c.T, c.H, c.D, dtype=torch.bfloat16, device=DEV),
                        out=torch.zeros(c.T, c.H, c.D, dtype=torch.bfloat16, device=DEV),
                        lse=torch.zeros(c.T, c.H, device=DEV), wo=torch.zeros_like(self.weight),
                        bo=torch.zeros_like(self.born), lo=torch.zeros_like(self.length))
        self.before = {k: v.clone() for k, v in self.state.items()}

    def run(self):
        c, o = self.c, self.out
        x, H, Hkv = self.x, c.H, c.Hkv
        sb.sa_paged4_append(c.pa, x[:, H:H + Hkv], x[:, H + Hkv:], c.ws, q=x[:, :H], q_out=o["q"], rope=self.rope,
                            halves=True, rope_pos=self.turn, weight=self.weight, born=self.born)
        sb.sa_paged4_attn(c.pa, o["q"], o["out"], c.ws, lse=o["lse"])
        sb.sa_paged4_weights(c.pa, o["q"], o["lse"], self.weight, c.ws)
        sb.sa_paged4_evict(c.pa, self.length, self.turn, 200, 40, self.weight, self.born, o["wo"], o["bo"], o["lo"], c.ws)

    def reset(self):
        for k, v in self.state.items():
            v.copy_(self.before[k])
        for v in self.out.values():
            v.zero_()

    def result(self):
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in list(self.state.items()) + list(self.out.items())}


def _same(a, b):
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


@pytest.mark.parametrize("G", [8, 48])
def test_a_step_from_a_graph_and_on_another_stream(G):
    s = Step(60, G, [300, 17, 1000, 250])
    s.run()
    want = s.result()
    assert s.out["lo"].tolist() == [200, 18, 200, 200]
    s.reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    _same(s.result(), want)
    s.reset()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for _ in range(3):
        s.reset()
        g.replay()
        _same(s.result(), want)
    assert sb.sa_check_device_status(s.c.ws) == sb.SA_OK


@pytest.mark.parametrize("G", [8, 48])
def test_steps_at_once(G):
    """Two steps with caches and workspaces of their own, on two streams at once, eagerly and
    from graphs."""
    steps = [Step(61, G, [3000, 17, 1000, 250]), Step(62, G, [64, 5000, 900])]
    want = []
    for s in steps:
        s.run()
        want.append(s.result())
    streams = [torch.cuda.Stream() for _ in steps]
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for use_graphs in (False, True):
        for _ in range(5):
            for s in steps:
                s.reset()
            torch.cuda.synchronize()
            for s, g, stream in zip(steps, graphs, streams):
                with torch.cuda.stream(stream):
                    g.replay() if use_graphs else s.run()
            for s, w in zip(steps, want):
                _same(s.result(), w)


@pytest.mark.parametrize("G", [4, 40])
def test_rows_past_four_gigabytes(G):
    """Pages whose bytes lie past 32 bits of offset: written, read, attended, weighed, moved."""
    n_pages, Hkv, P, D, lens = 140000, 8, 64, 128, [130, 70]
    H, B = Hkv * G, len(lens)
    r = np.random.RandomState(70)
    cache = [torch.empty(n_pages, Hkv, P, w, dtype=torch.uint8, device=DEV) for w in (D // 2, D // 2, D // 16, D // 16)]
    table = torch.tensor([[n_pages - 1, 139000, 138321], [0, 132000, -1]], dtype=torch.int32, device=DEV)
    rows = torch.from_numpy(r.standard_normal((sum(lens), 2 * Hkv, D))).bfloat16().to(DEV)
    seq = torch.from_numpy(np.repeat(np.arange(B), lens).astype(np.int32)).to(DEV)
    pos = torch.from_numpy(np.concatenate([np.arange(n) for n in lens]).astype(np.int32)).to(DEV)
    args = lambda s, p: sb.paged4_args(s, p, table, H, Hkv, D, P, n_pages, *cache, D ** -0.5)  # noqa: E731
    pa = args(seq, pos)
    ws = sb.new_paged4_workspace(pa)
    weight, born = torch.zeros(B, Hkv, 3 * P, device=DEV), torch.zeros(B, Hkv, 3 * P, dtype=torch.int32, device=DEV)
    sb.sa_paged4_append(pa, rows[:, :Hkv], rows[:, Hkv:], ws, weight=weight, born=born)

    def read():
        k, v = (torch.zeros(sum(lens), Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        sb.sa_paged4_read(pa, k, v, ws)
        return k, v
    k, v = read()
    # (a code is half a step of up to 1 of 6 scales away, a scale 2^-4 of itself)
    amax = rows.float().unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 16).flatten(-2)
    assert ((torch.cat([k, v], 1).float() - rows.float()).abs() <= amax * (1 / 6 + 2 ** -3)).all()
    last_seq, last_pos = torch.arange(B, dtype=torch.int32, device=DEV), torch.tensor(lens, dtype=torch.int32, device=DEV) - 1
    last = args(last_seq, last_pos)
    q = torch.from_numpy(r.standard_normal((B, H, D))).bfloat16().to(DEV)
    out, lse = torch.zeros_like(q), torch.zeros(B, H, device=DEV)
    last_ws = sb.new_paged4_workspace(last)
    sb.sa_paged4_attn(last, q, out, last_ws, lse=lse)
    sb.sa_paged4_weights(last, q, lse, weight, last_ws)
    at = np.cumsum([0] + lens)
    for b in range(B):
        for h in range(Hkv):
            kk, vv = (x[at[b]:at[b + 1], h].double().cpu() for x in (k, v))
            o, l, s, eps, mag = r4.attention(q[b, h * G:(h + 1) * G].double().cpu(), kk, vv, torch.ones(lens[b], dtype=torch.bool),
                                             D ** -0.5)
            sl = slice(h * G, (h + 1) * G)
            assert ((out[b, sl].double().cpu() - o).abs() <= r4.out_bound(o, mag, eps, lens[b], float(vv.abs().max()))).all()
            assert ((lse[b, sl].double().cpu() - l).abs() <= r4.lse_bound(l, eps, lens[b])).all()
            w = torch.softmax(s, -1).sum(0)
            # weights: logits and lse off by eps and the bound above, sums of G terms
            off = 2 * eps + float(r4.lse_bound(l, eps, lens[b]).max()) + 2.0 ** -20 + G * 2.0 ** -23
            assert ((weight[b, h, :lens[b]].double().cpu() - w).abs() <= w * off * 1.01).all()
    wo, bo = torch.zeros_like(weight), torch.zeros_like(born)
    left = torch.zeros(B, dtype=torch.int32, device=DEV)
    sb.sa_paged4_evict(pa, torch.tensor(lens, dtype=torch.int32, device=DEV), torch.tensor(lens, dtype=torch.int32, device=DEV) - 1,
                       60, 10, weight, born, wo, bo, left, ws)
    assert left.tolist() == [60, 60]
    k2, v2 = read()
    for b in range(B):
        for h in range(Hkv):
            src = r4.evict(lens[b], lens[b] - 1, 60, 10, weight[b, h].cpu().numpy(), born[b, h].cpu().numpy())
            src = torch.tensor(src, device=DEV)
            assert torch.equal(k2[at[b]:at[b] + 60, h], k[at[b] + src, h]) and torch.equal(v2[at[b]:at[b] + 60, h], v[at[b] + src, h])
            assert torch.equal(wo[b, h, :60], weight[b, h, src])
    assert sb.sa_check_device_status(ws) == sb.SA_OK and sb.sa_check_device_status(last_ws) == sb.SA_OK
