"""The paged-cache kernels against float64 definitions (tests/paged_ref.py) at
the sizes and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from indexer_selected_sparse_score_gb300 import binding as sb

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    """A paged cache on the CPU and the GPU: sequences of given lengths, their
    pages shuffled; every position past a sequence's last one, and every page no
    sequence names, holds NaN."""

    def __init__(self, seed, lens, D=128, P=64, Hkv=2, G=8, shared=0, extra=3, poison=True):
        r = np.random.RandomState(seed)
        g = torch.Generator().manual_seed(seed)
        self.B, self.D, self.P, self.Hkv, self.G, self.H = len(lens), D, P, Hkv, G, Hkv * G
        self.lens, self.shared, self.g = list(lens), shared, g
        need = [(n + P - 1) // P for n in lens]
        self.max_pages = max(max(need), 1)
        total = shared + sum(max(n - shared, 0) for n in need) + extra
        perm = r.permutation(total)
        self.table = torch.full((self.B, self.max_pages), -7, dtype=torch.int32)
        at = shared
        self.K = torch.randn(total, Hkv, P, D, generator=g).bfloat16()
        self.V = torch.randn(total, Hkv, P, D, generator=g).bfloat16()
        used = torch.zeros(total, P, dtype=torch.bool)
        for b, n in enumerate(need):
            for j in range(n):
                if j < shared:
                    page = perm[j]
                else:
                    page = perm[at]
                    at += 1
                self.table[b, j] = int(page)
                used[page, :max(0, min(P, lens[b] - j * P))] = True
        if poison:
            self.K.transpose(1, 2)[~used] = float("nan")
            self.V.transpose(1, 2)[~used] = float("nan")
        self.total = total
        self.scale = D ** -0.5

    def tokens(self, seq, pos):
        self.seq, self.pos = torch.tensor(seq, dtype=torch.int32), torch.tensor(pos, dtype=torch.int32)
        self.T = len(seq)
        self.q = torch.randn(self.T, self.H, self.D, generator=self.g).bfloat16()
        return self

    def upload(self):
        self.d = {n: getattr(self, n).to(DEV) for n in ("seq", "pos", "table", "K", "V", "q")}
        self.pa = sb.paged_args(self.d["seq"], self.d["pos"], self.d["table"], self.H, self.Hkv, self.D, self.P,
                                self.total, self.d["K"], self.d["V"], self.scale)
        return self

    def out(self, fill=7.0):
        return torch.full((self.T, self.H, self.D), fill, dtype=torch.bfloat16, device=DEV)

    def rows(self, t, h, keys):
        """(reference, bound) of the G heads of KV head h of token t over these keys."""
        tab = self.table[int(self.seq[t])]
        k, v = ref.gather(self.K, tab, h, keys, self.P), ref.gather(self.V, tab, h, keys, self.P)
        o, mag, eps = ref.attention(self.q[t, h * self.G:(h + 1) * self.G].double(), k, v, self.scale)
        return o, ref.attn_bound(o, mag, eps, len(keys))

    def check(self, out, keys_of, tokens=None):
        out = out.cpu().double()
        for t in (range(self.T) if tokens is None else tokens):
            for h in range(self.Hkv):
                o, bound = self.rows(t, h, keys_of(t, h))
                err = (out[t, h * self.G:(h + 1) * self.G] - o).abs()
                assert bool((err <= bound).all()), (t, h, float((err / bound).max()))


def status_ok(ws):
    assert sb.sa_check_device_status(ws) == sb.SA_OK


# ------------------------------------------------------------------ append ---

def run_append(c, k, v, **kw):
    ws = sb.new_paged_workspace(c.pa)
    sb.sa_paged_append(c.pa, k, v, ws, **kw)
    return ws


def check_append(c, k, v, q, freqs, halves, q_out, K0, V0):
    K, V = c.d["K"].cpu(), c.d["V"].cpu()
    want_K, want_V = K0.clone(), V0.clone()
    pos = c.pos.numpy()
    kr, kmag = ref.rotate(k.double(), pos, freqs, halves)
    for t in range(c.T):
        page, s = int(c.table[int(c.seq[t]), int(c.pos[t]) // c.P]), int(c.pos[t]) % c.P
        got = K[page, :, s].double()
        # fp32 rotation: coefficients to 2.5e-7, three roundings of 2^-24 each,
        # together below 5e-7 of |a| + |b|; then half a bf16 step
        e = 5e-7 * kmag[t]
        assert bool(((got - kr[t]).abs() <= 2.0 ** -8 * (kr[t].abs() + e) + e + 1e-38).all()), t
        want_K[page, :, s] = K[page, :, s]
        want_V[page, :, s] = v[t]
    # nothing else moved (NaN where it was NaN)
    assert torch.equal(K.view(torch.int16), want_K.view(torch.int16))
    assert torch.equal(V.view(torch.int16), want_V.view(torch.int16))
    if q is not None:
        qr, qmag = ref.rotate(q.double(), pos, freqs, halves)
        e = 5e-7 * qmag
        assert bool(((q_out.cpu().double() - qr).abs() <= 2.0 ** -8 * (qr.abs() + e) + e + 1e-38).all())


@pytest.mark.parametrize("D,P,Hkv,G,dim,halves,yarn", [
    (128, 64, 8, 8, 128, True, False), (128, 128, 1, 64, 64, False, True), (64, 16, 3, 5, 64, True, True),
    (64, 32, 2, 1, 16, False, False), (128, 16, 1, 3, 0, False, False), (128, 32, 5, 2, 48, True, False),
])
def test_append_rotates_and_writes(D, P, Hkv, G, dim, halves, yarn):
    lens = [1, P, P + 1, 3 * P - 1, 777]
    c = Case(1, lens, D, P, Hkv, G)
    seq, pos = [], []
    for b, n in enumerate(lens):  # the last few positions of every sequence, in shuffled order
        for p in range(max(0, n - 2 * P - 3), n):
            seq.append(b)
            pos.append(p)
    order = np.random.RandomState(0).permutation(len(seq))
    c.tokens([seq[i] for i in order], [pos[i] for i in order]).upload()
    base, fac, orig = (160000.0, 16.0, 4096) if yarn else (10000.0, 1.0, 0)
    freqs = ref.rope_freqs(dim, base, fac, orig)
    rope = sb.RopeArgs(dim, base, fac, orig, 32.0, 1.0)
    # k, v and q as slices of one projection
    x = torch.randn(c.T, (c.H + 2 * Hkv) * D, generator=c.g).bfloat16().to(DEV)
    q, k, v = (y.unflatten(1, (-1, D)) for y in x.split([c.H * D, Hkv * D, Hkv * D], dim=1))
    q_out = c.out()
    ws = run_append(c, k, v, q=q, q_out=q_out, rope=rope, halves=halves)
    status_ok(ws)
    check_append(c, k.cpu(), v.cpu(), q.cpu(), freqs, halves, q_out, c.K, c.V)


def test_append_far_positions_keep_their_angle():
    # a page table with one live page per sequence: positions up to 2^30 - 1
    P, D = 128, 128
    far = [2 ** 23 * 128 - 1, 2 ** 29 + 12345, 1_000_003, 65535]
    n_pages = len(far)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(3)
    k = torch.randn(1, 1, D, generator=g).bfloat16()
    freqs = ref.rope_freqs(D, 10000.0)
    for i, p in enumerate(far):
        # table rows of 2^23 entries, all but the last left out by pointing the row before its end
        max_pages = 2 ** 23
        full = torch.zeros(1, max_pages, dtype=torch.int32, device=DEV)
        full[0, p // P] = i
        K = torch.zeros(n_pages, 1, P, D, dtype=torch.bfloat16, device=DEV)
        V = torch.zeros_like(K)
        seq, pos = torch.zeros(1, dtype=torch.int32, device=DEV), torch.full((1,), p, dtype=torch.int32, device=DEV)
        pa = sb.paged_args(seq, pos, full, 1, 1, D, P, n_pages, K, V, 1.0)
        ws = sb.new_paged_workspace(pa)
        sb.sa_paged_append(pa, k.to(DEV), k.to(DEV), ws, rope=sb.RopeArgs(D, 10000.0, 1.0, 0, 32.0, 1.0), halves=True)
        status_ok(ws)
        # the frequency in turns is rounded to 2^-53 of itself on both sides (p f
        # 2^-53 of a radian each, 1.2e-7 at p = 2^30), added to the fp32 terms
        kr, mag = ref.rotate(k.double(), [p], freqs, True)
        e = (5e-7 + 2 * p * 2.0 ** -53) * mag[0]
        got = K[i, :, p % P].cpu().double()
        assert bool(((got - kr[0]).abs() <= 2.0 ** -8 * (kr[0].abs() + e) + e).all()), p
    del table


@pytest.mark.parametrize("D,P,Hkv,n", [(128, 64, 8, 1), (128, 16, 2, 50), (64, 128, 3, 300), (64, 32, 1, 33)])
def test_append_keeps_the_mean_of_pages_that_fill(D, P, Hkv, n):
    lens = [P, 2 * P, 2 * P + 5, P - 1, 5 * P] if n == 1 else [4 * P, 5 * P + 3, n]
    c = Case(4, lens, D, P, Hkv, 1)
    seq = [b for b, m in enumerate(lens) for _ in range(max(0, m - n), m)]
    pos = [p for m in lens for p in range(max(0, m - n), m)]
    c.tokens(seq, pos).upload()
    k = torch.randn(c.T, Hkv, D, generator=c.g).bfloat16().to(DEV)
    mean = torch.full((c.total, Hkv, D), 5.0, dtype=torch.bfloat16, device=DEV)
    ws = run_append(c, k, k, rope=sb.RopeArgs(D, 10000.0, 1.0, 0, 32.0, 1.0), halves=True, k_mean=mean)
    status_ok(ws)
    K, got = c.d["K"].cpu().double(), mean.cpu().double()
    full = {int(c.table[b, p // P]) for b, p in zip(seq, pos) if (p + 1) % P == 0}
    assert full
    for page in range(c.total):
        if page not in full:
            assert bool((got[page] == 5.0).all())
            continue
        m, e = K[page].mean(dim=1), 2.0 ** -24 * K[page].abs().sum(dim=1)  # fp32 sum of P rows
        assert bool(((got[page] - m).abs() <= 2.0 ** -8 * (m.abs() + e) + e).all())


def test_append_skips_and_flags_what_is_out_of_range():
    c = Case(5, [70, 70, 70], P=64)
    c.table[1, 1] = c.total          # a page id past the cache
    c.tokens([0, 3, -1, 1, 2, 0], [69, 5, 5, 68, 64 * 2, -1]).upload()
    k = torch.randn(c.T, c.Hkv, c.D, generator=c.g).bfloat16()
    q_out = c.out()
    ws = run_append(c, k.to(DEV), k.to(DEV), q=c.d["q"], q_out=q_out)
    assert sb.sa_check_device_status(ws) == sb.SA_ERR_DEVICE_DATA
    status_ok(ws)  # read and cleared
    want = c.K.clone()
    want[int(c.table[0, 1]), :, 5] = k[0]
    assert torch.equal(c.d["K"].cpu().view(torch.int16), want.view(torch.int16))
    got = q_out.cpu()
    assert torch.equal(got[0], c.q[0]) and torch.equal(got[3], c.q[3])
    assert bool((got[[1, 2, 4, 5]] == 7.0).all())


def test_append_in_place_queries():
    c = Case(6, [40], D=64, P=16, Hkv=1, G=4)
    c.tokens([0] * 7, range(33, 40)).upload()
    k = torch.randn(c.T, 1, 64, generator=c.g).bfloat16().to(DEV)
    rope = sb.RopeArgs(32, 10000.0, 1.0, 0, 32.0, 1.0)
    q_out = c.out()
    run_append(c, k, k, q=c.d["q"], q_out=q_out, rope=rope)
    run_append(c, k, k, q=c.d["q"], q_out=c.d["q"], rope=rope)
    assert torch.equal(q_out, c.d["q"])


# ------------------------------------------------------------------ scores ---

def check_scores(c, mean, scores, ld=None):
    got = scores.cpu()
    m = mean.cpu().double()
    for t in range(c.T):
        b, vis = int(c.seq[t]), (int(c.pos[t]) + 1) // c.P
        for h in range(c.Hkv):
            row = got[t, h, :c.max_pages].double()
            assert bool((row[vis:] == -float("inf")).all())
            if vis == 0:
                continue
            q = c.q[t, h * c.G:(h + 1) * c.G].double()
            k = m[c.table[b, :vis].long(), h]
            s = q.sum(dim=0) @ k.T * c.scale
            # fp32 sums of G queries and D products, each step off by 2^-23 at
            # most (truncating adds) of the sum of magnitudes
            a = q.abs().sum(dim=0) @ k.abs().T * c.scale
            assert bool(((row[:vis] - s).abs() <= (c.G + c.D + 4) * 2.0 ** -23 * a).all()), (t, h)


@pytest.mark.parametrize("D,P,Hkv,G", [(128, 64, 8, 8), (128, 32, 1, 64), (64, 16, 2, 3), (128, 128, 3, 1),
                                       (64, 128, 1, 128), (128, 16, 4, 5)])
def test_scores_of_a_decode_step(D, P, Hkv, G):
    lens = [1, P - 1, P, P + 1, 17 * P + 5, 40 * P, 3 * P]
    c = Case(7, lens, D, P, Hkv, G)
    c.tokens(range(len(lens)), [n - 1 for n in lens]).upload()
    mean = (torch.randn(c.total, Hkv, D, generator=c.g) / 8).bfloat16().to(DEV)
    scores = torch.full((c.T, Hkv, c.max_pages + 3), 9.0, device=DEV)
    ws = sb.new_paged_workspace(c.pa)
    sb.sa_page_scores(c.pa, c.d["q"], mean, scores, ws)
    status_ok(ws)
    check_scores(c, mean, scores)
    assert bool((scores[..., c.max_pages:] == 9.0).all())


@pytest.mark.parametrize("D,P,Hkv,G,new", [(128, 64, 4, 16, 300), (64, 16, 1, 3, 129), (128, 128, 2, 64, 64),
                                           (128, 32, 1, 1, 1000)])
def test_scores_of_prefill_chunks(D, P, Hkv, G, new):
    lens = [new + 900, new, new + 31]
    c = Case(8, lens, D, P, Hkv, G)
    seq = [b for b in range(3) for _ in range(new)]
    pos = [p for n in lens for p in range(n - new, n)]
    c.tokens(seq, pos).upload()
    mean = (torch.randn(c.total, Hkv, D, generator=c.g) / 8).bfloat16().to(DEV)
    scores = torch.empty(c.T, Hkv, c.max_pages, device=DEV)
    ws = sb.new_paged_workspace(c.pa)
    sb.sa_page_scores(c.pa, c.d["q"], mean, scores, ws)
    status_ok(ws)
    check_scores(c, mean, scores)


def test_scores_tokens_in_any_order_and_out_of_range():
    c = Case(9, [500, 300, 777], D=128, P=16, Hkv=2, G=4)
    r = np.random.RandomState(1)
    seq = r.randint(0, 3, size=200)
    pos = np.array([r.randint(0, c.lens[b]) for b in seq])
    seq[13], seq[140], pos[77] = 3, -1, 16 * c.max_pages
    c.tokens(seq.tolist(), pos.tolist()).upload()
    mean = (torch.randn(c.total, 2, 128, generator=c.g) / 8).bfloat16().to(DEV)
    scores = torch.full((c.T, 2, c.max_pages), 9.0, device=DEV)
    ws = sb.new_paged_workspace(c.pa)
    sb.sa_page_scores(c.pa, c.d["q"], mean, scores, ws)
    assert sb.sa_check_device_status(ws) == sb.SA_ERR_DEVICE_DATA
    assert bool((scores[[13, 140, 77]] == 9.0).all())
    keep = [t for t in range(200) if t not in (13, 140, 77)]
    c.T, c.seq, c.pos, c.q = len(keep), c.seq[keep], c.pos[keep], c.q[keep]
    check_scores(c, mean, scores[keep])


# --------------------------------------------------------- block attention ---

def make_idx(c, K, local, seed=0, tricks=True):
    """Random lists: distinct pages before the local ones, -1 at the end, and
    (with ``tricks``) an entry twice, local pages, -1 in the middle."""
    r = np.random.RandomState(seed)
    idx = np.full((c.T, c.Hkv, K), -1, dtype=np.int32)
    for t in range(c.T):
        last = int(c.pos[t]) // c.P
        f = max(last + 1 - local, 0)
        for h in range(c.Hkv):
            n = min(K, f, r.randint(0, K + 1) if K else 0)
            idx[t, h, :n] = np.sort(r.permutation(f)[:n])
            if tricks and K >= 3 and n >= 3 and (t + h) % 3 == 0:
                idx[t, h, 0] = idx[t, h, 2]
                idx[t, h, 1] = last if (t + h) % 2 else -1
    return torch.from_numpy(idx)


@pytest.mark.parametrize("D,P,Hkv,G,K,local", [
    (128, 64, 1, 64, 32, 2), (128, 64, 2, 8, 5, 1), (64, 16, 2, 3, 40, 0), (128, 128, 1, 16, 3, 1),
    (64, 128, 3, 1, 7, 2), (128, 16, 1, 128, 20, 9), (128, 32, 1, 100, 11, 0), (64, 64, 1, 48, 8, 1),
    (128, 64, 2, 8, 0, 1), (128, 64, 2, 8, 0, 0), (64, 32, 8, 5, 1, 3),
])
def test_block_attention_of_a_decode_step(D, P, Hkv, G, K, local):
    lens = [1, 2, P - 1, P, P + 1, 9 * P + 7, 45 * P, 50 * P + P // 2]
    c = Case(10, lens, D, P, Hkv, G)
    c.tokens(range(len(lens)), [n - 1 for n in lens]).upload()
    idx = make_idx(c, K, local)
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, K, local)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), K, local, out, ws)
    status_ok(ws)
    c.check(out, lambda t, h: ref.block_keys(int(c.pos[t]), P, idx[t, h].tolist(), local, c.max_pages))


@pytest.mark.parametrize("D,P,Hkv,G,K,local,new", [
    (128, 64, 1, 64, 12, 2, 200), (128, 128, 2, 8, 4, 1, 333), (64, 16, 1, 16, 30, 1, 170)])
def test_block_attention_of_a_prefill_chunk(D, P, Hkv, G, K, local, new):
    c = Case(11, [2000 + new, new], D, P, Hkv, G)
    c.tokens([0] * new + [1] * new, list(range(2000, 2000 + new)) + list(range(new))).upload()
    idx = make_idx(c, K, local, seed=3)
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, K, local)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), K, local, out, ws)
    status_ok(ws)
    c.check(out, lambda t, h: ref.block_keys(int(c.pos[t]), P, idx[t, h].tolist(), local, c.max_pages),
            tokens=list(range(0, 2 * new, 7)) + [2 * new - 1])


def test_block_attention_out_of_range_data_is_skipped_and_flagged():
    P = 32
    c = Case(12, [400, 400, 400, 400], P=P, Hkv=1, G=4)
    good = c.table.clone()
    c.table[2, 3] = -1
    c.tokens([0, 1, 2, 5, 3], [399, 200, 399, 10, 32 * c.max_pages]).upload()
    idx = torch.full((5, 1, 4), -1, dtype=torch.int32)
    idx[0, 0] = torch.tensor([1, 100000, 4, -9])     # past the sequence, below -1
    idx[1, 0] = torch.tensor([0, 9, 2, -1])          # 9 lies past the token's position
    idx[2, 0] = torch.tensor([3, 5, 6, -1])          # 3 is a bad page
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, 4, 1)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), 4, 1, out, ws)
    assert sb.sa_check_device_status(ws) == sb.SA_ERR_DEVICE_DATA
    assert bool((out[3:] == 7.0).all())
    c.table = good
    lists = [[1, 4], [0, 2], [5, 6]]
    c.check(out, lambda t, h: ref.block_keys(int(c.pos[t]), P, lists[t], 1, c.max_pages), tokens=range(3))


def test_block_attention_with_extreme_values():
    # logits of thousands apart: weights underflow, nothing overflows; equal
    # rows of +-3e38-ish values stay finite
    c = Case(13, [300, 200], D=64, P=16, Hkv=1, G=16)
    c.K *= 40
    c.V *= 1e37
    c.tokens([0, 1], [299, 199])
    c.q *= 40
    c.upload()
    idx = torch.tensor([[[0, 3, 7, -1]], [[2, 5, -1, -1]]], dtype=torch.int32)
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, 4, 2)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), 4, 2, out, ws)
    status_ok(ws)
    assert bool(torch.isfinite(out.float()).all())
    c.check(out, lambda t, h: ref.block_keys(int(c.pos[t]), 16, idx[t, h].tolist(), 2, c.max_pages))


# -------------------------------------------------------- prefix attention ---

@pytest.mark.parametrize("D,P,Hkv,G,shared,tails", [
    (128, 64, 8, 8, 5, [1, 64, 65, 200, 3]),
    (128, 128, 1, 64, 3, [1, 5, 129, 400, 77, 30, 2]),
    (64, 16, 2, 3, 21, [1, 2, 15, 16, 17, 300]),
    (128, 32, 1, 128, 9, [33, 1]),
    (64, 64, 1, 1, 1, [1]),
    (128, 16, 3, 5, 0, [1, 16, 500, 33]),
    (64, 128, 2, 100, 2, [1, 140, 9]),
    (128, 64, 2, 16, 33, [64] * 40),
])
def test_prefix_attention_of_a_decode_step(D, P, Hkv, G, shared, tails):
    lens = [shared * P + n for n in tails]
    c = Case(14, lens, D, P, Hkv, G, shared=shared)
    c.tokens(range(len(lens)), [n - 1 for n in lens]).upload()
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, shared_pages=shared)
    sb.sa_prefix_attn(c.pa, c.d["q"], shared, out, ws)
    status_ok(ws)
    c.check(out, lambda t, h: list(range(int(c.pos[t]) + 1)))


@pytest.mark.parametrize("D,P,Hkv,G,shared", [(128, 64, 2, 4, 7), (64, 32, 1, 16, 0), (128, 128, 1, 64, 2)])
def test_prefix_attention_with_several_tokens_per_sequence(D, P, Hkv, G, shared):
    lens = [shared * P + 90, shared * P + 300]
    c = Case(15, lens, D, P, Hkv, G, shared=shared)
    seq = [1] * 61 + [0] * 30
    pos = list(range(lens[1] - 61, lens[1])) + list(range(lens[0] - 30, lens[0]))
    c.tokens(seq, pos).upload()
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, shared_pages=shared)
    sb.sa_prefix_attn(c.pa, c.d["q"], shared, out, ws)
    status_ok(ws)
    c.check(out, lambda t, h: list(range(int(c.pos[t]) + 1)), tokens=range(0, 91, 3))


def test_prefix_attention_skips_tokens_it_cannot_serve():
    P, shared = 32, 3
    lens = [shared * P + 40] * 3
    c = Case(16, lens, P=P, shared=shared)
    c.tokens([0, 1, 2, 7, 1], [lens[0] - 1, shared * P - 1, shared * P, 100, 32 * c.max_pages]).upload()
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, shared_pages=shared)
    sb.sa_prefix_attn(c.pa, c.d["q"], shared, out, ws)
    assert sb.sa_check_device_status(ws) == sb.SA_ERR_DEVICE_DATA
    assert bool((out[[1, 3, 4]] == 7.0).all())
    c.check(out, lambda t, h: list(range(int(c.pos[t]) + 1)), tokens=[0, 2])


# ---------------------------------------------------------------- together ---

def test_decode_steps_through_the_paged_cache():
    """Append a prompt, then decode steps: append, fused block attention, full
    attention over the shared prefix; the cache is the only state."""
    D, P, Hkv, G, B, K, local = 128, 16, 2, 8, 3, 6, 1
    c = Case(17, [420, 360, 500], D, P, Hkv, G, shared=18)  # room for 20 steps
    c.K.zero_()
    c.V.zero_()
    rope = sb.RopeArgs(64, 10000.0, 1.0, 0, 32.0, 1.0)
    mean = torch.zeros(c.total, Hkv, D, dtype=torch.bfloat16, device=DEV)
    start = [400, 340, 470]
    # prompt: the shared pages once (sequence 0), then each sequence's own tokens
    seq = [0] * start[0] + [1] * (start[1] - 288) + [2] * (start[2] - 288)
    pos = list(range(start[0])) + list(range(288, start[1])) + list(range(288, start[2]))
    c.tokens(seq, pos).upload()
    x = torch.randn(3, c.T, Hkv, D, generator=c.g).bfloat16().to(DEV)
    ws = sb.new_paged_workspace(c.pa)
    sb.sa_paged_append(c.pa, x[0], x[1], ws, rope=rope, k_mean=mean)
    status_ok(ws)
    cache = dict(K=c.d["K"], V=c.d["V"])
    for step in range(20):
        p = [s + step for s in start]
        c.tokens([0, 1, 2], p)
        c.d.update({n: getattr(c, n).to(DEV) for n in ("seq", "pos", "q")})
        c.pa = sb.paged_args(c.d["seq"], c.d["pos"], c.d["table"], c.H, Hkv, D, P, c.total, cache["K"], cache["V"],
                             c.scale)
        kv = torch.randn(2, 3, Hkv, D, generator=c.g).bfloat16().to(DEV)
        ws = sb.new_paged_workspace(c.pa, K, local, 18)
        q = torch.empty_like(c.d["q"])
        sb.sa_paged_append(c.pa, kv[0], kv[1], ws, q=c.d["q"], q_out=q, rope=rope, k_mean=mean)
        idx = torch.empty(3, Hkv, K, dtype=torch.int32, device=DEV)
        out, out2, out3 = c.out(), c.out(), c.out()
        sb.sa_fused_block_attn(c.pa, q, mean, K, local, idx, out, ws)
        sb.sa_block_attn(c.pa, q, idx, K, local, out2, ws)
        sb.sa_prefix_attn(c.pa, q, 18, out3, ws)
        status_ok(ws)
        assert torch.equal(out, out2)
        if step % 5:
            continue
        c.q, c.K, c.V = q.cpu(), cache["K"].cpu(), cache["V"].cpu()
        m = mean.cpu().double()
        for t in range(3):
            f = max(p[t] // P + 1 - local, 0)
            for h in range(Hkv):
                qs = c.q[t, h * G:(h + 1) * G].double()
                k = m[c.table[t, :f].long(), h]
                s = qs.sum(dim=0) @ k.T * c.scale
                tol = 2 * (G + D + 4) * 2.0 ** -23 * (qs.abs().sum(dim=0) @ k.abs().T * c.scale)
                pick = idx[t, h].tolist()
                assert pick == sorted(pick) and len(set(pick)) == K and max(pick) < f
                kth = s[torch.tensor(pick)].min()
                rest = torch.ones(f, dtype=torch.bool)
                rest[pick] = False
                # every page left out scores no more than the weakest pick, up to both errors
                assert bool((s[rest] <= kth + tol[rest] + tol[pick].max()).all())
        c.check(out, lambda t, h: ref.block_keys(p[t], P, idx[t, h].tolist(), local, c.max_pages))
        c.check(out3, lambda t, h: list(range(p[t] + 1)))


def test_calls_captured_in_a_graph_follow_the_device_state():
    D, P, Hkv, G, K, local = 128, 32, 2, 4, 4, 1
    c = Case(18, [300, 200, 120], D, P, Hkv, G, shared=2, poison=False)
    c.tokens([0, 1, 2], [250, 180, 100]).upload()
    mean = (torch.randn(c.total, Hkv, D, generator=c.g) / 6).bfloat16().to(DEV)
    kv = torch.randn(2, 3, Hkv, D, generator=c.g).bfloat16().to(DEV)
    ws = sb.new_paged_workspace(c.pa, K, local, 2)
    q, out, out2 = torch.empty_like(c.d["q"]), c.out(), c.out()
    rope = sb.RopeArgs(128, 10000.0, 1.0, 0, 32.0, 1.0)

    def step():
        sb.sa_paged_append(c.pa, kv[0], kv[1], ws, q=c.d["q"], q_out=q, rope=rope, halves=True, k_mean=mean)
        sb.sa_fused_block_attn(c.pa, q, mean, K, local, None, out, ws)
        sb.sa_prefix_attn(c.pa, q, 2, out2, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for add in (0, 1, 5):
        c.d["pos"].add_(add)
        kv.normal_()
        g.replay()
        got = [x.clone() for x in (out, out2, q, mean, c.d["K"], c.d["V"])]
        step()
        for a, b in zip(got, (out, out2, q, mean, c.d["K"], c.d["V"])):
            assert torch.equal(a, b)
    status_ok(ws)


def test_two_streams_with_a_workspace_each():
    cs = [Case(19 + i, [900, 1200, 700], 128, 64, 2, 8, shared=4).tokens([0, 1, 2], [899, 1199, 699]).upload()
          for i in range(2)]
    ws = [sb.new_paged_workspace(c.pa, shared_pages=4) for c in cs]
    outs = [c.out() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        for c, w, o, s in zip(cs, ws, outs, streams):
            sb.sa_prefix_attn(c.pa, c.d["q"], 4, o, w, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        c.check(o, lambda t, h: list(range(int(c.pos[t]) + 1)))


def test_results_repeat_bit_for_bit():
    c = Case(21, [3000, 2500, 1777, 900], 128, 64, 2, 8, shared=10)
    c.tokens(range(4), [2999, 2499, 1776, 899]).upload()
    idx = make_idx(c, 9, 2, tricks=False).to(DEV)
    ws = sb.new_paged_workspace(c.pa, 9, 2, 10)
    first = None
    for _ in range(5):
        a, b = c.out(), c.out()
        sb.sa_block_attn(c.pa, c.d["q"], idx, 9, 2, a, ws)
        sb.sa_prefix_attn(c.pa, c.d["q"], 10, b, ws)
        if first is None:
            first = (a, b)
        assert torch.equal(a, first[0]) and torch.equal(b, first[1])


def test_page_table_rows_may_be_strided():
    c = Case(22, [500, 300], 64, 32, 1, 4)
    c.tokens([0, 1], [499, 299]).upload()
    wide = torch.full((2, c.max_pages + 11), -3, dtype=torch.int32, device=DEV)
    wide[:, :c.max_pages] = c.d["table"]
    c.pa = sb.paged_args(c.d["seq"], c.d["pos"], wide[:, :c.max_pages], c.H, c.Hkv, c.D, c.P, c.total, c.d["K"],
                         c.d["V"], c.scale)
    out = c.out()
    ws = sb.new_paged_workspace(c.pa)
    sb.sa_prefix_attn(c.pa, c.d["q"], 0, out, ws)
    status_ok(ws)
    c.check(out, lambda t, h: list(range(int(c.pos[t]) + 1)))


def test_a_long_cache_passes_32_bit_offsets():
    # 2^31 elements lie past the first 17 million rows of 128 values
    P, D, Hkv = 128, 128, 1
    n_pages = (1 << 31) // (P * D) + 40
    K = torch.zeros(n_pages, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    c = Case(23, [1500, 800], D, P, Hkv, 16, extra=0)
    K[-c.total:] = c.K.to(DEV)
    V[-c.total:] = c.V.to(DEV)
    c.tokens([0, 1], [1499, 799]).upload()
    table = torch.where(c.d["table"] >= 0, c.d["table"] + (n_pages - c.total), c.d["table"])
    c.pa = sb.paged_args(c.d["seq"], c.d["pos"], table, c.H, Hkv, D, P, n_pages, K, V, c.scale)
    out, out2 = c.out(), c.out()
    idx = make_idx(c, 5, 1, tricks=False)
    ws = sb.new_paged_workspace(c.pa, 5, 1)
    sb.sa_prefix_attn(c.pa, c.d["q"], 0, out, ws)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), 5, 1, out2, ws)
    kv = torch.randn(2, 2, Hkv, D, generator=c.g).bfloat16().to(DEV)
    sb.sa_paged_append(c.pa, kv[0], kv[1], ws)
    status_ok(ws)
    c.check(out, lambda t, h: list(range(int(c.pos[t]) + 1)))
    c.check(out2, lambda t, h: ref.block_keys(int(c.pos[t]), P, idx[t, h].tolist(), 1, c.max_pages))
    for t in range(2):
        page = int(table[t, int(c.pos[t]) // P])
        assert torch.equal(K[page, :, int(c.pos[t]) % P], kv[0, t])


# ------------------------------------------------- masks, scales, large lists ---

@pytest.mark.parametrize("Hkv,G,T_per,B", [(9, 2, 1, 5), (17, 1, 1, 3), (3, 4, 40, 2), (1, 8, 15, 2)])
def test_scores_with_nan_means_of_unseen_pages(Hkv, G, T_per, B):
    P, D = 16, 128
    lens = [T_per + 16 * 20 + 7 * b for b in range(B)]
    c = Case(30, lens, D, P, Hkv, G)
    c.tokens([b for b in range(B) for _ in range(T_per)], [p for n in lens for p in range(n - T_per, n)]).upload()
    mean = (torch.randn(c.total, Hkv, D, generator=c.g) / 4).bfloat16()
    seen = torch.zeros(c.total, dtype=torch.bool)
    for b, n in enumerate(lens):
        seen[c.table[b, :n // P].long()] = True
    mean[~seen] = float("nan")
    mean = mean.to(DEV)
    scores = torch.empty(c.T, Hkv, c.max_pages, device=DEV)
    ws = sb.new_paged_workspace(c.pa)
    sb.sa_page_scores(c.pa, c.d["q"], mean, scores, ws)
    status_ok(ws)
    check_scores(c, mean, scores)


@pytest.mark.parametrize("scale", [0.0, -0.07, 0.3])
@pytest.mark.parametrize("shared", [0, 3])
def test_attention_at_other_scales(scale, shared):
    P = 32
    c = Case(31, [shared * P + 77, shared * P + 300], 128, P, 1, 16, shared=shared)
    c.scale = scale
    c.tokens([0, 1], [n - 1 for n in c.lens]).upload()
    out, out2 = c.out(), c.out()
    idx = make_idx(c, 4, 1, seed=2)
    ws = sb.new_paged_workspace(c.pa, 4, 1, shared)
    sb.sa_prefix_attn(c.pa, c.d["q"], shared, out, ws)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), 4, 1, out2, ws)
    status_ok(ws)
    c.check(out, lambda t, h: list(range(int(c.pos[t]) + 1)))
    c.check(out2, lambda t, h: ref.block_keys(int(c.pos[t]), P, idx[t, h].tolist(), 1, c.max_pages))


@pytest.mark.parametrize("D,P,G,K", [(128, 16, 8, 700), (64, 16, 64, 700), (128, 128, 40, 90)])
def test_block_attention_over_long_lists(D, P, G, K):
    n = 100 * P if P == 128 else 800 * P
    c = Case(32, [n - 5], D, P, 1, G)
    c.tokens([0, 0], [n - 6, n // 2]).upload()
    idx = make_idx(c, K, 2, seed=5, tricks=False)
    idx[0, 0] = torch.arange(K, dtype=torch.int32) + (3 if P != 128 else 1)
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, K, 2)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), K, 2, out, ws)
    status_ok(ws)
    c.check(out, lambda t, h: ref.block_keys(int(c.pos[t]), P, idx[t, h].tolist(), 2, c.max_pages))


def test_block_attention_rows_without_any_key_are_zero():
    c = Case(33, [100, 100], 128, 16, 2, 8)
    c.tokens([0, 1], [99, 50]).upload()
    idx = torch.full((2, 2, 5), -1, dtype=torch.int32)
    idx[1, 1, 2] = 1
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, 5, 0)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), 5, 0, out, ws)
    status_ok(ws)
    assert bool((out[0] == 0).all()) and bool((out[1, :8] == 0).all()) and bool((out[1, 8:] != 0).any())
    c.check(out, lambda t, h: ref.block_keys(int(c.pos[t]), 16, idx[t, h].tolist(), 0, c.max_pages))


@pytest.mark.parametrize("G,shared", [(8, 0), (8, 2), (64, 2), (128, 1)])
def test_prefix_attention_with_uneven_long_tails(G, shared):
    P, D = 64, 128
    tails = [1, 2900, 3, 64, 1500, 1, 700, 130, 5, 2048]
    c = Case(34, [shared * P + n for n in tails], D, P, 2 if G <= 64 else 1, G, shared=shared)
    c.tokens(range(len(tails)), [n - 1 for n in c.lens]).upload()
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, shared_pages=shared)
    for _ in range(3):  # the claims start from zero at every call
        out.fill_(7.0)
        sb.sa_prefix_attn(c.pa, c.d["q"], shared, out, ws)
    status_ok(ws)
    c.check(out, lambda t, h: list(range(int(c.pos[t]) + 1)))


def test_prefix_attention_when_every_token_lies_inside_the_shared_pages():
    c = Case(35, [200, 200], 128, 32, 1, 8, shared=7)
    c.tokens([0, 1], [100, 199]).upload()
    out = c.out()
    ws = sb.new_paged_workspace(c.pa, shared_pages=7)
    sb.sa_prefix_attn(c.pa, c.d["q"], 7, out, ws)
    assert sb.sa_check_device_status(ws) == sb.SA_ERR_DEVICE_DATA
    assert bool((out == 7.0).all())


def test_prefix_attention_with_a_bad_shared_page():
    P, shared = 16, 11
    c = Case(36, [shared * P + 9, shared * P + 40], 128, P, 1, 16, shared=shared)
    c.tokens([0, 1], [n - 1 for n in c.lens]).upload()
    for bad in ([4], list(range(8)), list(range(shared))):
        table = c.d["table"].clone()
        table[0, bad] = c.total + 5
        pa = sb.paged_args(c.d["seq"], c.d["pos"], table, c.H, 1, 128, P, c.total, c.d["K"], c.d["V"], c.scale)
        out = c.out()
        ws = sb.new_paged_workspace(pa, shared_pages=shared)
        sb.sa_prefix_attn(pa, c.d["q"], shared, out, ws)
        assert sb.sa_check_device_status(ws) == sb.SA_ERR_DEVICE_DATA
        c.check(out, lambda t, h: [p for p in range(int(c.pos[t]) + 1) if p // P not in bad])


def test_prefix_attention_raises_its_reference_along_the_keys():
    # keys grow along the sequence, so that every tile passes the one before by
    # far more than the lazy margin
    P, shared, D = 64, 8, 128
    c = Case(37, [shared * P + 500, shared * P + 200], D, P, 1, 64, shared=shared)
    for b, n in enumerate(c.lens):
        for j in range((n + P - 1) // P):
            page = int(c.table[b, j])
            if b == 0 or j >= shared:
                c.K[page] = (c.K[page].float() * (1 + 3.0 * j)).bfloat16()
    c.tokens([0, 1], [n - 1 for n in c.lens]).upload()
    out, out2 = c.out(), c.out()
    idx = make_idx(c, 9, 1, seed=1, tricks=False)
    ws = sb.new_paged_workspace(c.pa, 9, 1, shared)
    sb.sa_prefix_attn(c.pa, c.d["q"], shared, out, ws)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), 9, 1, out2, ws)
    status_ok(ws)
    c.check(out, lambda t, h: list(range(int(c.pos[t]) + 1)))
    c.check(out2, lambda t, h: ref.block_keys(int(c.pos[t]), P, idx[t, h].tolist(), 1, c.max_pages))


@pytest.mark.parametrize("new,Hkv,G,K,local", [(150, 2, 8, 5, 1), (1, 3, 5, 7, 2), (64, 1, 64, 0, 2)])
def test_fused_block_attention(new, Hkv, G, K, local):
    D, P = 128, 32
    lens = [900 + new, 31 + new, 400 + new]
    c = Case(38, lens, D, P, Hkv, G)
    c.tokens([b for b in range(3) for _ in range(new)], [p for n in lens for p in range(n - new, n)]).upload()
    mean = (torch.randn(c.total, Hkv, D, generator=c.g) / 5).bfloat16().to(DEV)
    ws = sb.new_paged_workspace(c.pa, K, local)
    idx = torch.full((c.T, Hkv, max(K, 1)), 77, dtype=torch.int32, device=DEV)
    out, out2, out3 = c.out(), c.out(), c.out()
    sb.sa_fused_block_attn(c.pa, c.d["q"], mean, K, local, idx if K else None, out, ws)
    sb.sa_fused_block_attn(c.pa, c.d["q"], mean, K, local, None, out2, ws)
    sb.sa_block_attn(c.pa, c.d["q"], idx if K else None, K, local, out3, ws)
    status_ok(ws)
    assert torch.equal(out, out2) and torch.equal(out, out3)
    if K == 0:
        return
    # the picks are the exact top-k of the scores this call's scorer gives
    scores = torch.empty(c.T, Hkv, c.max_pages, device=DEV)
    sb.sa_page_scores(c.pa, c.d["q"], mean, scores, ws)
    s = scores.cpu()
    for t in range(c.T):
        f = max(int(c.pos[t]) // P + 1 - local, 0)
        for h in range(Hkv):
            order = sorted(range(f), key=lambda j: (-float(s[t, h, j]), j))[:K]
            assert idx[t, h].tolist() == sorted(order) + [-1] * (K - len(order)), (t, h)


def test_calls_run_on_the_stream_they_are_given():
    # the calls run on the stream they are given, whichever is current
    c = Case(39, [300], 128, 64, 1, 8).tokens([0], [299]).upload()
    ws = sb.new_paged_workspace(c.pa)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = c.out(), c.out()
    torch.cuda.synchronize()
    sb.sa_prefix_attn(c.pa, c.d["q"], 0, a, ws, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        sb.sa_prefix_attn(c.pa, c.d["q"], 0, b, ws)
    side.synchronize()
    assert torch.equal(a, b)
    c.check(a, lambda t, h: list(range(300)))


# ------------------------------------------------------- many tokens at once ---

@pytest.mark.parametrize("D,P,Hkv,G,lens,new,order,ld", [
    (128, 16, 8, 2, [5001], 700, "rising", 0),
    (64, 16, 4, 4, [4001, 2500], 600, "rising", 0),
    (128, 64, 8, 1, [16384], 1300, "rising", 0),          # whole blocks of pages, rows 16-byte aligned
    (128, 32, 8, 16, [9000], 513, "rising", 288),
    (128, 16, 8, 3, [3007, 1200, 2999], 300, "mixed", 0),
    (64, 16, 8, 1, [3000, 16, 700], 400, "falling", 191),
])
def test_scores_of_large_chunks(D, P, Hkv, G, lens, new, order, ld):
    r = np.random.RandomState(5)
    c = Case(40, lens, D, P, Hkv, G)
    at = [(b, p) for b, n in enumerate(lens) for p in range(max(n - new, 0), n)]
    if order == "mixed":
        at = [at[i] for i in r.permutation(len(at))]
    elif order == "falling":
        at = at[::-1]
    bad = [17, len(at) // 2, len(at) - 1] if order == "mixed" else []
    seq, pos = [b for b, _ in at], [p for _, p in at]
    for t in bad:
        seq[t] = len(lens) if t == 17 else -3
    c.tokens(seq, pos)
    mean = (torch.randn(c.total, Hkv, D, generator=c.g) / 8).bfloat16()
    seen = torch.zeros(c.total, dtype=torch.bool)
    for b, n in enumerate(lens):
        seen[c.table[b, :n // P].long()] = True
    mean[~seen] = float("nan")
    lost = order == "falling"
    if lost:  # a page whose id is out of range scores -inf
        c.table[0, 5] = c.total
    c.upload()
    width = ld or c.max_pages
    scores = torch.full((c.T, Hkv, width), 9.0, device=DEV)
    ws = sb.new_paged_workspace(c.pa)
    sb.sa_page_scores(c.pa, c.d["q"], mean.to(DEV), scores, ws)
    assert sb.sa_check_device_status(ws) == (sb.SA_ERR_DEVICE_DATA if bad or lost else sb.SA_OK)
    got = scores.cpu().double()
    q = c.q.double().view(c.T, Hkv, G, D)
    assert bool((got[..., c.max_pages:] == 9.0).all()) and bool((got[bad] == 9.0).all())
    for b, n in enumerate(lens):
        tok = [t for t in range(c.T) if seq[t] == b]
        k = torch.zeros(Hkv, c.max_pages, D, dtype=torch.float64)
        ids = c.table[b, :n // P].long().clamp(max=c.total - 1)
        k[:, :n // P] = mean[ids].double().nan_to_num().transpose(0, 1)
        s = torch.einsum("thd,hjd->thj", q[tok].sum(2), k) * c.scale
        # as check_scores: G sums and D products in fp32
        bound = torch.einsum("thd,hjd->thj", q[tok].abs().sum(2), k.abs()) * c.scale * (G + D + 4) * 2.0 ** -23
        vis = (torch.tensor([pos[t] for t in tok]) + 1) // P
        live = (torch.arange(c.max_pages)[None] < vis[:, None])[:, None].expand(-1, Hkv, -1).clone()
        if lost and b == 0:
            live[..., 5] = False
        row = got[tok][..., :c.max_pages]
        assert bool((row[~live] == -float("inf")).all())
        assert bool(((row - s).abs() <= bound)[live].all())


@pytest.mark.parametrize("D,P,Hkv,G,dim,halves", [(128, 64, 8, 3, 128, True), (64, 16, 3, 1, 32, False),
                                                  (128, 128, 1, 64, 64, False), (64, 128, 5, 1, 64, True)])
def test_append_of_many_tokens(D, P, Hkv, G, dim, halves):
    lens = [5 * P + 3, 2000, 17, 901]
    c = Case(41, lens, D, P, Hkv, G)
    seq, pos = [b for b, n in enumerate(lens) for _ in range(n)], [p for n in lens for p in range(n)]
    order = np.random.RandomState(2).permutation(len(seq))
    c.tokens([seq[i] for i in order], [pos[i] for i in order]).upload()
    rope = sb.RopeArgs(dim, 10000.0, 1.0, 0, 32.0, 1.0)
    k, v = (torch.randn(c.T, Hkv, D, generator=c.g).bfloat16().to(DEV) for _ in range(2))
    mean, q_out = torch.full((c.total, Hkv, D), 5.0, dtype=torch.bfloat16, device=DEV), c.out()
    ws = run_append(c, k, v, q=c.d["q"], q_out=q_out, rope=rope, halves=halves, k_mean=mean)
    status_ok(ws)
    check_append(c, k.cpu(), v.cpu(), c.q, ref.rope_freqs(dim, 10000.0), halves, q_out, c.K, c.V)
    K, got = c.d["K"].cpu().double(), mean.cpu().double()
    full = torch.zeros(c.total, dtype=torch.bool)
    for b, n in enumerate(lens):
        full[c.table[b, :n // P].long()] = True
    assert bool((got[~full] == 5.0).all())
    m, e = K[full].mean(dim=2), 2.0 ** -24 * K[full].abs().sum(dim=2)  # fp32 sum of P rows
    assert bool(((got[full] - m).abs() <= 2.0 ** -8 * (m.abs() + e) + e).all())


# ------------------------------------------------------------ shared pieces ---

@pytest.mark.parametrize("D,P,G,T", [(128, 128, 64, 32), (64, 128, 128, 16), (128, 64, 16, 96)])
@pytest.mark.parametrize("lost", ["first", "first two tiles", "odd tiles", "even tiles", "most"])
def test_prefix_attention_with_shared_tiles_lost(D, P, G, T, lost):
    # several tiles of 128 shared keys to a CTA, some without a page: where a
    # piece begins with one, the tiles after it count as ever.  Logits several
    # units apart, so that a tile's weights are far from equal.
    tiles, spt = 96, 128 // P
    shared = tiles * spt
    bad_tiles = dict(zip(("first", "first two tiles", "odd tiles", "even tiles", "most"),
                         ([0], [0, 1], range(1, tiles, 2), range(0, tiles, 2), range(0, tiles - 5))))[lost]
    c = Case(50, [shared * P + 9, shared * P + 200, shared * P + 128], D, P, 1, G, shared=shared)
    c.tokens([t % 3 for t in range(T)], [c.lens[t % 3] - 1 - t // 3 % 9 for t in range(T)])
    c.q *= 5
    c.upload()
    table = c.d["table"].clone()
    bad = torch.tensor([j * spt + i for j in bad_tiles for i in range(spt)])
    table[0, bad.to(DEV)] = -1
    pa = sb.paged_args(c.d["seq"], c.d["pos"], table, c.H, 1, D, P, c.total, c.d["K"], c.d["V"], c.scale)
    out = c.out()
    ws = sb.new_paged_workspace(pa, shared_pages=shared)
    sb.sa_prefix_attn(pa, c.d["q"], shared, out, ws)
    assert sb.sa_check_device_status(ws) == sb.SA_ERR_DEVICE_DATA
    keep = torch.ones(shared, dtype=torch.bool)
    keep[bad] = False
    pos = torch.arange(shared * P)[keep.repeat_interleave(P)]
    c.check(out, lambda t, h: torch.cat([pos, torch.arange(shared * P, int(c.pos[t]) + 1)]), tokens=range(0, T, 5))


# --------------------------------------------------------------------- NaN ---

@pytest.mark.parametrize("T,D,P,Hkv,G,K,shared", [
    (1, 128, 64, 2, 8, 32, 0), (1, 64, 16, 1, 16, 200, 300), (1, 128, 128, 1, 64, 9, 40),   # units cut over CTAs
    (3, 128, 64, 1, 40, 60, 70), (40, 128, 32, 2, 16, 6, 9), (150, 64, 64, 1, 64, 3, 5),
    (333, 128, 64, 1, 8, 1, 1),                                                             # units of one CTA each
])
def test_nan_stays_in_the_rows_it_belongs_to(T, D, P, Hkv, G, K, shared):
    # a head of NaN in the first query, and a NaN key of KV head 0 that only the
    # last token (alone in its sequence) sees: NaN there however the work is cut,
    # and nowhere else
    n = max((K + 3) * P, (shared + 2) * P) + T + 7
    c = Case(51, [n, n], D, P, Hkv, G, shared=shared)
    c.tokens([0] * (T - 1) + [1], [n - 1 - t for t in range(T)])
    c.q[0, G // 2] = float("nan")
    last = int(c.pos[T - 1])
    c.K[int(c.table[1, last // P]), 0, last % P] = float("nan")
    c.upload()
    idx = torch.full((T, Hkv, max(K, 1)), -1, dtype=torch.int32)
    for t in range(T):
        idx[t, :, :K] = torch.arange(K, dtype=torch.int32)
    out, out2, out3 = c.out(), c.out(), c.out()
    ws = sb.new_paged_workspace(c.pa, K, 2, shared)
    sb.sa_block_attn(c.pa, c.d["q"], idx.to(DEV), K, 2, out, ws)
    sb.sa_prefix_attn(c.pa, c.d["q"], shared, out2, ws)
    sb.sa_prefix_attn(c.pa, c.d["q"], 0, out3, sb.new_paged_workspace(c.pa))
    status_ok(ws)
    want = torch.zeros(T, c.H, D, dtype=torch.bool)
    want[0, G // 2] = True
    want[T - 1, :G] = True
    for o in (out, out2, out3):
        assert torch.equal(torch.isnan(o.cpu()), want)
    c.q[0, G // 2] = 0  # (the oracle's bound is one for a group's heads; this head is not compared below)
    for o, keys in ((out, lambda t: ref.block_keys(int(c.pos[t]), P, range(K), 2, c.max_pages)),
                    (out2, lambda t: list(range(int(c.pos[t]) + 1))), (out3, lambda t: list(range(int(c.pos[t]) + 1)))):
        for t in range(0, T, 29):
            for h in range(Hkv):
                r, bound = c.rows(t, h, keys(t))
                err = (o[t, h * G:(h + 1) * G].cpu().double() - r).abs()
                rows = ~want[t, h * G:(h + 1) * G, 0]
                assert bool((err <= bound)[rows].all()), (t, h)


# --------------------------------------------------------------- infinities ---

@pytest.mark.parametrize("D,P,Hkv,G,lens,new", [
    (128, 64, 8, 1, [16384], 1300), (64, 16, 4, 4, [4001, 2500], 600), (128, 16, 8, 2, [5001], 700),  # chunks
    (128, 64, 8, 8, [4000, 700, 64, 2222], 1), (64, 16, 2, 3, [777, 300], 2), (128, 32, 1, 64, [3000], 1),
])
def test_scores_of_infinite_means_and_sums(D, P, Hkv, G, lens, new):
    c = Case(52, lens, D, P, Hkv, G)
    at = [(b, p) for b, n in enumerate(lens) for p in range(max(n - new, 0), n)]
    c.tokens([b for b, _ in at], [p for _, p in at])
    mean = (torch.randn(c.total, Hkv, D, generator=c.g) / 8).bfloat16()
    r = np.random.RandomState(7)
    for b, n in enumerate(lens):
        for j in range(0, n // P, 3):  # one infinite value of a mean, and two (the score may be NaN)
            mean[int(c.table[b, j]), r.randint(Hkv), r.randint(D)] = float("inf") * (1 if j % 2 else -1)
            if j % 4 == 0:
                mean[int(c.table[b, j]), r.randint(Hkv), r.randint(D)] = float("inf")
    # the last token's queries of the last KV head: one value infinite
    c.q[-1, -1, 5] = float("-inf")
    mean[:, :, 5] = mean[:, :, 5] + 0.01
    c.upload()
    scores = torch.full((c.T, Hkv, c.max_pages), 9.0, device=DEV)
    ws = sb.new_paged_workspace(c.pa)
    sb.sa_page_scores(c.pa, c.d["q"], mean.to(DEV), scores, ws)
    status_ok(ws)
    got, q, kinds = scores.cpu().double(), c.q.double().view(c.T, Hkv, G, D), [0, 0, 0]
    for b, n in enumerate(lens):
        tok = [t for t in range(c.T) if int(c.seq[t]) == b]
        k = mean[c.table[b, :n // P].long()].double().transpose(0, 1)
        s = torch.einsum("thd,hjd->thj", q[tok].sum(2), k) * c.scale
        # as check_scores: G sums and D products in fp32
        bound = torch.einsum("thd,hjd->thj", q[tok].abs().sum(2), k.abs()) * c.scale * (G + D + 4) * 2.0 ** -23
        live = (torch.arange(n // P)[None] < ((c.pos[tok] + 1) // P)[:, None])[:, None].expand(-1, Hkv, -1)
        row = got[tok][..., :n // P]
        nan, inf = torch.isnan(s), torch.isinf(s)
        assert torch.equal(torch.isnan(row)[live], nan[live])
        assert torch.equal(row[live & inf], s[live & inf])
        fine = live & ~nan & ~inf
        assert bool(((row - s).abs() <= bound)[fine].all())
        kinds = [x + int(y[live].sum()) for x, y in zip(kinds, (nan, inf, fine))]
    assert kinds[1] > 0 and (kinds[2] > 0 or c.T * Hkv == 1)
