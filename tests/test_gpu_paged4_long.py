"""The 4-bit cache at the lengths and batches that its pipelines reach their steady state
at: rings and windows of page ids that come round, CTAs and warps with parts of
several heads and sequences, more tokens than a CTA has threads, against float64 on the
device with bounds that a lost group of 32 slots shows through (tests/paged4_bounds.py)."""
import numpy as np
import pytest
import torch

import paged4_bounds as pb
from indexer_selected_sparse_score_gb300 import binding as sb

pytestmark = pytest.mark.gpu
DEV = "cuda"
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


class Big:
    """A cache made on the device: codes of any kind, scales of 1/4 .. 15/16, pages in
    shuffled order; slots past a sequence's end, and pages without a name, have NaN
    scales.  lost: the share of pages that the table does not name."""

    def __init__(self, seed, lens, D=128, P=64, Hkv=2, G=8, lost=0.0):
        r = np.random.RandomState(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.B, self.D, self.P, self.Hkv, self.G, self.H = len(lens), D, P, Hkv, G, Hkv * G
        self.lens, self.g, self.r = np.asarray(lens), g, r
        need = -(-self.lens // P)
        self.max_pages, self.total = int(need.max()) + 1, int(need.sum()) + 1
        perm, at = r.permutation(self.total), 0
        table = np.full((self.B, self.max_pages), -5, np.int64)
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        self.lost = lost > 0
        if lost:
            gone = r.uniform(size=table.shape) < lost
            table[gone & (table >= 0)] = r.choice([-1, self.total, 1 << 30])
        self.table = torch.from_numpy(table).to(DEV)
        shape = (self.total, Hkv, P)
        self.cache = [torch.randint(0, 256, shape + (D // 2,), dtype=torch.uint8, generator=g, device=DEV) for _ in range(2)]
        self.scales = [torch.randint(0x28, 0x38, shape + (D // 16,), dtype=torch.uint8, generator=g, device=DEV) for _ in range(2)]
        for b, n in enumerate(need):  # the rest of the last page
            page, used = table[b, n - 1], int(self.lens[b]) - (n - 1) * P
            if 0 <= page < self.total and used < P:
                for s in self.scales:
                    s[page, :, used:] = 0x7F
        self.scale = float(np.float32(0.4 * D ** -0.5))

    def tokens(self, seq, pos):
        self.seq, self.pos, self.T = np.asarray(seq), np.asarray(pos), len(seq)
        dev = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).to(DEV)  # noqa: E731
        self.q = torch.randn(self.T, self.H, self.D, generator=self.g, device=DEV).bfloat16()
        self.args = [dev(self.seq), dev(self.pos), self.table.int()]
        self.pa = sb.paged4_args(*self.args, self.H, self.Hkv, self.D, self.P, self.total, *self.cache, *self.scales, self.scale)
        self.ws = sb.new_paged4_workspace(self.pa)
        valid = (self.seq >= 0) & (self.seq < self.B) & (self.pos >= 0) & (self.pos < self.max_pages * self.P)
        self.valid = valid
        self.status = sb.SA_ERR_DEVICE_DATA if self.lost or not valid.all() else sb.SA_OK
        return self

    def rows(self, b, h, n):
        """Keys and values of n slots of one sequence and head in float64, and which of them are in a page."""
        page = self.table[b, :-(-n // self.P)]
        ok = (page >= 0) & (page < self.total)
        page = torch.where(ok, page, 0)
        e2m1 = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=DEV)
        out = []
        for c, s in zip(self.cache, self.scales):
            c, s = c[page, h].flatten(0, 1)[:n], s[page, h].flatten(0, 1)[:n]
            x = e2m1[torch.stack([c & 15, c >> 4], dim=-1).flatten(-2).long()]
            out.append(x * s.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=-1))
        ok = ok.repeat_interleave(self.P)[:n]
        return torch.where(ok[:, None], out[0], 0.0), torch.where(ok[:, None], out[1], 0.0), ok

    def check(self, weights=True):
        """Attention, log-sums and slot weights of the call."""
        out = torch.full_like(self.q, 7.0)
        lse = torch.full((self.T, self.H), 7.0, device=DEV)
        sb.sa_paged4_attn(self.pa, self.q, out, self.ws, lse=lse)
        assert sb.sa_check_device_status(self.ws) == self.status
        w0 = torch.rand(self.B, self.Hkv, self.max_pages * self.P + 3, generator=self.g, device=DEV)
        w = w0.clone()
        if weights:
            sb.sa_paged4_weights(self.pa, self.q, lse, w, self.ws)
            assert sb.sa_check_device_status(self.ws) == self.status
        skipped = torch.from_numpy(~self.valid).to(DEV)
        assert (out[skipped] == 7).all() and (lse[skipped] == 7).all()
        first_w, G = w0.double(), self.G
        touched = torch.zeros_like(w0, dtype=torch.bool)
        for b in range(self.B):
            at = np.nonzero(self.valid & (self.seq == b))[0]
            if not len(at):
                continue
            n = int(self.pos[at].max()) + 1
            pos = torch.from_numpy(self.pos[at]).to(DEV)
            at = torch.from_numpy(at).to(DEV)
            for h in range(self.Hkv):
                k, v, ok = self.rows(b, h, n)
                slots = torch.arange(n, device=DEV)
                sl = slice(h * G, (h + 1) * G)
                gained, off = torch.zeros(n, dtype=torch.float64, device=DEV), torch.zeros(n, dtype=torch.float64, device=DEV)
                for i in range(0, len(at), 128):
                    rows, last = at[i:i + 128], pos[i:i + 128]
                    q = self.q[rows, sl].double().flatten(0, 1)
                    seen = ((slots <= last[:, None]) & ok).repeat_interleave(G, dim=0)
                    o, l, spread, eps, p = pb.attention(q, k, v, seen, self.scale)
                    empty = ~seen.any(dim=1)
                    got, got_l = out[rows, sl].double().flatten(0, 1), lse[rows, sl].double().flatten()
                    assert (got[empty] == 0).all() and (got_l[empty] == -torch.inf).all(), (b, h)
                    err, bound = (got - o).norm(dim=-1), pb.row_bound(o, spread, eps, n)
                    assert (err <= bound)[~empty].all(), (b, h, i, float((err / bound)[~empty].max()))
                    err, bound = (got_l - l).abs(), pb.lse_bound(l, eps, n)
                    assert (err <= bound)[~empty].all(), (b, h, i, float((err / bound)[~empty].max()))
                    gained += p.sum(dim=0)
                    # a weight: logit and log-sum (as checked above) off, the exponential and its
                    # argument's rounding (arguments up to 32: 2^-18)
                    off += p.sum(dim=0) * (eps + float(bound[~empty].max() if (~empty).any() else 0) + 2.0 ** -18)
                if weights:
                    want = first_w[b, h, :n] + gained
                    bound = 1.01 * off + (len(at) * G + 8) * 2.0 ** -23 * want
                    err = (w[b, h, :n].double() - want).abs()
                    assert (err <= bound).all(), (b, h, float((err / bound).max()))
                    touched[b, h, :n] = True
        assert torch.equal(w[~touched], w0[~touched])
        again, again_l = torch.empty_like(out).fill_(7.0), torch.empty_like(lse).fill_(7.0)
        sb.sa_paged4_attn(self.pa, self.q, again, self.ws, lse=again_l)
        assert torch.equal(again, out) and torch.equal(again_l, lse)
        sb.sa_check_device_status(self.ws)


def _lens(seed, B, lo, hi):
    return np.random.RandomState(seed).randint(lo, hi + 1, size=B)


def _last(lens, new):
    seq = np.repeat(np.arange(len(lens)), new)
    return seq, np.concatenate([np.arange(n - new, n) for n in lens])


@pytest.mark.parametrize("D,P,G,lost", [(128, 64, 8, 0), (128, 16, 8, 0.02), (64, 128, 4, 0), (64, 16, 8, 0.02), (128, 32, 16, 0.02),
                                        (64, 64, 12, 0)])
def test_decode_steps_of_long_contexts(D, P, G, lost):
    lens = _lens(1, 64, 8192, 16383)
    Big(1, lens, D, P, 8, G, lost).tokens(*_last(lens, 1)).check()


@pytest.mark.parametrize("D,P,G,lost", [(128, 64, 4, 0), (128, 16, 3, 0.02), (64, 32, 4, 0)])
def test_drafted_tokens_of_long_contexts(D, P, G, lost):
    lens = _lens(2, 24, 8192, 16383)
    Big(2, lens, D, P, 8, G, lost).tokens(*_last(lens, 4)).check()


@pytest.mark.parametrize("D,P,G,lost", [(128, 64, 64, 0), (128, 16, 48, 0.02), (64, 128, 128, 0), (64, 16, 24, 0.02), (128, 128, 96, 0)])
def test_many_heads_over_one_of_long_contexts(D, P, G, lost):
    lens = _lens(3, 48, 16384, 40000)
    Big(3, lens, D, P, 1, G, lost).tokens(*_last(lens, 1)).check()


@pytest.mark.parametrize("D,P,Hkv,G,B,new,lost", [(128, 128, 4, 8, 2, 700, 0), (128, 16, 2, 8, 6, 330, 0.02), (64, 64, 8, 4, 6, 300, 0),
                                                  (64, 16, 4, 16, 3, 200, 0.02), (128, 64, 8, 3, 4, 410, 0.02)])
def test_chunks_of_long_prompts(D, P, Hkv, G, B, new, lost):
    lens = _lens(4, B, 9000, 12000)
    Big(4, lens, D, P, Hkv, G, lost).tokens(*_last(lens, new)).check()


def _in_any_order(seed, lens, new, bad):
    """`new` tokens of every sequence, next to one another, the sequences shuffled; and skipped ones between."""
    r = np.random.RandomState(seed)
    tok = []
    for b in r.permutation(len(lens)):
        first = max(0, lens[b] - new)
        tok += [(b, p) for p in range(first, lens[b])]
        if bad and r.uniform() < 0.1:
            tok += [(-1, 3), (len(lens), 0), (b, -1)][:r.randint(1, 4)]
    return np.array(tok).T


@pytest.mark.parametrize("B,new,D,P,Hkv,G,bad", [
    (300, 1, 128, 64, 2, 8, False),   # more than 256 tokens of at most 64 columns
    (700, 1, 64, 16, 1, 4, True),     # more tokens than a CTA has threads, several groups of 32 a warp
    (1100, 1, 128, 32, 1, 16, True),
    (257, 1, 128, 64, 2, 1, False),
    (90, 3, 128, 64, 2, 8, True),     # three drafted tokens of 90 sequences
    (65, 2, 128, 64, 2, 8, False),    # units of two tokens, more than 64 of them
    (120, 2, 128, 16, 1, 8, True),    # .. more tokens than threads of 192 a CTA
    (150, 2, 64, 32, 2, 8, True),     # .. than of 256
    (400, 4, 64, 64, 1, 2, True),
    (130, 5, 128, 64, 1, 3, True),
    (260, 1, 128, 64, 1, 40, True),   # many columns, one token each
    (90, 7, 64, 64, 2, 8, True),
    (300, 3, 128, 64, 1, 48, True),   # units of 144 columns
])
def test_large_batches_of_short_sequences(B, new, D, P, Hkv, G, bad):
    lens = _lens(5, B, max(1, new - 1), 700)
    Big(5, lens, D, P, Hkv, G).tokens(*_in_any_order(6, lens, new, bad)).check()


@pytest.mark.parametrize("new,G", [(1, 8), (2, 8), (1, 32), (5, 16)])
def test_a_padded_and_a_mixed_batch(new, G):
    """A table of 64 rows with 8 live sequences, and decode steps beside a prompt's chunk."""
    lens = np.concatenate([_lens(7, 8, 500, 3000), np.ones(56, int)])
    seq, pos = _last(lens[:8], new)
    pad = 64 * new - len(seq)
    c = Big(7, lens, 128, 64, 2, G)
    c.tokens(np.concatenate([seq, np.full(pad, -1)]), np.concatenate([pos, np.zeros(pad, int)])).check()
    lens = np.concatenate([_lens(8, 40, 100, 900), [1500], _lens(9, 22, 100, 900)])
    seq, pos = _last(lens, 1)
    cut = int(np.nonzero(seq == 40)[0][0])
    chunk = np.arange(1500 - 200 * new, 1500)
    c = Big(8, lens, 128, 64, 2, G)
    c.tokens(np.concatenate([seq[:cut], np.full(len(chunk), 40), seq[cut + 1:]]),
             np.concatenate([pos[:cut], chunk, pos[cut + 1:]])).check()


def test_evictions_in_turn_leave_exactly_the_budget():
    budget, recent, B, Hkv = 96, 16, 200, 2
    now = _lens(10, B, 0, 300)
    c = Big(9, np.full(B, 400), 64, 32, Hkv, 1).tokens([], [])
    ld = c.max_pages * c.P
    weight = torch.rand(B, Hkv, ld, generator=c.g, device=DEV)
    born = torch.arange(ld, dtype=torch.int32, device=DEV).repeat(B, Hkv, 1)
    newest = torch.from_numpy(now.astype(np.int32)).to(DEV) - 1
    for more in (0, 1, 7, 1, 60):
        now, newest = now + more, newest + more
        length, left = torch.from_numpy(now.astype(np.int32)).to(DEV), torch.full((B,), -1, dtype=torch.int32, device=DEV)
        for b in range(B):  # the new slots' records
            born[b, :, now[b] - more:now[b]] = newest[b] + 1 - more + torch.arange(more, dtype=torch.int32, device=DEV)
            weight[b, :, now[b] - more:now[b]] = 0
        wo, bo = weight.clone(), born.clone()
        sb.sa_paged4_evict(c.pa, length, newest, budget, recent, weight, born, wo, bo, left, c.ws)
        assert sb.sa_check_device_status(c.ws) == sb.SA_OK
        assert left.tolist() == np.minimum(now, budget).tolist()
        for b in range(0, B, 17):
            n, keep = int(now[b]), min(int(now[b]), budget)
            for h in range(Hkv):
                w, t = weight[b, h, :n].cpu().numpy().astype(np.float64), born[b, h, :n].cpu().numpy()
                w[t > int(newest[b]) - recent] = np.inf
                best = sorted(t[np.lexsort((np.arange(n), -w))[:keep]].tolist())
                assert sorted(bo[b, h, :keep].tolist()) == best
        now, weight, born = np.minimum(now, budget), wo, bo
