"""One workspace for calls of every kind in turn, as include/sa.h allows: what the
4-bit attention keeps in its header between calls is no other call's scratch."""
import pytest
import torch

from gpu_run import ensure_built
from indexer_selected_sparse_score_gb300 import binding as sb
from indexer_selected_sparse_score_gb300 import workloads as wl
from test_gpu_paged import Case as Case16
from test_gpu_paged4 import Case as Case4, step
from tolerances import check_attn

pytestmark = pytest.mark.gpu
DEV = "cuda"
HEADER = 4096


class Others:
    """The calls of the 16-bit cache and the fused step, on a workspace that is given."""

    def __init__(self):
        lens = [700, 1500, 96, 333]
        self.c = c = Case16(3, lens, P=16, Hkv=2, G=8, shared=4, poison=False).tokens(*step(lens)).upload()
        self.out = c.out()
        self.mean = torch.randn(c.total, c.Hkv, c.D, generator=c.g).bfloat16().to(DEV)
        pages = torch.arange(8, dtype=torch.int32)
        has = c.pos[:, None] // c.P + 1 > pages  # (the 96 positions have six)
        self.idx = torch.where(has, pages, -1)[:, None].expand(c.T, c.Hkv, 8).contiguous().to(DEV)
        self.picks = torch.zeros(c.T, c.Hkv, 8, dtype=torch.int32, device=DEV)
        self.scores = torch.zeros(c.T, c.Hkv, c.max_pages, device=DEV)
        w = wl.generate(wl.CONFIGS["c1"])
        self.dp = sb.upload(w)
        self.step_out = torch.zeros(w.T, w.H, w.D, dtype=torch.bfloat16, device=DEV)
        self.bytes = max(sb.sa_paged_workspace_size(c.pa, 8, 2, 4), sb.sa_paged_workspace_size(c.pa, 0, 0, 0),
                         sb.sa_workspace_size(self.dp.ia, self.dp.aa, self.dp.K))

    def calls(self):
        c, d = self.c, self.dp
        return {
            "prefix": lambda ws: sb.sa_prefix_attn(c.pa, c.d["q"], 4, self.out, ws),
            "whole": lambda ws: sb.sa_prefix_attn(c.pa, c.d["q"], 0, self.out, ws),
            "block": lambda ws: sb.sa_block_attn(c.pa, c.d["q"], self.idx, 8, 2, self.out, ws),
            "fused": lambda ws: sb.sa_fused_block_attn(c.pa, c.d["q"], self.mean, 8, 2, self.picks, self.out, ws),
            "scores": lambda ws: sb.sa_page_scores(c.pa, c.d["q"], self.mean, self.scores, ws),
            "step": lambda ws: sb.sa_fused_decode(d.ia, d.aa, d.K, None, self.step_out, ws),
        }


@pytest.fixture(scope="module")
def others():
    ensure_built()
    return Others()


def _workspace(n):
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)
    sb.sa_workspace_init(ws)
    return ws


def test_no_call_writes_into_the_header(others):
    lens = [900, 33, 3000]
    small = [Case4(1, lens, G=G, Hkv=1).tokens(*step(lens)).upload() for G in (8, 16, 48)]
    n = max([others.bytes] + [sb.sa_paged4_workspace_size(c.pa) for c in small])
    ws = _workspace(n)
    calls = dict(others.calls())
    for i, c in enumerate(small):
        out, lse = torch.zeros_like(c.d["q"]), torch.zeros(c.T, c.H, device=DEV)
        weight = torch.zeros(c.B, c.Hkv, c.max_pages * c.P, device=DEV)
        born = torch.zeros_like(weight, dtype=torch.int32)
        left = torch.tensor(lens, dtype=torch.int32, device=DEV)
        calls[f"attn4 {i}"] = lambda ws, c=c, out=out, lse=lse: sb.sa_paged4_attn(c.pa, c.d["q"], out, ws, lse=lse)
        calls[f"weights4 {i}"] = lambda ws, c=c, lse=lse, weight=weight: sb.sa_paged4_weights(c.pa, c.d["q"], lse, weight, ws)
        calls[f"evict4 {i}"] = lambda ws, c=c, weight=weight, born=born, left=left: sb.sa_paged4_evict(
            c.pa, left, left - 1, 30, 3, weight, born, torch.zeros_like(weight), torch.zeros_like(born),
            torch.zeros_like(left), ws)
    for name, call in calls.items():
        call(ws)
        assert sb.sa_check_device_status(ws) == sb.SA_OK, name
        assert not ws[:HEADER].any(), name


@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("lens", [[3000], [40000], [2000, 900, 17, 1200], [30000, 5, 12000]])
def test_attention_in_turn_with_other_calls(others, G, lens):
    """Units cut into fewer and into more than 16 parts, eagerly and from a graph."""
    c = Case4(2, lens, G=G, Hkv=1).tokens(*step(lens)).upload()
    out, lse = c.attn()
    c.check_attn(out, lse)
    ws = _workspace(max(others.bytes, sb.sa_paged4_workspace_size(c.pa)))
    got, got_l = torch.zeros_like(out), torch.zeros_like(lse)

    def mine():
        sb.sa_paged4_attn(c.pa, c.d["q"], got, ws, lse=got_l)

    def check(what):
        assert sb.sa_check_device_status(ws) == sb.SA_OK, what
        assert torch.equal(got, out) and torch.equal(got_l, lse), what
        got.fill_(7)
        got_l.fill_(7)

    for name, call in others.calls().items():
        call(ws)
        mine()
        check(name)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(ws)
            mine()
        for _ in range(2):
            g.replay()
            check(name + ", graph")


def test_the_other_calls_give_the_same_on_a_shared_workspace(others):
    lens = [40000]
    c = Case4(3, lens, G=8, Hkv=1).tokens(*step(lens)).upload()
    out, lse = torch.zeros_like(c.d["q"]), torch.zeros(c.T, c.H, device=DEV)
    n = max(others.bytes, sb.sa_paged4_workspace_size(c.pa))
    shared = _workspace(n)
    buffers = (others.out, others.picks, others.scores, others.step_out)

    def results(call, ws):
        for x in buffers:
            x.zero_()
        call(ws)
        return [x.clone() for x in buffers]
    for name, call in others.calls().items():
        want = results(call, _workspace(n))
        sb.sa_paged4_attn(c.pa, c.d["q"], out, shared, lse=lse)
        got = results(call, shared)
        assert sb.sa_check_device_status(shared) == sb.SA_OK, name
        if name == "step":
            check_attn(got[3].double().cpu().numpy(), want[3].double().cpu().numpy())
        else:
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
