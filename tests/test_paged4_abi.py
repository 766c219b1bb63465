"""Argument checks of the 4-bit paged calls (no GPU needed): a bad argument returns
its error before anything is enqueued, and the Python calls refuse tensors that
the library would misread."""
import ctypes

import pytest
import torch

from indexer_selected_sparse_score_gb300 import binding, build

INV, UNS, WS = binding.SA_ERR_INVALID_ARG, binding.SA_ERR_UNSUPPORTED, binding.SA_ERR_WORKSPACE
OK = binding.SA_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _pa(**kw):
    base = dict(B=2, T=3, H=16, H_kv=2, D=128, P=64, n_pages=10, max_pages=5, q_seq=16, q_pos=16, page_table=16,
                table_stride=0, K=256, V=256, scale=0.088)
    more = dict(K_scale=256, V_scale=256, k_gain=1.0, v_gain=1.0)
    for k, v in kw.items():
        (more if k in more else base)[k] = v
    p = binding.PagedArgs(*[base[f] for f, _ in binding.PagedArgs._fields_])
    return binding.Paged4Args(p, more["K_scale"], more["V_scale"], more["k_gain"], more["v_gain"])


def _ref(pa):
    return ctypes.byref(pa) if pa is not None else None


BIG = 1 << 40


def _append(lib, pa, **kw):
    a = dict(k=256, ks=0, v=256, vs=0, q=None, qs=0, qo=None, rope=None, halves=0, turn=None, w=None, b=None, ld=320,
             ws=256, nb=BIG)
    a.update(kw)
    return lib.sa_paged4_append(_ref(pa), a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["qo"],
                                ctypes.byref(a["rope"]) if a["rope"] is not None else None, a["halves"], a["turn"],
                                a["w"], a["b"], a["ld"], a["ws"], a["nb"], None)


def _read(lib, pa, **kw):
    a = dict(k=256, v=256, ws=256, nb=BIG)
    a.update(kw)
    return lib.sa_paged4_read(_ref(pa), a["k"], a["v"], a["ws"], a["nb"], None)


def _attn(lib, pa, **kw):
    a = dict(q=256, out=256, lse=None, ws=256, nb=BIG)
    a.update(kw)
    return lib.sa_paged4_attn(_ref(pa), a["q"], a["out"], a["lse"], a["ws"], a["nb"], None)


def _weights(lib, pa, **kw):
    a = dict(q=256, lse=256, w=256, ld=320, ws=256, nb=BIG)
    a.update(kw)
    return lib.sa_paged4_weights(_ref(pa), a["q"], a["lse"], a["w"], a["ld"], a["ws"], a["nb"], None)


def _evict(lib, pa, **kw):
    a = dict(n=4096, new=8192, budget=100, recent=10, w=1 << 20, b=2 << 20, wo=3 << 20, bo=4 << 20, ld=320, no=16384,
             ws=256, nb=BIG)
    a.update(kw)
    return lib.sa_paged4_evict(_ref(pa), a["n"], a["new"], a["budget"], a["recent"], a["w"], a["b"], a["wo"], a["bo"],
                               a["ld"], a["no"], a["ws"], a["nb"], None)


CALLS = (_append, _read, _attn, _weights, _evict)

SHAPES = [
    (None, INV),
    (dict(B=0), INV), (dict(H=15), INV), (dict(n_pages=0), INV), (dict(max_pages=0), INV),
    (dict(D=96), UNS), (dict(D=512), UNS), (dict(P=48), UNS), (dict(P=8), UNS),
    (dict(H=258, H_kv=2), UNS), (dict(n_pages=1 << 24, H_kv=2), UNS), (dict(max_pages=(1 << 24) + 1), UNS),
    (dict(table_stride=4), INV), (dict(page_table=17), INV), (dict(page_table=None), INV),
    (dict(k_gain=0.0), INV), (dict(v_gain=3.0), INV), (dict(k_gain=-1.0), INV), (dict(v_gain=float("inf")), INV),
    (dict(k_gain=float("nan")), INV), (dict(k_gain=2.0 ** -61), INV), (dict(v_gain=2.0 ** 61), INV),
    (dict(K=None), INV), (dict(K_scale=None), INV), (dict(K=264), INV), (dict(K_scale=257), INV), (dict(V_scale=8), INV),
]


@pytest.mark.parametrize("kw,status", SHAPES)
def test_shapes_are_checked_by_every_call(lib, kw, status):
    pa = None if kw is None else _pa(**kw)
    for call in CALLS:
        assert call(lib, pa) == status, call.__name__
    pointers = kw is not None and (set(kw) & {"K", "K_scale", "page_table"}) and None in kw.values()
    if not pointers:
        assert lib.sa_paged4_workspace_size(_ref(pa)) == 0


def test_value_pointers(lib):
    for kw in (dict(V=None), dict(V_scale=None)):
        for call in (_append, _read, _attn, _evict):
            assert call(lib, _pa(**kw)) == INV
    assert _read(lib, _pa(T=0, V=None), v=None) == OK         # keys alone
    for call in (_append, _read, _attn, _weights):
        for kw in (dict(T=-1), dict(q_seq=None), dict(q_pos=None), dict(q_seq=18)):
            assert call(lib, _pa(**kw)) == INV
        assert call(lib, _pa(T=1 << 27)) == UNS


def test_gains_at_the_ends(lib):
    for g in (2.0 ** -60, 0.5, 2.0 ** 60):
        assert lib.sa_paged4_workspace_size(_ref(_pa(k_gain=g, v_gain=g))) > 4096


def test_append_arguments(lib):
    pa = _pa()
    rope = binding.RopeArgs(32, 10000.0, 1.0, 0, 32.0, 1.0)
    for kw in (dict(k=None), dict(v=None), dict(k=264), dict(ks=128), dict(ks=260), dict(vs=-8), dict(q=256), dict(qo=256),
               dict(q=264, qo=256), dict(turn=257), dict(w=256), dict(b=256), dict(w=256, b=256, ld=319),
               dict(w=258, b=256), dict(w=256, b=257), dict(ws=264)):
        assert _append(lib, pa, **kw) == INV, kw
    for dim in (16, 48, -32, 160):
        assert _append(lib, pa, rope=binding.RopeArgs(dim, 10000.0, 1.0, 0, 32.0, 1.0)) == INV
    assert _append(lib, pa, rope=binding.RopeArgs(32, 1.0, 1.0, 0, 32.0, 1.0)) == INV
    assert _append(lib, pa, rope=rope, ws=None) == WS
    assert _append(lib, pa, rope=rope, nb=255) == WS
    assert _append(lib, _pa(T=0, K=None, V=None, K_scale=None, V_scale=None), k=None, v=None) == OK


def test_read_attention_and_weights_arguments(lib):
    pa = _pa()
    need = lib.sa_paged4_workspace_size(_ref(pa))
    assert _read(lib, pa, k=264) == INV and _read(lib, pa, v=257) == INV and _read(lib, pa, ws=None) == WS
    for kw in (dict(q=None), dict(q=264), dict(out=None), dict(out=258), dict(lse=258), dict(ws=8)):
        assert _attn(lib, pa, **kw) == INV, kw
    for kw in (dict(q=None), dict(q=264), dict(lse=None), dict(lse=258), dict(w=None), dict(w=257), dict(ld=319)):
        assert _weights(lib, pa, **kw) == INV, kw
    for bad in (float("nan"), float("inf")):
        assert _attn(lib, _pa(scale=bad)) == INV and _weights(lib, _pa(scale=bad)) == INV
    assert _attn(lib, pa, nb=4096) == WS and _weights(lib, pa, nb=4096) == WS and _attn(lib, pa, ws=None) == WS
    assert need > 4096


def test_evict_arguments(lib):
    pa = _pa()
    for kw in (dict(n=None), dict(new=None), dict(w=None), dict(b=None), dict(wo=None), dict(bo=None), dict(no=None),
               dict(budget=0), dict(budget=-3), dict(recent=-1), dict(recent=101), dict(ld=319), dict(n=4097),
               dict(w=(1 << 20) + 2), dict(bo=(4 << 20) + 1),
               dict(wo=1 << 20), dict(bo=2 << 20), dict(wo=2 << 20), dict(bo=1 << 20), dict(bo=3 << 20),
               dict(wo=(1 << 20) + 16), dict(no=4096), dict(no=8196)):
        assert _evict(lib, pa, **kw) == INV, kw
    assert _evict(lib, pa, ws=None) == WS and _evict(lib, pa, nb=4095) == WS
    assert _evict(lib, _pa(B=1 << 20, H_kv=128, H=128, n_pages=1)) == UNS


# ----------------------------------------------------------- Python calls ---

def _args(B=2, T=3, H=4, Hkv=2, D=64, P=16, n=6, mp=3, **kw):
    u8 = torch.uint8
    t = dict(seq=torch.zeros(T, dtype=torch.int32), pos=torch.zeros(T, dtype=torch.int32),
             table=torch.zeros(B, mp, dtype=torch.int32), K=torch.zeros(n, Hkv, P, D // 2, dtype=u8),
             V=torch.zeros(n, Hkv, P, D // 2, dtype=u8), Ks=torch.zeros(n, Hkv, P, D // 16, dtype=u8),
             Vs=torch.zeros(n, Hkv, P, D // 16, dtype=u8))
    t.update(kw)
    return binding.paged4_args(t["seq"], t["pos"], t["table"], H, Hkv, D, P, n, t["K"], t["V"], t["Ks"], t["Vs"], 0.1)


def test_python_cache_tensors():
    pa = _args()
    assert pa.p.B == 2 and pa.p.max_pages == 3 and pa.k_gain == 1.0
    scales = torch.zeros(6, 2, 16, 4).to(torch.float8_e4m3fn)
    assert _args(Ks=scales, Vs=scales).K_scale == scales.data_ptr()
    u8 = torch.uint8
    for kw in (dict(K=torch.zeros(6, 2, 16, 64, dtype=u8)), dict(K=torch.zeros(6, 2, 16, 32)),
               dict(Ks=torch.zeros(6, 2, 16, 4)), dict(V=torch.zeros(6, 16, 2, 32, dtype=u8)),
               dict(Vs=torch.zeros(6, 2, 16, 8, dtype=u8)[..., ::2]), dict(K=torch.zeros(5, 2, 16, 32, dtype=u8)),
               dict(seq=torch.zeros(3, dtype=torch.int64)), dict(pos=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(binding.SAError):
            _args(**kw)


def test_python_calls_refuse_what_would_be_misread():
    pa, ws = _args(), torch.zeros(1 << 20, dtype=torch.uint8)
    bf = torch.bfloat16
    k = torch.zeros(3, 2, 64, dtype=bf)
    q, lse = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 4)
    w, b = torch.zeros(2, 2, 48), torch.zeros(2, 2, 48, dtype=torch.int32)
    n = torch.zeros(2, dtype=torch.int32)

    def refused(f, *a, **kw):
        with pytest.raises(binding.SAError) as e:
            f(*a, stream=0, **kw)
        assert e.value.status == INV

    for bad in (k.float(), k[:2], k[:, :1].expand(3, 2, 64), k.transpose(0, 1)):
        refused(binding.sa_paged4_append, pa, bad, k, ws)
        refused(binding.sa_paged4_append, pa, k, bad, ws)
    refused(binding.sa_paged4_append, pa, k, k, ws, rope_pos=torch.zeros(3, dtype=torch.int64))
    refused(binding.sa_paged4_append, pa, k, k, ws, rope_pos=torch.zeros(2, dtype=torch.int32))
    refused(binding.sa_paged4_append, pa, k, k, ws, weight=w, born=w)
    refused(binding.sa_paged4_append, pa, k, k, ws, weight=w[:1], born=b)
    refused(binding.sa_paged4_append, pa, k, k, ws, weight=w, born=torch.zeros(2, 2, 50, dtype=torch.int32))
    refused(binding.sa_paged4_append, pa, k, k, ws, weight=w[..., ::2], born=b[..., ::2])
    refused(binding.sa_paged4_append, pa, k, k, ws, weight=w[..., :24].contiguous(), born=b[..., :24].contiguous())
    refused(binding.sa_paged4_append, pa, k, k, ws, weight=w)
    refused(binding.sa_paged4_read, pa, k.float(), k, ws)
    refused(binding.sa_paged4_read, pa, k[:2], None, ws)
    for out in (q.float(), q[:, :3], q.transpose(0, 1)):
        refused(binding.sa_paged4_attn, pa, q, out, ws)
        refused(binding.sa_paged4_attn, pa, out, q, ws)
    refused(binding.sa_paged4_attn, pa, q, q.clone(), ws, lse=lse.double())
    refused(binding.sa_paged4_attn, pa, q, q.clone(), ws, lse=lse[:2])
    refused(binding.sa_paged4_weights, pa, q, lse[:, :2], w, ws)
    refused(binding.sa_paged4_weights, pa, q, lse, w.double(), ws)
    refused(binding.sa_paged4_weights, pa, q, lse, w.view(4, 48), ws)
    good = [n, n + 5, 4, 1, w, b, w.clone(), b.clone(), n.clone()]
    for i, bad in ((0, n.long()), (0, n[:1]), (1, n.float()), (2, 0), (3, 5), (4, w[:1]), (4, w.half()), (5, w),
                   (6, torch.zeros(2, 2, 49)), (6, w), (7, b), (8, n[:1]), (8, n)):
        a = list(good)
        a[i] = bad
        if i == 6 and bad is w:
            a[4] = w
        refused(binding.sa_paged4_evict, pa, *a[:9], ws)


def test_every_call_is_exported():
    for name in ("sa_paged4_append", "sa_paged4_read", "sa_paged4_attn", "sa_paged4_weights", "sa_paged4_evict",
                 "sa_paged4_workspace_size"):
        assert name in binding.EXPORTED and hasattr(binding, name)
