"""Argument checks of the paged-cache calls (no GPU needed): a bad argument
returns its error before anything is enqueued."""
import ctypes

import pytest

from indexer_selected_sparse_score_gb300 import binding, build

INV, UNS, WS = binding.SA_ERR_INVALID_ARG, binding.SA_ERR_UNSUPPORTED, binding.SA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _pa(**kw):
    base = dict(B=2, T=3, H=16, H_kv=2, D=128, P=64, n_pages=10, max_pages=5, q_seq=16, q_pos=16, page_table=16,
                table_stride=0, K=256, V=256, scale=0.088)
    base.update(kw)
    return binding.PagedArgs(*[base[f] for f, _ in binding.PagedArgs._fields_])


def _ref(pa):
    return ctypes.byref(pa) if pa is not None else None


SHAPES = [
    (None, INV),
    (dict(B=0), INV), (dict(T=-1), INV), (dict(H=0), INV), (dict(H_kv=0), INV), (dict(H=15), INV),
    (dict(n_pages=0), INV), (dict(max_pages=0), INV),
    (dict(D=96), UNS), (dict(D=512), UNS), (dict(P=48), UNS), (dict(P=8), UNS), (dict(P=256), UNS),
    (dict(H=258, H_kv=2), UNS),                       # 129 heads per KV head
    (dict(n_pages=1 << 24, H_kv=2), UNS),             # 2^31 cache rows
    (dict(max_pages=(1 << 24) + 1), UNS),             # positions past 2^30
    (dict(T=1 << 27), UNS),
    (dict(table_stride=4), INV), (dict(table_stride=-5), INV),
    (dict(q_seq=None), INV), (dict(q_pos=None), INV), (dict(page_table=None), INV),
    (dict(q_seq=18), INV), (dict(page_table=17), INV),
]
CACHE = [(dict(K=None), INV), (dict(V=None), INV), (dict(K=264), INV), (dict(V=257), INV)]


def _append(lib, pa, **kw):
    a = dict(k=256, ks=0, v=256, vs=0, q=None, qs=0, qo=None, rope=None, halves=0, mean=None, ws=256, nb=256)
    a.update(kw)
    return lib.sa_paged_append(_ref(pa), a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["qo"],
                               ctypes.byref(a["rope"]) if a["rope"] is not None else None, a["halves"], a["mean"],
                               a["ws"], a["nb"], None)


def _scores(lib, pa, **kw):
    a = dict(q=256, mean=256, scores=256, ld=5, ws=256, nb=256)
    a.update(kw)
    return lib.sa_page_scores(_ref(pa), a["q"], a["mean"], a["scores"], a["ld"], a["ws"], a["nb"], None)


def _block(lib, pa, **kw):
    a = dict(q=256, idx=256, K=4, local=1, out=256, ws=256, nb=1 << 30)
    a.update(kw)
    return lib.sa_block_attn(_ref(pa), a["q"], a["idx"], a["K"], a["local"], a["out"], a["ws"], a["nb"], None)


def _fused(lib, pa, **kw):
    a = dict(q=256, mean=256, K=4, local=1, idx=None, out=256, ws=256, nb=1 << 30)
    a.update(kw)
    return lib.sa_fused_block_attn(_ref(pa), a["q"], a["mean"], a["K"], a["local"], a["idx"], a["out"], a["ws"],
                                   a["nb"], None)


def _prefix(lib, pa, **kw):
    a = dict(q=256, shared=2, out=256, ws=256, nb=1 << 30)
    a.update(kw)
    return lib.sa_prefix_attn(_ref(pa), a["q"], a["shared"], a["out"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("kw,status", SHAPES)
def test_shapes_are_checked_by_every_call(lib, kw, status):
    pa = None if kw is None else _pa(**kw)
    for call in (_append, _scores, _block, _fused, _prefix):
        assert call(lib, pa) == status, call.__name__
        assert lib.sa_last_error_detail()
    assert lib.sa_paged_workspace_size(_ref(pa), 4, 1, 2) == 0


@pytest.mark.parametrize("kw,status", CACHE)
def test_cache_pointers_are_checked(lib, kw, status):
    for call in (_append, _block, _fused, _prefix):
        assert call(lib, _pa(**kw)) == status, call.__name__


def _rope(**kw):
    base = dict(dim=64, base=10000.0, factor=1.0, original_seq_len=0, beta_fast=32.0, beta_slow=1.0)
    base.update(kw)
    return binding.RopeArgs(*[base[f] for f, _ in binding.RopeArgs._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(k=264), INV), (dict(mean=8), INV),
    (dict(q=256), INV), (dict(qo=256), INV),                        # q and q_out go together
    (dict(q=256, qo=256, qs=16 * 128 + 8), INV),                    # in place needs dense queries
    (dict(ks=2 * 128 - 8), INV), (dict(vs=2 * 128 + 4), INV), (dict(q=256, qo=512, qs=128), INV), (dict(ks=-8), INV),
    (dict(rope=_rope(dim=72)), INV), (dict(rope=_rope(dim=144)), INV), (dict(rope=_rope(dim=-16)), INV),
    (dict(rope=_rope(base=1.0)), INV), (dict(rope=_rope(base=float("nan"))), INV), (dict(rope=_rope(factor=0.0)), INV),
    (dict(rope=_rope(original_seq_len=4096, beta_slow=0.0)), INV),
    (dict(ws=None), WS), (dict(nb=255), WS), (dict(ws=264), INV),
])
def test_append_rejects_bad_arguments(lib, kw, status):
    assert _append(lib, _pa(), **kw) == status
    assert lib.sa_last_error_detail()


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(mean=None), INV), (dict(scores=None), INV), (dict(scores=258), INV), (dict(ld=4), INV),
    (dict(q=264), INV), (dict(ws=None), WS), (dict(nb=128), WS),
])
def test_scores_reject_bad_arguments(lib, kw, status):
    assert _scores(lib, _pa(), **kw) == status


@pytest.mark.parametrize("call", [_block, _fused])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(out=None), INV), (dict(out=264), INV), (dict(K=-1), INV), (dict(local=-1), INV),
    (dict(idx=258), INV), (dict(ws=None), WS), (dict(nb=128), WS),
])
def test_block_attention_rejects_bad_arguments(lib, call, kw, status):
    assert call(lib, _pa(), **kw) == status


def test_block_attention_needs_a_list_and_the_fused_call_a_local_page(lib):
    assert _block(lib, _pa(), idx=None) == INV
    assert _fused(lib, _pa(), local=0) == INV
    assert _fused(lib, _pa(), mean=None) == INV


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(out=None), INV), (dict(shared=-1), INV), (dict(shared=6), INV), (dict(ws=None), WS),
    (dict(nb=128), WS),
])
def test_prefix_attention_rejects_bad_arguments(lib, kw, status):
    assert _prefix(lib, _pa(), **kw) == status


@pytest.mark.parametrize("scale", [float("nan"), float("inf")])
def test_scale_must_be_finite(lib, scale):
    for call in (_scores, _block, _fused, _prefix):
        assert call(lib, _pa(scale=scale)) == INV


def test_no_tokens_enqueue_nothing(lib):
    pa = _pa(T=0, q_seq=None, q_pos=None, page_table=None, K=None, V=None)
    assert _append(lib, pa, k=None, v=None) == binding.SA_OK
    assert _scores(lib, pa, q=None, mean=None, scores=None) == binding.SA_OK
    assert _block(lib, pa, q=None, idx=None, out=None) == binding.SA_OK
    assert _prefix(lib, pa, q=None, out=None) == binding.SA_OK


def test_workspace_grows_with_what_it_holds(lib):
    n = lib.sa_paged_workspace_size(_ref(_pa()), 0, 1, 0)
    assert n >= 256 and n % 256 == 0
    assert lib.sa_paged_workspace_size(_ref(_pa()), 4, 1, 0) > n
    assert lib.sa_paged_workspace_size(_ref(_pa()), -1, 1, 0) == 0
    assert lib.sa_paged_workspace_size(_ref(_pa()), 0, -1, 0) == 0
    assert lib.sa_paged_workspace_size(_ref(_pa()), 0, 0, 6) == 0


def test_strides_of_python_tensors():
    import torch
    bf = dict(dtype=torch.bfloat16)
    x = torch.zeros(4, 2, 128, **bf)
    assert binding._token_rows("k", x, 2, 128, 4) == (x.data_ptr(), 256)
    y = torch.zeros(4, 6, 128, **bf)[:, 1:3]
    assert binding._token_rows("k", y, 2, 128, 4) == (y.data_ptr(), 768)
    assert binding._token_rows("k", None, 2, 128, 4) == (None, 0) and binding._token_rows("k", 256, 2, 128, 4) == (256, 0)
    for bad in (torch.zeros(4, 2, 256, **bf)[..., ::2], torch.zeros(2, 4, 128, **bf).transpose(0, 1), x.view(4, 256)):
        with pytest.raises(binding.SAError):
            binding._token_rows("k", bad, 2, 128, 4)
    with pytest.raises(binding.SAError):
        binding.paged_args(x, x, torch.zeros(5, 2, dtype=torch.int32).T, 16, 2, 128, 64, 10, x, x, 1.0)


def test_tensors_the_library_would_misread_are_refused(lib):
    import torch
    B, T, H, Hkv, D, P, n = 3, 4, 16, 2, 128, 64, 10
    i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    seq, pos, table = torch.zeros(T, **i32), torch.zeros(T, **i32), torch.zeros(B, 5, **i32)
    cache = torch.zeros(n, Hkv, P, D, **bf)

    def args(**kw):
        a = dict(q_seq=seq, q_pos=pos, page_table=table, K=cache, V=cache)
        a.update(kw)
        return binding.paged_args(a["q_seq"], a["q_pos"], a["page_table"], H, Hkv, D, P, n, a["K"], a["V"], 1.0)

    pa = args()
    for kw in (dict(q_seq=seq.long()), dict(q_pos=pos.long()), dict(q_pos=torch.zeros(2 * T, **i32)[::2]),
               dict(q_pos=pos[1:]), dict(page_table=table.long()), dict(page_table=table[:1].expand(B, 5)),
               dict(K=cache.float()), dict(V=torch.zeros(n, 2, Hkv, P, D, **bf)[:, 0])):
        with pytest.raises(binding.SAError):
            args(**kw)
    # tokens that share one row, as a broadcast leaves them
    k, q, ws = torch.zeros(T, Hkv, D, **bf), torch.zeros(T, H, D, **bf), torch.zeros(1 << 16, dtype=torch.uint8)
    for x in (k[:1].expand(T, Hkv, D), k.float()):
        with pytest.raises(binding.SAError):
            binding.sa_paged_append(pa, x, k, ws)
    bad_q = torch.zeros(T, 2 * H, D, **bf)[:, :H]
    mean, scores, idx = torch.zeros(n, Hkv, D, **bf), torch.zeros(T, Hkv, 8), torch.zeros(T, Hkv, 4, **i32)
    for call in (lambda: binding.sa_paged_append(pa, k, k, ws, q=q, q_out=bad_q),
                 lambda: binding.sa_page_scores(pa, bad_q, mean, scores, ws),
                 lambda: binding.sa_page_scores(pa, q, mean.float(), scores, ws),
                 lambda: binding.sa_page_scores(pa, q, mean, scores.double(), ws),
                 lambda: binding.sa_page_scores(pa, q, mean, torch.zeros(T, 2 * Hkv, 8)[:, :Hkv], ws),
                 lambda: binding.sa_block_attn(pa, bad_q, idx, 4, 1, q, ws),
                 lambda: binding.sa_block_attn(pa, q, idx.long(), 4, 1, q, ws),
                 lambda: binding.sa_block_attn(pa, q, idx, 4, 1, bad_q, ws),
                 lambda: binding.sa_fused_block_attn(pa, q, mean, 4, 1, idx.long(), q, ws),
                 lambda: binding.sa_prefix_attn(pa, q, 1, q.float(), ws)):
        with pytest.raises(binding.SAError):
            call()


def test_lists_past_2_30_entries_are_refused(lib):
    assert _block(lib, _pa(), K=(1 << 30) + 1) == UNS
    assert _fused(lib, _pa(), K=(1 << 30) + 1) == UNS
    assert lib.sa_paged_workspace_size(_ref(_pa()), (1 << 30) + 1, 1, 0) == 0


class _Elsewhere:
    """A tensor that says it lies on another device."""

    def __init__(self, x):
        self._x = x

    def __getattr__(self, name):
        return getattr(self._x, name)

    def get_device(self):
        return self._x.get_device() + 1


def test_types_and_sizes_the_library_would_misread_are_refused(lib):
    # a tensor of the right width but another type, or smaller than the call
    # reads or writes, never reaches the library
    import torch
    B, T, H, Hkv, D, P, n, K = 3, 4, 16, 2, 128, 64, 10, 4
    i32, bf, f16 = dict(dtype=torch.int32), dict(dtype=torch.bfloat16), dict(dtype=torch.float16)
    seq, table = torch.zeros(T, **i32), torch.zeros(B, 5, **i32)
    cache = torch.zeros(n, Hkv, P, D, **bf)

    def args(**kw):
        a = dict(q_seq=seq, q_pos=seq, page_table=table, K=cache, V=cache)
        a.update(kw)
        return binding.paged_args(a["q_seq"], a["q_pos"], a["page_table"], H, Hkv, D, P, n, a["K"], a["V"], 1.0)

    for kw in (dict(q_seq=seq.float()), dict(q_pos=seq.float()), dict(page_table=table.float()), dict(K=cache.half()),
               dict(V=cache.half()), dict(K=cache[:-1]), dict(V=cache[:, :1].contiguous()),
               dict(K=torch.zeros(n, P, Hkv, D, **bf)), dict(V=cache.view(-1)[:-8]), dict(K=_Elsewhere(cache)),
               dict(page_table=_Elsewhere(table))):
        with pytest.raises(binding.SAError):
            args(**kw)
    pa = args()
    k, q, ws = torch.zeros(T, Hkv, D, **bf), torch.zeros(T, H, D, **bf), torch.zeros(1 << 16, dtype=torch.uint8)
    mean, scores, idx = torch.zeros(n, Hkv, D, **bf), torch.zeros(T, Hkv, 8), torch.zeros(T, Hkv, K, **i32)
    wide = torch.zeros(T, Hkv, K + 1, **i32)
    bad_q = (q.half(), q[:-1], q[:, :-1].contiguous(), torch.zeros(T, H, 64, **bf), _Elsewhere(q))
    calls = []
    for x in (k.half(), k[:-1], k[:, :1], torch.zeros(T, Hkv, 64, **bf), _Elsewhere(k)):
        calls += [lambda x=x: binding.sa_paged_append(pa, x, k, ws), lambda x=x: binding.sa_paged_append(pa, k, x, ws)]
    for x in bad_q:
        calls += [lambda x=x: binding.sa_paged_append(pa, k, k, ws, q=x, q_out=q),
                  lambda x=x: binding.sa_paged_append(pa, k, k, ws, q=q, q_out=x),
                  lambda x=x: binding.sa_page_scores(pa, x, mean, scores, ws),
                  lambda x=x: binding.sa_block_attn(pa, x, idx, K, 1, q, ws),
                  lambda x=x: binding.sa_block_attn(pa, q, idx, K, 1, x, ws),
                  lambda x=x: binding.sa_fused_block_attn(pa, x, mean, K, 1, idx, q, ws),
                  lambda x=x: binding.sa_fused_block_attn(pa, q, mean, K, 1, idx, x, ws),
                  lambda x=x: binding.sa_prefix_attn(pa, x, 1, q, ws),
                  lambda x=x: binding.sa_prefix_attn(pa, q, 1, x, ws)]
    for x in (mean.half(), mean[:-1], mean[:, :1].contiguous(), _Elsewhere(mean)):
        calls += [lambda x=x: binding.sa_paged_append(pa, k, k, ws, k_mean=x),
                  lambda x=x: binding.sa_page_scores(pa, q, x, scores, ws),
                  lambda x=x: binding.sa_fused_block_attn(pa, q, x, K, 1, idx, q, ws)]
    for x in (idx.float(), idx[:-1], wide, idx[:, :, :-1].contiguous(), _Elsewhere(idx)):
        calls += [lambda x=x: binding.sa_block_attn(pa, q, x, K, 1, q, ws),
                  lambda x=x: binding.sa_fused_block_attn(pa, q, mean, K, 1, x, q, ws)]
    for x in (scores.int(), scores[:-1], scores[:, :1].contiguous(), scores[..., :4], scores.view(T * Hkv, 8)[:-1],
              scores.view(T * Hkv, 8)[:, :4], scores.view(-1)[:T * Hkv * 5 - 1], torch.zeros(T, Hkv, 8, 2)[..., 0],
              scores.view(T * Hkv // 2, 16), scores.view(1, T * Hkv, 8)):
        calls.append(lambda x=x: binding.sa_page_scores(pa, q, mean, x, ws))
    calls.append(lambda: binding.sa_page_scores(pa, q, mean, scores, ws, ld=9))
    calls.append(lambda: binding.sa_prefix_attn(pa, q, 1, q, _Elsewhere(ws)))
    for i, call in enumerate(calls):
        with pytest.raises(binding.SAError) as e:
            call()
        assert e.value.status == INV, i


def test_layouts_the_library_reads_right_are_taken():
    import torch
    bf = dict(dtype=torch.bfloat16)
    q = torch.zeros(6, 16, 128, **bf)
    for x in (q, q.view(6, 16 * 128), q.view(-1), q.view(2, 3, 16, 128), q.view(96, 128)):
        assert binding._dense("q", x, torch.bfloat16, 6, 16 * 128) == q.data_ptr()
    for x in (q, q.view(6, 16 * 128), q.view(-1)):  # more tokens than the call's
        assert binding._dense("q", x, torch.bfloat16, 4, 16 * 128) == q.data_ptr()
    assert binding._dense("q", q, torch.bfloat16, 0, 16 * 128) == q.data_ptr()
    assert binding._dense("q", None, torch.bfloat16, 4, 8) is None and binding._dense("q", 256, torch.bfloat16, 4, 8) == 256
    assert binding._token_rows("k", q, 8, 128, 5) == (q.data_ptr(), 16 * 128)
    pa = _pa(T=6, H=16, H_kv=2, max_pages=5)
    s = torch.zeros(6, 2, 8)
    for x, ld in ((s, 8), (s[..., :5], 8), (s.view(12, 8), 8), (s.view(12, 8)[:, :5], 8), (s.view(-1), 5),
                  (torch.zeros(7, 2, 5), 5)):
        assert binding._score_rows(pa, x, None, None) == (x.data_ptr(), ld)
    one = _pa(T=6, H=16, H_kv=1, max_pages=5)
    assert binding._score_rows(one, s[:, 1:], None, None) == (s[:, 1:].data_ptr(), 16)
    assert binding._score_rows(pa, s.view(-1), 8, None) == (s.data_ptr(), 8)
