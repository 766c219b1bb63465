"""The paged-cache operators at the sizes they are used at, with their plain forms.

Four operators over a paged key/value cache ([pages, kv heads, positions per
page, head dim], a page table per sequence):

  append   new keys and values into the pages, rotary embedding applied on the
           way (queries rotated alongside), mean key of every page that fills
  scores   the cheap score of every complete page for every query and kv head:
           scale * sum over the group's heads of q . mean key
  blocks   attention over the pages an index list names and the newest pages
  prefix   decode attention for a batch whose sequences share their first pages

``prepare`` makes what a serving loop holds before the call, ``run`` makes one
call, ``exact`` evaluates the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one decode step of a GQA model: one new token per sequence
        dict(name="append_decode_b64", op="append", B=64, new=1, H=64, Hkv=8, D=128, P=64, lo=512, hi=2047,
             rope=128, halves=True, yarn=False, pos_seed=1),
        # a ragged prefill batch: 24 prompts in one call
        dict(name="append_prefill_ragged", op="append", B=24, new=600, H=64, Hkv=8, D=128, P=64, lo=0, hi=333,
             rope=128, halves=True, yarn=False, pos_seed=2),
        # a 4096-token chunk far into one long sequence, one kv head, the last
        # 64 values rotated with YaRN
        dict(name="append_chunk_mqa", op="append", B=1, new=4096, H=64, Hkv=1, D=128, P=128, lo=28672, hi=28672,
             rope=64, halves=False, yarn=True, pos_seed=3),
        # page scores of a few short decodes: the smallest call
        dict(name="scores_decode_b4", op="scores", B=4, new=1, H=16, Hkv=2, D=128, P=32, lo=2048, hi=4095, pos_seed=4),
        # page scores of a long-context decode batch
        dict(name="scores_decode_b64", op="scores", B=64, new=1, H=64, Hkv=8, D=128, P=64, lo=32768, hi=65535,
             pos_seed=5),
        # page scores of a prefill chunk: many queries over the same pages
        dict(name="scores_chunk", op="scores", B=1, new=4096, H=64, Hkv=4, D=128, P=64, lo=28672, hi=28672,
             pos_seed=6),
        # one long-context query: latency alone
        dict(name="blocks_decode_b1", op="blocks", B=1, new=1, H=16, Hkv=2, D=128, P=64, lo=40000, hi=60000, K=32,
             local=2, pos_seed=7),
        # a decode batch over one kv head: 2048 selected keys and a window
        dict(name="blocks_decode_b64_mqa", op="blocks", B=64, new=1, H=64, Hkv=1, D=128, P=64, lo=32768, hi=65535,
             K=32, local=2, pos_seed=8),
        # a prefill chunk, every query with a list of its own
        dict(name="blocks_chunk_gqa", op="blocks", B=2, new=777, H=32, Hkv=4, D=128, P=128, lo=12000, hi=30000, K=12,
             local=1, pos_seed=9),
        # a handful of samples of one short prompt
        dict(name="prefix_b4", op="prefix", B=4, new=1, H=16, Hkv=2, D=128, P=32, shared=130, lo=1, hi=255,
             pos_seed=10),
        # a decode batch behind one long document
        dict(name="prefix_b64_gqa", op="prefix", B=64, new=1, H=64, Hkv=8, D=128, P=64, shared=512, lo=1, hi=1500,
             pos_seed=11),
        # the largest: 64 heads over one kv head, every head of every sequence
        # against the same 32 K keys
        dict(name="prefix_b128_mqa", op="prefix", B=128, new=1, H=64, Hkv=1, D=128, P=128, shared=256, lo=1, hi=900,
             pos_seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "scores", "blocks", "prefix"])
    D = rng.choice([64, 128, 128])
    P = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if Hkv == 1:
        G = rng.choice([16, 32, 48, 64, 64])
    c = dict(op=op, H=Hkv * G, Hkv=Hkv, D=D, P=P, pos_seed=rng.randrange(1 << 20))
    if op == "append":
        if rng.random() < 0.5:
            c.update(B=_log_int(rng, 1, 128), new=1, lo=rng.randrange(0, 500), hi=rng.randrange(500, 2047))
        else:
            B = _log_int(rng, 1, 24)
            c.update(B=B, new=_log_int(rng, 2, 12000 // B), lo=0, hi=_log_int(rng, 1, 2000))
        c.update(rope=rng.choice([0, 32, 64, D]), halves=rng.random() < 0.5, yarn=rng.random() < 0.3)
    elif op == "scores":
        if rng.random() < 0.5:
            hi = _log_int(rng, 500, 65535)
            c.update(B=_log_int(rng, 1, 64), new=1, lo=hi // 2, hi=hi)
        else:
            p = _log_int(rng, 1, 20000)
            c.update(B=rng.choice([1, 2, 3]), new=_log_int(rng, 2, 1300), lo=p // 2, hi=p)
    elif op == "blocks":
        keys = _log_int(rng, 100, 2048)
        c.update(K=max(1, keys // P), local=rng.choice([1, 1, 2, 3]))
        if rng.random() < 0.6:
            hi = _log_int(rng, 300, 40000)
            c.update(B=_log_int(rng, 1, 32), new=1, lo=hi // 3, hi=hi)
        else:
            p = _log_int(rng, 1, 20000)
            c.update(B=rng.choice([1, 2, 3]), new=_log_int(rng, 2, 400), lo=p // 2, hi=p)
    else:
        c.update(B=_log_int(rng, 1, 100), new=rng.choice([1, 1, 1, 2]), shared=max(1, _log_int(rng, 100, 24000) // P),
                 lo=rng.choice([0, 1, 40]), hi=_log_int(rng, 50, 1500))
    return c


# ---------------------------------------------------------------- geometry ---

def _layout(c):
    """Host arrays of a case: the sequence and position of every token, the
    pages each sequence holds, and its page table (pages in shuffled order;
    shared pages first in every row)."""
    r = np.random.RandomState(c["pos_seed"])
    B, new, P = c["B"], c["new"], c["P"]
    shared = c.get("shared", 0)
    start = shared * P + r.randint(c["lo"], c["hi"] + 1, size=B)
    if new > 1 and B > 1:
        count = r.randint(max(1, new // 2), new + 1, size=B)
    else:
        count = np.full(B, new)
    seq = np.repeat(np.arange(B), count).astype(np.int32)
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, count)]).astype(np.int32)
    pages = (start + count + P - 1) // P
    total = shared + int((pages - shared).sum())
    perm = r.permutation(total).astype(np.int32)
    max_pages = int(pages.max())
    table = np.zeros((B, max_pages), np.int32)
    at = shared
    for b in range(B):
        table[b, :shared] = perm[:shared]
        n = int(pages[b]) - shared
        table[b, shared:pages[b]] = perm[at:at + n]
        at += n
    return dict(seq=seq, pos=pos, start=start, count=count, table=table, total=total, max_pages=max_pages,
                T=len(seq))


def _rope_params(c):
    """(base, factor, original length, beta_fast, beta_slow): the long-context
    parameters of the compressed caches, or a plain table."""
    return (160000.0, 16.0, 65536, 32.0, 1.0) if c["yarn"] else (10000.0, 1.0, 0, 32.0, 1.0)


def work(case):
    g = _layout(case)
    T, H, Hkv, D, P = g["T"], case["H"], case["Hkv"], case["D"], case["P"]
    if case["op"] == "append":
        full = int(((g["pos"] + 1) % P == 0).sum())
        # new rows in and out, queries in and out, the full pages' older rows and their means
        older = sum(int(s % P) for s, n in zip(g["start"], g["count"]) if s // P < (s + n) // P)
        by = 2 * 2 * 2 * T * Hkv * D + 2 * 2 * T * H * D + 2 * Hkv * D * (older + full)
        return {"bytes": by, "flops": 6 * T * (H + Hkv) * case["rope"] // 2 + full * P * Hkv * D}
    vis = (g["pos"].astype(np.int64) + 1) // P
    if case["op"] == "scores":
        rows = sum(int((s + n) // P) for s, n in zip(g["start"], g["count"]))
        by = 2 * T * H * D + 2 * rows * Hkv * D + 4 * T * Hkv * g["max_pages"]
        return {"bytes": by, "flops": int(2 * vis.sum() * Hkv * D + T * H * D)}
    if case["op"] == "blocks":
        first = np.maximum(g["pos"] // P - (case["local"] - 1), 0)
        keys = np.minimum(first, case["K"]) * P + g["pos"] + 1 - first * P
        # pages that several queries of a sequence name are read once at best
        per_seq = [keys[g["seq"] == b].sum() for b in range(case["B"])]
        most = (g["start"] + g["count"])
        rows = sum(min(int(k), int(m)) for k, m in zip(per_seq, most))
        by = 4 * T * H * D + 4 * rows * Hkv * D + 4 * T * Hkv * case["K"]
        return {"bytes": by, "flops": int(4 * keys.sum() * H * D)}
    rows = case["shared"] * P + int((g["start"] + g["count"] - case["shared"] * P).sum())
    keys = int((g["pos"].astype(np.int64) + 1).sum())
    return {"bytes": 4 * T * H * D + 4 * rows * Hkv * D, "flops": 4 * keys * H * D}


# ------------------------------------------------------------------ inputs ---

def prepare(case, seed):
    g = _layout(case)
    T, H, Hkv, D, P = g["T"], case["H"], case["Hkv"], case["D"], case["P"]
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32) * scale).bfloat16()

    st = dict(case=case, g=g,
              seq=torch.from_numpy(g["seq"]).to(DEV), pos=torch.from_numpy(g["pos"]).to(DEV),
              table=torch.from_numpy(g["table"]).to(DEV), scale=D ** -0.5)
    op = case["op"]
    if op == "append":
        # q, k and v are slices of one projection's output, as a model has them
        qkv = normal(T, (H + 2 * Hkv) * D)
        st["q"] = qkv[:, :H * D].view(T, H, D)
        st["k"] = qkv[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
        st["v"] = qkv[:, (H + Hkv) * D:].view(T, Hkv, D)
        st["K"], st["V"] = normal(g["total"], Hkv, P, D), normal(g["total"], Hkv, P, D)
        st["mean"] = normal(g["total"], Hkv, D, scale=P ** -0.5)
        st["q_out"] = torch.zeros(T, H, D, device=DEV, dtype=torch.bfloat16)
        full = np.nonzero((g["pos"] + 1) % P == 0)[0]
        st["full_rows"] = torch.from_numpy(full).to(DEV)
        st["freq"] = _frequencies(case)
    else:
        st["q"] = normal(T, H, D)
        st["out"] = torch.zeros(T, H, D, device=DEV, dtype=torch.bfloat16)
    if op == "scores":
        st["mean"] = normal(g["total"], Hkv, D, scale=P ** -0.5)
        st["scores"] = torch.zeros(T, Hkv, g["max_pages"], device=DEV, dtype=torch.float32)
    if op in ("blocks", "prefix"):
        st["K"], st["V"] = normal(g["total"], Hkv, P, D), normal(g["total"], Hkv, P, D)
    if op == "blocks":
        st["idx"] = _lists(st, gen)
    if op == "prefix":
        # the longest suffix, known to whoever built the batch
        st["suffix"] = int((g["start"] + g["count"]).max()) - case["shared"] * P
    if own:
        from indexer_selected_sparse_score_gb300 import binding as sb
        st["pa"] = sb.paged_args(st["seq"], st["pos"], st["table"], H, Hkv, D, P, g["total"], st.get("K"),
                                 st.get("V"), st["scale"])
        st["ws"] = sb.new_paged_workspace(st["pa"], case.get("K", 0), case.get("local", 0), case.get("shared", 0))
        if op == "append":
            base, factor, orig, fast, slow = _rope_params(case)
            st["rope"] = sb.RopeArgs(case["rope"], base, factor, orig, fast, slow)
    return st


def _lists(st, gen):
    """Distinct pages before the local ones, in ascending order, -1 at the end."""
    c, g = st["case"], st["g"]
    nb, K = g["max_pages"], c["K"]
    first = (st["pos"].long() // c["P"] - (c["local"] - 1)).clamp(min=0)
    out = []
    for i in range(0, g["T"], 512):
        f = first[i:i + 512]
        r = torch.rand(len(f), c["Hkv"], max(nb, K), generator=gen, device=DEV)
        blk = torch.arange(max(nb, K), device=DEV)
        r = torch.where(blk < f[:, None, None], r, torch.full_like(r, -1.0))
        val, ind = r.topk(K, dim=-1)
        ind = torch.where(val < 0, torch.full_like(ind, 1 << 30), ind).sort(dim=-1).values
        out.append(torch.where(ind == 1 << 30, torch.full_like(ind, -1), ind))
    return torch.cat(out).to(torch.int32).contiguous()


# --------------------------------------------------------------------- run ---

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    return {"append": _append, "scores": _scores, "blocks": _blocks, "prefix": _prefix}[op](st)


def _run_own(st, op):
    from indexer_selected_sparse_score_gb300 import binding as sb
    c = st["case"]
    if op == "append":
        sb.sa_paged_append(st["pa"], st["k"], st["v"], st["ws"], q=st["q"], q_out=st["q_out"], rope=st["rope"],
                           halves=c["halves"], k_mean=st["mean"])
        return dict(K=st["K"], V=st["V"], q=st["q_out"], mean=st["mean"])
    if op == "scores":
        sb.sa_page_scores(st["pa"], st["q"], st["mean"], st["scores"], st["ws"])
        return st["scores"]
    if op == "blocks":
        sb.sa_block_attn(st["pa"], st["q"], st["idx"], c["K"], c["local"], st["out"], st["ws"])
        return st["out"]
    sb.sa_prefix_attn(st["pa"], st["q"], c["shared"], st["out"], st["ws"])
    return st["out"]


# ------------------------------------------------------------- plain forms ---

def _frequencies(c):
    """Rotation frequencies of the pairs, in 64 bits."""
    dim = c["rope"]
    base, factor, orig, fast, slow = _rope_params(c)
    i = torch.arange(dim // 2, device=DEV, dtype=torch.float64)
    f = base ** (-2 * i / max(dim, 1))
    if orig > 0 and dim > 0:
        def dim_of(turns):
            return dim * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        low = max(math.floor(dim_of(fast)), 0)
        high = min(math.ceil(dim_of(slow)), dim - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    return f


def _rotate(x, cos, sin, dim, halves):
    """Rotates the last ``dim`` values of x ([T, heads, D], 32 bits)."""
    if dim == 0:
        return x
    keep, r = x[..., :-dim], x[..., -dim:]
    cos, sin = cos[:, None], sin[:, None]
    if halves:
        a, b = r[..., :dim // 2], r[..., dim // 2:]
        return torch.cat([keep, a * cos - b * sin, a * sin + b * cos], dim=-1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([keep, torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)], dim=-1)


def _append(st):
    c, P = st["case"], st["case"]["P"]
    ang = st["pos"].double()[:, None] * st["freq"]
    cos, sin = ang.cos().float(), ang.sin().float()
    page = st["table"][st["seq"].long(), (st["pos"] // P).long()].long()
    slot = (st["pos"] % P).long()
    st["K"][page, :, slot] = _rotate(st["k"].float(), cos, sin, c["rope"], c["halves"]).bfloat16()
    st["V"][page, :, slot] = st["v"]
    st["q_out"].copy_(_rotate(st["q"].float(), cos, sin, c["rope"], c["halves"]))
    done = page[st["full_rows"]]
    st["mean"][done] = st["K"][done].float().mean(dim=2).bfloat16()
    return dict(K=st["K"], V=st["V"], q=st["q_out"], mean=st["mean"])


def _spans(g):
    """(sequence, first token, last token + 1) of each sequence's tokens."""
    at = 0
    for b, n in enumerate(g["count"]):
        yield b, at, at + int(n)
        at += int(n)


def _scores(st):
    c, g = st["case"], st["g"]
    P, Hkv = c["P"], c["Hkv"]
    qs = st["q"].float().view(g["T"], Hkv, -1, c["D"]).sum(dim=2) * st["scale"]
    out = st["scores"]
    blk = torch.arange(g["max_pages"], device=DEV)
    seen = blk[None] < ((st["pos"].long() + 1) // P)[:, None]
    if c["new"] == 1:  # a decode step: every sequence at once
        m = st["mean"][st["table"].long()].float()                 # [B, pages, kv heads, D]
        s = torch.einsum("thd,tphd->thp", qs, m)
        return torch.where(seen[:, None], s, torch.full_like(s, -math.inf), out=out)
    for b, i, j in _spans(g):
        m = st["mean"][st["table"][b].long()].float()              # [pages, kv heads, D]
        s = torch.einsum("thd,phd->thp", qs[i:j], m)
        out[i:j] = torch.where(seen[i:j, None], s, torch.full_like(s, -math.inf))
    return out


def _attend(q, k, v, ok, scale):
    """q [n, heads, G, D], k and v [n, heads, keys, D], ok [n, heads, keys]."""
    s = (q @ k.transpose(-1, -2)) * scale
    s = torch.where(ok[:, :, None], s, torch.full_like(s, -math.inf))
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (s - m).exp()
    den = p.sum(dim=-1, keepdim=True)
    return (p @ v) / torch.where(den == 0, torch.ones_like(den), den)


def _blocks(st):
    c, g = st["case"], st["g"]
    P, Hkv, D, local = c["P"], c["Hkv"], c["D"], c["local"]
    step = max(1, (1 << 28) // (Hkv * (c["K"] + local) * P * D))
    heads = torch.arange(Hkv, device=DEV)
    inside = torch.arange(P, device=DEV)
    for i in range(0, g["T"], step):
        pos, seq = st["pos"][i:i + step].long(), st["seq"][i:i + step].long()
        n = len(pos)
        first = (pos // P - (local - 1)).clamp(min=0)
        last = first[:, None] + torch.arange(local, device=DEV)
        blk = torch.cat([st["idx"][i:i + step].long(), last[:, None].expand(n, Hkv, local)], dim=-1)
        listed_ok = (blk >= 0) & (blk < first[:, None, None])
        listed_ok[..., c["K"]:] = (last <= (pos // P)[:, None])[:, None]
        blk = torch.where(listed_ok, blk, torch.zeros_like(blk))
        page = st["table"].long()[seq[:, None, None], blk]
        k = st["K"][page, heads[None, :, None]].float().flatten(2, 3)
        v = st["V"][page, heads[None, :, None]].float().flatten(2, 3)
        key = (blk[..., None] * P + inside).flatten(2)
        ok = listed_ok[..., None].expand(-1, -1, -1, P).flatten(2) & (key <= pos[:, None, None])
        q = st["q"][i:i + step].float().view(n, Hkv, -1, D)
        st["out"][i:i + step] = _attend(q, k, v, ok, st["scale"]).view(n, -1, D)
    return st["out"]


def _prefix(st):
    c, g = st["case"], st["g"]
    P, Hkv, D, T = c["P"], c["Hkv"], c["D"], g["T"]
    q = st["q"].float().view(T, Hkv, -1, D)
    G = q.shape[2]
    # the shared part, once for the whole batch: [kv heads, T * G, keys]
    pages = st["table"][0, :c["shared"]].long()
    k = st["K"][pages].transpose(0, 1).flatten(1, 2).float()
    v = st["V"][pages].transpose(0, 1).flatten(1, 2).float()
    qh = q.transpose(0, 1).reshape(Hkv, T * G, D)
    m1, l1, o1 = [], [], []
    step = max(1, (1 << 29) // (Hkv * k.shape[1]))
    for i in range(0, T * G, step):
        s = (qh[:, i:i + step] @ k.transpose(-1, -2)) * st["scale"]
        m = s.amax(dim=-1, keepdim=True)
        p = (s - m).exp()
        m1.append(m)
        l1.append(p.sum(dim=-1, keepdim=True))
        o1.append(p @ v)
    m1, l1, o1 = (torch.cat(x, dim=1).view(Hkv, T, G, -1).transpose(0, 1) for x in (m1, l1, o1))
    # every sequence's own keys
    n = (st["suffix"] + P - 1) // P
    own_pages = st["table"][:, c["shared"]:c["shared"] + n].long()[st["seq"].long()]
    ks = st["K"][own_pages].transpose(1, 2).flatten(2, 3).float()   # [T, kv heads, keys, D]
    vs = st["V"][own_pages].transpose(1, 2).flatten(2, 3).float()
    key = c["shared"] * P + torch.arange(ks.shape[2], device=DEV)
    s = (q @ ks.transpose(-1, -2)) * st["scale"]
    s = torch.where((key <= st["pos"].long()[:, None])[:, None, None], s, torch.full_like(s, -math.inf))
    m = torch.maximum(m1, s.amax(dim=-1, keepdim=True))
    a, p = (m1 - m).exp(), (s - m).exp()
    o = (o1 * a + p @ vs) / (l1 * a + p.sum(dim=-1, keepdim=True))
    st["out"].copy_(o.reshape(T, -1, D))
    return st["out"]


# ------------------------------------------------------------------- exact ---

def exact(case, seed):
    """The definitions in 64 bits, key by key and page by page."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "scores": _exact_scores, "blocks": _exact_attention,
            "prefix": _exact_attention}[case["op"]](st)


def _exact_append(st):
    c, g = st["case"], st["g"]
    T, D, P, dim = g["T"], c["D"], c["P"], c["rope"]
    base, factor, orig, fast, slow = _rope_params(c)
    freq = np.zeros(dim // 2)
    for i in range(dim // 2):
        f = 1.0 / base ** (2.0 * i / dim)
        if orig:
            low = max(math.floor(dim * math.log(orig / (fast * 2 * math.pi)) / (2 * math.log(base))), 0)
            high = min(math.ceil(dim * math.log(orig / (slow * 2 * math.pi)) / (2 * math.log(base))), dim - 1)
            w = min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0)
            f = f * (1 - w) + f / factor * w
        freq[i] = f
    ang = np.outer(g["pos"].astype(np.float64), freq)
    z = torch.from_numpy(np.cos(ang) + 1j * np.sin(ang)).to(DEV)[:, None]

    def turned(x):
        x = x.double().clone()
        if dim == 0:
            return x
        t = x[..., D - dim:]
        if c["halves"]:
            w = torch.complex(t[..., :dim // 2], t[..., dim // 2:]) * z
            x[..., D - dim:] = torch.cat([w.real, w.imag], dim=-1)
        else:
            w = torch.view_as_complex(t.reshape(T, -1, dim // 2, 2).contiguous()) * z
            x[..., D - dim:] = torch.view_as_real(w).flatten(-2)
        return x

    K, V, mean = st["K"].double(), st["V"].double(), st["mean"].double()
    kr = turned(st["k"])
    pages, slots = g["table"][g["seq"], g["pos"] // P], g["pos"] % P
    pg, sl = torch.from_numpy(pages).long().to(DEV), torch.from_numpy(slots).long().to(DEV)
    K[pg, :, sl] = kr
    V[pg, :, sl] = st["v"].double()
    full = sorted({int(p) for p, s in zip(pages, slots) if s == P - 1})
    if full:  # the mean is that of the stored rows
        f = torch.tensor(full, device=DEV)
        mean[f] = K[f].bfloat16().double().sum(dim=2) / P
    return dict(K=K, V=V, q=turned(st["q"]), mean=mean)


def _exact_scores(st):
    c, g = st["case"], st["g"]
    T, Hkv = g["T"], c["Hkv"]
    out = torch.full((T, Hkv, g["max_pages"]), -math.inf, dtype=torch.float64, device=DEV)
    q = st["q"].double().view(T, Hkv, -1, c["D"])
    for b, i, j in _spans(g):
        m = st["mean"][st["table"][b].long()].double()
        for h in range(Hkv):
            s = sum(q[i:j, h, n] @ m[:, h].T for n in range(q.shape[2])) * st["scale"]
            vis = (st["pos"][i:j].long() + 1) // c["P"]
            hide = torch.arange(s.shape[1], device=DEV)[None] >= vis[:, None]
            out[i:j, h] = s.masked_fill(hide, -math.inf)
    return out


def _exact_attention(st):
    c, g = st["case"], st["g"]
    P, Hkv, D = c["P"], c["Hkv"], c["D"]
    G = c["H"] // Hkv
    out = torch.zeros(g["T"], c["H"], D, dtype=torch.float64, device=DEV)
    for b, i, j in _spans(g):
        n_pages = (int(g["pos"][j - 1]) + P) // P
        pages = st["table"][b, :n_pages].long()
        key = torch.arange(n_pages * P, device=DEV)
        for h in range(Hkv):
            k = st["K"][pages, h].reshape(-1, D).double()
            v = st["V"][pages, h].reshape(-1, D).double()
            for t in range(i, j, 64):
                e = min(t + 64, j)
                pos = st["pos"][t:e].long()
                allow = key[None] <= pos[:, None]
                if c["op"] == "blocks":
                    first = (pos // P - c["local"] + 1).clamp(min=0)
                    named = torch.zeros(e - t, n_pages + 1, dtype=torch.bool, device=DEV)
                    ids = st["idx"][t:e, h].long()
                    ids = torch.where((ids < 0) | (ids >= first[:, None]), torch.full_like(ids, n_pages), ids)
                    named.scatter_(1, ids, True)
                    near = torch.arange(n_pages, device=DEV)[None] >= first[:, None]
                    allow &= (named[:, :n_pages] | near).repeat_interleave(P, dim=1)
                q = st["q"][t:e].view(e - t, Hkv, G, D)[:, h].double()
                s = (q.reshape(-1, D) @ k.T * st["scale"]).view(e - t, G, -1)
                s = s.masked_fill(~allow[:, None], -math.inf)
                out[t:e].view(e - t, Hkv, G, D)[:, h] = torch.softmax(s, dim=-1) @ v
    return out
