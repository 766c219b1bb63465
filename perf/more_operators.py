"""A paged cache that is kept small, at the sizes it is used at, with the plain forms.

Keys and values held in 4 bits ([pages, kv heads, positions per page, head dim]
codes of e2m1, an e4m3 scale for every 16 values of a row), and slots freed by the
attention weight that each has gathered:

  append   new keys and values into the pages: rotation at a position that need
           not be the slot's number, quantisation, the queries alongside, the
           slots' records begun; then the rows read back as the cache holds them
  attn     attention over whole sequences of the 4-bit cache, with the logarithm
           of every row's sum of exponentials
  weights  every slot's attention weight, summed over the call's tokens and the
           heads that share it, added to the slot's record
  evict    the slots that keep their place by weight and age, per sequence and kv
           head; freed slots take the rows from behind the new end

``prepare`` makes what a serving loop holds before the call, ``run`` makes one
pass, ``exact`` evaluates the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one decode step of a grouped-query model whose caches have been evicted
        # from: slots below 2048, positions far past them
        dict(name="append_decode_b64", op="append", B=64, new=1, H=64, Hkv=8, D=128, P=64, lo=512, hi=2047, gone=60000,
             rope=128, halves=True, gain=0, pos_seed=1),
        # a ragged prefill batch: 24 prompts in one call
        dict(name="append_prefill_ragged", op="append", B=24, new=600, H=64, Hkv=8, D=128, P=64, lo=0, hi=333, gone=0,
             rope=64, halves=False, gain=-1, pos_seed=2),
        # one long-context query: latency alone
        dict(name="attn_decode_b1", op="attn", B=1, new=1, H=16, Hkv=2, D=128, P=64, lo=30000, hi=50000, pos_seed=3),
        # a decode batch of short chats, heads of 64
        dict(name="attn_decode_b16_d64", op="attn", B=16, new=1, H=32, Hkv=8, D=64, P=32, lo=100, hi=3000, pos_seed=4),
        # a decode batch with long contexts: the cache is streamed once
        dict(name="attn_decode_b64_gqa", op="attn", B=64, new=1, H=64, Hkv=8, D=128, P=64, lo=8192, hi=16383,
             pos_seed=5),
        # the same over one kv head
        dict(name="attn_decode_b64_mqa", op="attn", B=64, new=1, H=64, Hkv=1, D=128, P=64, lo=32768, hi=65535,
             pos_seed=6),
        # four drafted tokens per sequence, to be verified in one call
        dict(name="attn_draft_b32", op="attn", B=32, new=4, H=32, Hkv=8, D=128, P=64, lo=2048, hi=8191, pos_seed=7),
        # the next chunk of two prompts
        dict(name="attn_chunk_gqa", op="attn", B=2, new=777, H=32, Hkv=4, D=128, P=128, lo=6000, hi=12000, pos_seed=8),
        # a decode step's weights
        dict(name="weights_decode_b64", op="weights", B=64, new=1, H=64, Hkv=8, D=128, P=64, lo=2048, hi=8191,
             pos_seed=9),
        # a prompt chunk's weights, before the prompt is cut to a budget
        dict(name="weights_chunk", op="weights", B=1, new=1024, H=32, Hkv=4, D=128, P=64, lo=8192, hi=8192, pos_seed=10),
        # every sequence of a decode batch back to its budget, one page's slots gone
        dict(name="evict_decode_b64", op="evict", B=64, H=64, Hkv=8, D=128, P=64, lo=2112, hi=2112, budget=2048,
             recent=256, steady=True, pos_seed=11),
        # two long prompts cut to a budget before they decode
        dict(name="evict_prompt_b2", op="evict", B=2, H=32, Hkv=4, D=128, P=64, lo=16384, hi=32768, budget=2048,
             recent=128, steady=False, pos_seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "weights", "evict"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16]) if Hkv > 1 else rng.choice([8, 16, 24, 32, 48, 64])
    c = dict(op=op, H=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128, 128]), P=rng.choice([16, 32, 64, 128]),
             pos_seed=rng.randrange(1 << 20))
    if op == "append":
        if rng.random() < 0.5:
            c.update(B=_log_int(rng, 1, 128), new=rng.choice([1, 1, 3]), lo=rng.randrange(0, 500),
                     hi=rng.randrange(500, 2047))
        else:
            B = _log_int(rng, 1, 24)
            c.update(B=B, new=_log_int(rng, 2, 10000 // B), lo=0, hi=_log_int(rng, 1, 2000))
        c.update(rope=rng.choice([0, 32, 64, c["D"]]), halves=rng.random() < 0.5, gain=rng.choice([0, 0, -2, 3]),
                 gone=rng.choice([0, 0, 1000, 90000]))
    elif op == "evict":
        if rng.random() < 0.5:
            budget = _log_int(rng, 64, 4000)
            c.update(B=_log_int(rng, 1, 64), lo=budget, hi=budget + rng.choice([1, 16, 64, 200]), steady=True)
        else:
            hi = _log_int(rng, 500, 32768)
            budget = max(1, hi // rng.choice([2, 3, 8, 16]))
            c.update(B=rng.choice([1, 2, 3, 4]), lo=hi // 2, hi=hi, steady=False)
        c.update(budget=budget, recent=int(budget * rng.choice([0, 0.1, 0.5, 1])))
    else:
        kind = rng.random()
        if kind < 0.6:
            hi = _log_int(rng, 60, 32000)
            c.update(B=_log_int(rng, 1, max(1, min(64, 400000 // hi))), new=1, lo=hi // 3, hi=hi)
        elif kind < 0.8:
            hi = _log_int(rng, 60, 8000)
            c.update(B=_log_int(rng, 1, 16), new=rng.randrange(2, 9), lo=hi // 3, hi=hi)
        else:
            p = _log_int(rng, 1, 10000)
            c.update(B=rng.choice([1, 2]), new=_log_int(rng, 9, 500), lo=p // 2, hi=p)
    return c


# ---------------------------------------------------------------- geometry ---

def _layout(c):
    """Host arrays of a case: the sequence and slot of every token, the pages each
    sequence holds and its page table (pages in shuffled order).  `start` is a
    sequence's length before the call; an eviction has no tokens."""
    r = np.random.RandomState(c["pos_seed"])
    B, P, new = c["B"], c["P"], c.get("new", 0)
    start = r.randint(c["lo"], c["hi"] + 1, size=B)
    count = r.randint(max(1, new // 2), new + 1, size=B) if new > 8 and B > 1 else np.full(B, new)
    seq = np.repeat(np.arange(B), count).astype(np.int32)
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, count)]).astype(np.int32)
    pages = (start + count + P - 1) // P
    total, max_pages = int(pages.sum()), int(pages.max())
    perm = r.permutation(total).astype(np.int32)
    table = np.zeros((B, max_pages), np.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
    turn = (pos + r.randint(0, c.get("gone", 0) + 1, size=B)[seq]).astype(np.int32) if new else pos
    return dict(seq=seq, pos=pos, turn=turn, start=start, count=count, table=table, total=total, max_pages=max_pages,
                T=len(seq))


def work(case):
    g = _layout(case)
    T, H, Hkv, D = g["T"], case["H"], case["Hkv"], case["D"]
    row = D // 2 + D // 16  # bytes of a row in 4 bits
    n = int((g["start"] + g["count"]).sum())  # slots of all sequences
    if case["op"] == "append":
        # rows in, codes out and in again, rows out, queries in and out, records
        by = 4 * T * Hkv * D + 4 * T * Hkv * row + 4 * T * Hkv * D + 4 * T * H * D + 8 * T * Hkv
        return {"bytes": by, "flops": 6 * T * (H + Hkv) * case["rope"] // 2 + 4 * T * Hkv * D}
    if case["op"] == "evict":
        keep = np.minimum(g["start"], case["budget"])
        tail = g["start"] - keep
        near = np.minimum(tail, case["recent"])
        rest = (case["budget"] - case["recent"]) * (tail - near) / np.maximum(g["start"] - case["recent"], 1)
        moved = float((near + rest).sum())  # of a head, where weights and places are independent
        return {"bytes": 8 * Hkv * (n + int(keep.sum())) + 4 * moved * Hkv * row, "flops": n * Hkv}
    keys = int((g["pos"].astype(np.int64) + 1).sum())
    if case["op"] == "attn":
        return {"bytes": 2 * n * Hkv * row + 4 * T * H * D + 4 * T * H, "flops": 4 * keys * H * D}
    return {"bytes": n * Hkv * (row + 8) + 2 * T * H * D + 4 * T * H, "flops": 2 * keys * H * D}


# ------------------------------------------------------------------ inputs ---

def prepare(case, seed):
    g = _layout(case)
    T, H, Hkv, D, P, B = g["T"], case["H"], case["Hkv"], case["D"], case["P"], case["B"]
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)

    def held():
        """Pages of rows of normal values as the cache holds them."""
        codes = torch.empty(g["total"], Hkv, P, D // 2, device=DEV, dtype=torch.uint8)
        scales = torch.empty(g["total"], Hkv, P, D // 16, device=DEV, dtype=torch.uint8)
        step = max(1, (1 << 26) // (Hkv * P * D))
        for i in range(0, g["total"], step):
            codes[i:i + step], scales[i:i + step] = _quantise(normal(min(step, g["total"] - i), Hkv, P, D).bfloat16().float())
        return codes, scales

    st = dict(case=case, g=g, scale=D ** -0.5,
              seq=torch.from_numpy(g["seq"]).to(DEV), pos=torch.from_numpy(g["pos"]).to(DEV),
              table=torch.from_numpy(g["table"]).to(DEV), k_gain=2.0 ** case.get("gain", 0), v_gain=1.0)
    st["K"], st["Ks"] = held()
    st["V"], st["Vs"] = held()
    ld = (g["max_pages"] * P + 3) // 4 * 4
    op = case["op"]
    if op == "append":
        # q, k and v are slices of one projection's output, as a model has them
        qkv = normal(T, (H + 2 * Hkv) * D).bfloat16()
        st["q"] = qkv[:, :H * D].view(T, H, D)
        st["k"] = qkv[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
        st["v"] = qkv[:, (H + Hkv) * D:].view(T, Hkv, D)
        st["q_out"] = torch.zeros(T, H, D, device=DEV, dtype=torch.bfloat16)
        st["k_out"] = torch.zeros(T, Hkv, D, device=DEV, dtype=torch.bfloat16)
        st["v_out"] = torch.zeros(T, Hkv, D, device=DEV, dtype=torch.bfloat16)
        st["turn"] = torch.from_numpy(g["turn"]).to(DEV)
        i = torch.arange(case["rope"] // 2, device=DEV, dtype=torch.float64)
        st["freq"] = 10000.0 ** (-2 * i / max(case["rope"], 1))
    elif op in ("attn", "weights"):
        st["q"] = normal(T, H, D).bfloat16()
        st["out"] = torch.zeros(T, H, D, device=DEV, dtype=torch.bfloat16)
        st["lse"] = torch.zeros(T, H, device=DEV, dtype=torch.float32)
        # token t of sequence b as place (b, i) of a rectangle
        first = np.concatenate([[0], np.cumsum(g["count"])[:-1]])
        st["at"] = torch.from_numpy(g["seq"].astype(np.int64) * int(g["count"].max()) +
                                    np.arange(T) - first[g["seq"]]).to(DEV)
    if op == "weights":
        _attn(st)  # the step's attention left the rows' sums
    if op in ("append", "weights", "evict"):
        # weights as they gather: few slots hold most of them; a prompt's first
        # chunk finds none
        st["weight"] = normal(B, Hkv, ld).mul(2).exp() * (0.01 if case.get("new", 1) <= 8 else 0.0)
        st["born"] = torch.arange(ld, device=DEV, dtype=torch.int32).expand(B, Hkv, ld).contiguous()
    if op == "evict":
        st["length"] = torch.from_numpy(g["start"].astype(np.int32)).to(DEV)
        st["newest"] = st["length"] - 1
        if case["steady"]:
            # earlier evictions have mixed the slots: all but the last few, which
            # were appended since, come in any order
            mixed = torch.rand(B, Hkv, ld, generator=gen, device=DEV)
            old = torch.arange(ld, device=DEV) < (st["length"] - (case["hi"] - case["budget"]))[:, None, None]
            st["born"] = torch.where(old, mixed, 1 + st["born"]).argsort(dim=-1).to(torch.int32)
        st["weight_out"] = torch.zeros_like(st["weight"])
        st["born_out"] = torch.zeros_like(st["born"])
        st["length_out"] = torch.zeros_like(st["length"])
    if own:
        from indexer_selected_sparse_score_gb300 import binding as sb
        st["pa"] = sb.paged4_args(st["seq"], st["pos"], st["table"], H, Hkv, D, P, g["total"], st["K"], st["V"],
                                  st["Ks"], st["Vs"], st["scale"], st["k_gain"], st["v_gain"])
        st["ws"] = sb.new_paged4_workspace(st["pa"])
        if op == "append":
            st["rope_args"] = sb.RopeArgs(case["rope"], 10000.0, 1.0, 0, 32.0, 1.0)
    return st


# --------------------------------------------------------------------- run ---

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    return {"append": _append, "attn": _attn, "weights": _weights, "evict": _evict}[op](st)


def _run_own(st, op):
    from indexer_selected_sparse_score_gb300 import binding as sb
    c, pa, ws = st["case"], st["pa"], st["ws"]
    if op == "append":
        sb.sa_paged4_append(pa, st["k"], st["v"], ws, q=st["q"], q_out=st["q_out"], rope=st["rope_args"],
                            halves=c["halves"], rope_pos=st["turn"], weight=st["weight"], born=st["born"])
        sb.sa_paged4_read(pa, st["k_out"], st["v_out"], ws)
    elif op == "attn":
        sb.sa_paged4_attn(pa, st["q"], st["out"], ws, lse=st["lse"])
    elif op == "weights":
        sb.sa_paged4_weights(pa, st["q"], st["lse"], st["weight"], ws)
    else:
        sb.sa_paged4_evict(pa, st["length"], st["newest"], c["budget"], c["recent"], st["weight"], st["born"],
                           st["weight_out"], st["born_out"], st["length_out"], ws)
    return _outputs(st, op)


def _outputs(st, op):
    if op == "append":
        return dict(k=st["k_out"], v=st["v_out"], q=st["q_out"], weight=st["weight"], born=st["born"])
    if op == "attn":
        return dict(out=st["out"], lse=st["lse"])
    if op == "weights":
        return st["weight"]
    # the moved rows are bytes that keep their values
    return dict(K=st["K"], V=st["V"], Ks=st["Ks"], Vs=st["Vs"], weight=st["weight_out"], born=st["born_out"],
                length=st["length_out"])


# ------------------------------------------------------------- plain forms ---

def _quantise(z):
    """Codes and scales of rows of D values in 32 bits: s = e4m3(amax / 6) of every
    16, at least the smallest; the e2m1 value nearest z / s (ties to the even code),
    by comparisons with the exact products of s and the midpoints."""
    z = z.unflatten(-1, (-1, 16))
    a = z.abs()
    s = (a.amax(dim=-1) / 6).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    f = s.float()[..., None]
    code = (a > 0.25 * f).to(torch.uint8) + (a >= 0.75 * f) + (a > 1.25 * f) + (a >= 1.75 * f) + (a > 2.5 * f) + (
        a >= 3.5 * f) + (a > 5 * f)
    code = (code + 8 * torch.signbit(z)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _values(codes, scales):
    """The values of rows of codes and scales, in 32 bits."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    table = torch.cat([table, -table])
    x = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    x = table[x.int()].unflatten(-1, (-1, 16))
    return (x * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _rotate(x, cos, sin, dim, halves):
    """Rotates the last ``dim`` values of x ([T, heads, D])."""
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
    seq, pos = st["seq"].long(), st["pos"].long()
    ang = st["turn"].double()[:, None] * st["freq"]
    cos, sin = ang.cos(), ang.sin()
    # (64 bits: a rotated key may lie next to a rounding's border)
    k = _rotate(st["k"].double(), cos, sin, c["rope"], c["halves"]).bfloat16()
    st["q_out"].copy_(_rotate(st["q"].float(), cos.float(), sin.float(), c["rope"], c["halves"]))
    page, slot = st["table"][seq, pos // P].long(), pos % P
    st["K"][page, :, slot], st["Ks"][page, :, slot] = _quantise(k.float() / st["k_gain"])
    st["V"][page, :, slot], st["Vs"][page, :, slot] = _quantise(st["v"].float() / st["v_gain"])
    st["weight"][seq, :, pos] = 0.0
    st["born"][seq, :, pos] = st["turn"][:, None]
    st["k_out"].copy_(_values(st["K"][page, :, slot], st["Ks"][page, :, slot]) * st["k_gain"])
    st["v_out"].copy_(_values(st["V"][page, :, slot], st["Vs"][page, :, slot]) * st["v_gain"])
    return _outputs(st, "append")


def _rectangle(st, x, fill):
    """x [T, ...] as [B, most tokens, ...]."""
    g = st["g"]
    B, n = len(g["count"]), int(g["count"].max())
    out = torch.full((B * n,) + x.shape[1:], fill, device=DEV, dtype=x.dtype)
    out[st["at"]] = x
    return out.unflatten(0, (B, n))


def _whole(st, codes, scales):
    """Rows of whole sequences in 32 bits: [B, kv heads, slots, D]."""
    t = st["table"].long()
    return _values(st[codes][t].transpose(1, 2).flatten(2, 3), st[scales][t].transpose(1, 2).flatten(2, 3))


def _logits(st):
    """[B, kv heads, tokens, group, slots], -inf past each token's slot."""
    c = st["case"]
    q = _rectangle(st, st["q"].float(), 0.0)
    q = q.unflatten(2, (c["Hkv"], -1)).transpose(1, 2)                  # [B, kv heads, tokens, group, D]
    k = _whole(st, "K", "Ks") * (st["k_gain"] * st["scale"])
    s = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (q.shape[2], -1))
    last = _rectangle(st, st["pos"], -1)
    seen = torch.arange(k.shape[2], device=DEV) <= last[:, None, :, None, None]
    return s.masked_fill_(~seen, -math.inf)


def _tokens(st, x):
    """[B, kv heads, tokens, group, ...] as [T, heads, ...]."""
    x = x.transpose(1, 2).flatten(2, 3).flatten(0, 1)
    return x[st["at"]]


def _attn(st):
    s = _logits(st)
    m = s.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    p = s.sub_(m).exp_()
    den = p.sum(dim=-1, keepdim=True)
    v = _whole(st, "V", "Vs") * st["v_gain"]
    o = (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4]) / den
    st["out"].copy_(_tokens(st, o))
    st["lse"].copy_(_tokens(st, m + den.log())[..., 0])
    return _outputs(st, "attn")


def _weights(st):
    c = st["case"]
    lse = _rectangle(st, st["lse"], 0.0).unflatten(2, (c["Hkv"], -1)).transpose(1, 2)
    p = _logits(st).sub_(lse[..., None]).exp_()
    p = p.sum(dim=(2, 3))
    st["weight"][..., :p.shape[-1]] += p
    return _outputs(st, "weights")


def _evict(st):
    c, P = st["case"], st["case"]["P"]
    w, born, n = st["weight"], st["born"], st["length"].long()[:, None, None]
    ld = w.shape[-1]
    j = torch.arange(ld, device=DEV)
    safe = born > (st["newest"] - c["recent"])[:, None, None]
    key = torch.where(safe, torch.full_like(w, math.inf), w).masked_fill(j >= n, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(safe).scatter_(-1, order[..., :c["budget"]], True) & (j < n)
    end = n.clamp(max=c["budget"])
    hole, mover = ~kept & (j < end), kept & (j >= end)
    # the i-th free slot takes the i-th row from behind the end
    most = int(min(c["budget"], max(1, c["hi"] - c["budget"] + 1)))
    to = torch.where(hole, j, ld).sort(dim=-1).values[..., :most]
    frm = torch.where(mover, j, ld).sort(dim=-1).values[..., :most]
    b, h, i = (to < ld).nonzero(as_tuple=True)
    dst, src = to[b, h, i], frm[b, h, i]
    pd, ps = st["table"][b, dst // P].long(), st["table"][b, src // P].long()
    for x in ("K", "V", "Ks", "Vs"):
        st[x][pd, h, dst % P] = st[x][ps, h, src % P]
    for x in ("weight", "born"):
        y = st[x].clone()
        y[b, h, dst] = y[b, h, src]
        st[x + "_out"].copy_(torch.where(j < end, y, st[x + "_out"]))
    st["length_out"].copy_(end[:, 0, 0])
    return _outputs(st, "evict")


# ------------------------------------------------------------------- exact ---

_E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence and head by head."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attn": _exact_attn, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](st)


def _held64(codes, scales):
    """Rows as the cache holds them: bit fields of the codes and scales spelled out."""
    c = torch.stack([codes % 16, torch.div(codes, 16, rounding_mode="floor")], dim=-1).flatten(-2).long()
    e, m = (c % 8) // 2, c % 2
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e.double() - 1)) * (1 - 2 * (c // 8))
    s = scales.long()
    e, m = (s % 128) // 8, s % 8
    f = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e.double() - 7))
    return v * f.double().repeat_interleave(16, dim=-1)


def _to_grid(z):
    """Rows of 64-bit values quantised: (values as held)."""
    z = z.reshape(z.shape[:-1] + (-1, 16))
    a = np.abs(z)
    top = a.max(axis=-1)
    grid = np.concatenate([np.arange(1, 8) * 2.0 ** -9,
                           ((1 + np.arange(8) / 8) * 2.0 ** np.arange(-6, 9)[:, None]).ravel()[:-1]])
    edge = (grid[1:] + grid[:-1]) / 2                     # ties go to the even mantissa
    at = np.searchsorted(edge, top / 6, side="left")
    tie = (at < len(edge)) & (edge[np.minimum(at, len(edge) - 1)] == top / 6)
    s = grid[at + (tie & (at % 2 == 0))]                  # grid[i] has mantissa i + 1 (mod 8)
    u = a / s[..., None]
    edge = (_E2M1[1:] + _E2M1[:-1]) / 2
    at = np.searchsorted(edge, u, side="left")
    tie = (at < 7) & (edge[np.minimum(at, 6)] == u)
    return (np.sign(z) * _E2M1[at + (tie & (at % 2 == 1))] * s[..., None]).reshape(z.shape[:-2] + (-1,))


def _exact_append(st):
    c, g = st["case"], st["g"]
    T, D, dim = g["T"], c["D"], c["rope"]
    freq = np.array([1.0 / 10000.0 ** (2.0 * i / dim) for i in range(dim // 2)])
    ang = np.outer(g["turn"].astype(np.float64), freq)
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

    weight, born = st["weight"].double(), st["born"].clone()
    for b in range(c["B"]):
        s, n = int(g["start"][b]), int(g["count"][b])
        weight[b, :, s:s + n] = 0
        born[b, :, s:s + n] = torch.from_numpy(g["turn"][g["seq"] == b]).to(DEV)
    k = turned(st["k"]).bfloat16().double().cpu().numpy() / st["k_gain"]  # the rotated key is a bf16 value
    v = st["v"].double().cpu().numpy() / st["v_gain"]
    return dict(k=torch.from_numpy(_to_grid(k) * st["k_gain"]), v=torch.from_numpy(_to_grid(v) * st["v_gain"]),
                q=turned(st["q"]), weight=weight, born=born)


def _spans(g):
    at = 0
    for b, n in enumerate(g["count"]):
        yield b, at, at + int(n)
        at += int(n)


def _rows64(st, b, h, what, gain):
    g, P = st["g"], st["case"]["P"]
    n = int(g["start"][b] + g["count"][b])
    pages = st["table"][b, :(n + P - 1) // P].long()
    return _held64(st[what][pages, h], st[what + "s"][pages, h]).flatten(0, 1)[:n] * gain


def _exact_rows(st, use):
    """Calls use(b, h, tokens, logits [tokens, group, slots]) for blocks of tokens."""
    c, g = st["case"], st["g"]
    G = c["H"] // c["Hkv"]
    for b, i, j in _spans(g):
        for h in range(c["Hkv"]):
            k = _rows64(st, b, h, "K", st["k_gain"])
            for t in range(i, j, 64):
                e = min(t + 64, j)
                q = st["q"][t:e, h * G:(h + 1) * G].double()
                s = (q.flatten(0, 1) @ k.T * st["scale"]).view(e - t, G, -1)
                hide = torch.arange(k.shape[0], device=DEV)[None] > st["pos"][t:e].long()[:, None]
                use(b, h, slice(t, e), s.masked_fill(hide[:, None], -math.inf))


def _exact_attn(st):
    c, g = st["case"], st["g"]
    G = c["H"] // c["Hkv"]
    out = torch.zeros(g["T"], c["H"], c["D"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(g["T"], c["H"], dtype=torch.float64, device=DEV)
    held = {}

    def use(b, h, t, s):
        if held.get("at") != (b, h):
            held.update(at=(b, h), v=_rows64(st, b, h, "V", st["v_gain"]))
        out[t, h * G:(h + 1) * G] = torch.softmax(s, dim=-1) @ held["v"]
        lse[t, h * G:(h + 1) * G] = torch.logsumexp(s, dim=-1)

    _exact_rows(st, use)
    return dict(out=out, lse=lse)


def _exact_weights(st):
    G = st["case"]["H"] // st["case"]["Hkv"]
    weight = st["weight"].double()

    def use(b, h, t, s):
        p = torch.exp(s - st["lse"][t, h * G:(h + 1) * G].double()[..., None])
        weight[b, h, :s.shape[-1]] += p.sum(dim=(0, 1))

    _exact_rows(st, use)
    return weight


def _exact_evict(st):
    c, g, P = st["case"], st["g"], st["case"]["P"]
    cache = {x: st[x].cpu().numpy().copy() for x in ("K", "V", "Ks", "Vs")}
    w, born = st["weight"].double().cpu().numpy(), st["born"].cpu().numpy()
    w_out, born_out = np.zeros_like(w), np.zeros_like(born)
    for b, n in enumerate(int(x) for x in g["start"]):
        keep = min(n, c["budget"])
        for h in range(c["Hkv"]):
            safe = born[b, h, :n] >= n - c["recent"]              # the newest token is number n - 1
            rank = np.lexsort((np.arange(n), -w[b, h, :n], ~safe))
            # slots that are safe rank by place alone
            k = int(safe.sum())
            rank[:k] = np.sort(rank[:k])
            chosen = np.sort(rank[:keep])
            holes = np.setdiff1d(np.arange(keep), chosen)
            movers = chosen[chosen >= keep]
            src = np.arange(keep)
            src[holes] = movers
            w_out[b, h, :keep], born_out[b, h, :keep] = w[b, h, src], born[b, h, src]
            row = g["table"][b]
            for x in cache.values():
                x[row[holes // P], h, holes % P] = x[row[movers // P], h, movers % P]
    return dict(K=torch.from_numpy(cache["K"]), V=torch.from_numpy(cache["V"]), Ks=torch.from_numpy(cache["Ks"]),
                Vs=torch.from_numpy(cache["Vs"]), weight=torch.from_numpy(w_out), born=torch.from_numpy(born_out),
                length=torch.from_numpy(np.minimum(g["start"], c["budget"]).astype(np.int32)))
