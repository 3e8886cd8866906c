"""Measured cases of the serving step's operators over the paged KV cache.

Three kinds of pass, each the calls that a serving loop makes:
  tables   block tables and slot maps grown on the GPU from request lengths, and
           the blocks given back again (a batch that is admitted and preempted)
  decode   one query token per sequence over the paged cache, scores capped by a
           tanh, biased by distance, or limited to a document / window
  prefill  new tokens of every sequence over the paged cache, with the same score
           rules, a prefix visible to every query, and caches of 8-bit codes

`run` computes them in plain torch operations in 32 bits; with `own` set it calls
the library.  `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

D = 128  # head dimension of every attention case
_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of the 64-sequence layer workload: a token each, a block for some.
        {"name": "tables-step-64", "op": "tables", "B": 64, "bs": 16, "blocks": 20000, "start_lo": 1,
         "start_hi": 4095, "new_lo": 1, "new_hi": 1, "lens": 1},
        # Up to 8 drafted tokens for each of 1024 sequences in 256-token blocks.
        {"name": "tables-draft-1024", "op": "tables", "B": 1024, "bs": 256, "blocks": 32768, "start_lo": 256,
         "start_hi": 8184, "new_lo": 1, "new_hi": 8, "lens": 2},
        # 512 prompts admitted at once into a large pool: about a million slots.
        {"name": "tables-admit-512", "op": "tables", "B": 512, "bs": 16, "blocks": 262144, "start_lo": 0,
         "start_hi": 0, "new_lo": 1, "new_hi": 4096, "lens": 3},
        # A handful of short chats: latency of one capped decode call.
        {"name": "decode-cap-short", "op": "decode", "dtype": "bf16", "cache": "16", "Hq": 16, "Hkv": 8, "bs": 256,
         "B": 4, "ctx_lo": 1, "ctx_hi": 500, "softcap": 50.0, "alibi": False, "window": 0, "lens": 4},
        # The 64-sequence multi-head layer with distance-biased scores.
        {"name": "decode-alibi-b64", "op": "decode", "dtype": "fp16", "cache": "16", "Hq": 32, "Hkv": 32, "bs": 16,
         "B": 64, "ctx_lo": 1, "ctx_hi": 4096, "softcap": 0.0, "alibi": True, "window": 0, "lens": 5},
        # Long contexts of which a layer with local attention reads the last 4000 tokens, capped.
        {"name": "decode-cap-window-32k", "op": "decode", "dtype": "bf16", "cache": "16", "Hq": 32, "Hkv": 8,
         "bs": 16, "B": 16, "ctx_lo": 20000, "ctx_hi": 32768, "softcap": 30.0, "alibi": False, "window": 4000,
         "lens": 6},
        # The 128-sequence grouped-query layer over an E4M3 cache, capped.
        {"name": "decode-cap-e4m3-b128", "op": "decode", "dtype": "bf16", "cache": "e4m3", "Hq": 16, "Hkv": 8,
         "bs": 256, "B": 128, "ctx_lo": 256, "ctx_hi": 8192, "softcap": 50.0, "alibi": False, "window": 0, "lens": 7},
        # Whole prompts with capped scores: the largest case.
        {"name": "prefill-cap-8x4k", "op": "prefill", "dtype": "bf16", "cache": "16", "Hq": 32, "Hkv": 8, "bs": 16,
         "B": 8, "start_lo": 0, "start_hi": 0, "n_lo": 3700, "n_hi": 4096, "softcap": 50.0, "alibi": False,
         "doc_lo": 0, "doc_hi": 0, "prefix": 0.0, "lens": 8},
        # Packed documents of ragged lengths: a query sees its own document only.
        {"name": "prefill-documents-2x8k", "op": "prefill", "dtype": "bf16", "cache": "16", "Hq": 16, "Hkv": 8,
         "bs": 256, "B": 2, "start_lo": 0, "start_hi": 0, "n_lo": 8000, "n_hi": 8192, "softcap": 0.0, "alibi": False,
         "doc_lo": 60, "doc_hi": 2500, "prefix": 0.0, "lens": 9},
        # Short prompts, multi-head, whose first part is visible to every query, with distance-biased scores.
        {"name": "prefill-prefix-alibi", "op": "prefill", "dtype": "fp16", "cache": "16", "Hq": 32, "Hkv": 32,
         "bs": 16, "B": 12, "start_lo": 0, "start_hi": 300, "n_lo": 33, "n_hi": 700, "softcap": 0.0, "alibi": True,
         "doc_lo": 0, "doc_hi": 0, "prefix": 0.5, "lens": 10},
        # Chunked prefill: the last 512 positions of long contexts over an E4M3 cache.
        {"name": "prefill-e4m3-chunk", "op": "prefill", "dtype": "bf16", "cache": "e4m3", "Hq": 32, "Hkv": 8,
         "bs": 16, "B": 8, "start_lo": 3000, "start_hi": 7680, "n_lo": 512, "n_hi": 512, "softcap": 0.0,
         "alibi": False, "doc_lo": 0, "doc_hi": 0, "prefix": 0.0, "lens": 11},
        # A few short spans over an int8 cache: latency.
        {"name": "prefill-int8-short", "op": "prefill", "dtype": "fp16", "cache": "int8", "Hq": 16, "Hkv": 8,
         "bs": 64, "B": 3, "start_lo": 0, "start_hi": 500, "n_lo": 1, "n_hi": 100, "softcap": 0.0, "alibi": False,
         "doc_lo": 0, "doc_hi": 0, "prefix": 0.0, "lens": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "decode", "prefill", "prefill"])
    lens = rng.randrange(1 << 30)
    if op == "tables":
        bs = rng.choice([16, 32, 64, 256])
        B = _log_int(rng, 1, 1024)
        new = _log_int(rng, 1, 4096 if B <= 512 else 500)
        start = rng.choice([0, _log_int(rng, 1, 8000)])
        need = B * ((start + new) // bs + 2)
        return {"op": "tables", "B": B, "bs": bs, "blocks": min(262144, need + _log_int(rng, 1, 200000)),
                "start_lo": min(start, 1), "start_hi": start, "new_lo": 1, "new_hi": new, "lens": lens}
    Hq, Hkv = rng.choice([(8, 8), (16, 8), (32, 8), (64, 8), (32, 32), (16, 16), (4, 1)])
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "cache": rng.choice(["16", "16", "e4m3", "int8"]),
            "Hq": Hq, "Hkv": Hkv, "bs": rng.choice([16, 32, 64, 256]),
            "softcap": rng.choice([0.0, 30.0, 50.0]), "alibi": rng.random() < 0.3, "lens": lens}
    if op == "decode":
        hi = _log_int(rng, 16, 32768)
        B = _log_int(rng, 1, max(1, min(700, 500000 // hi)))
        window = rng.choice([0, 0, _log_int(rng, 1, 5000)])
        return {**case, "B": B, "ctx_lo": max(1, hi // rng.choice([1, 2, 100])), "ctx_hi": hi, "window": window}
    n = _log_int(rng, 1, 4096)
    start = rng.choice([0, _log_int(rng, 1, 8192)])
    # the padded score matrix of the plain form stays below the largest listed case's
    B = _log_int(rng, 1, max(1, min(64, 3_500_000_000 // (Hq * n * (start + n)))))
    doc = rng.choice([0, 0, _log_int(rng, 2, 3000)])
    return {**case, "B": B, "start_lo": start // 2, "start_hi": start, "n_lo": max(1, n // rng.choice([1, 2, 50])),
            "n_hi": n, "doc_lo": max(1, doc // 20) if doc else 0, "doc_hi": doc,
            "prefix": rng.choice([0.0, 0.0, 0.3, 1.0])}


# ------------------------------------------------------------------ lengths: by the case alone
def _tables_lens(case):
    r = random.Random(case["lens"])
    starts = [r.randint(case["start_lo"], case["start_hi"]) for _ in range(case["B"])]
    ends = [s + r.randint(case["new_lo"], case["new_hi"]) for s in starts]
    return starts, ends


def _decode_lens(case):
    r = random.Random(case["lens"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    first = [max(0, c - case["window"]) if case["window"] else 0 for c in ctx]
    return ctx, first


def _prefill_lens(case):
    """(starts, new tokens, prefix lengths, first visible key of every query in order)."""
    r = random.Random(case["lens"])
    starts = [r.randint(case["start_lo"], case["start_hi"]) for _ in range(case["B"])]
    ns = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["B"])]
    prefix = [int(case["prefix"] * r.random() * (s + n)) for s, n in zip(starts, ns)]
    first = []
    for s, n in zip(starts, ns):
        at, nxt = 0, 0
        for p in range(s + n):
            if case["doc_hi"] and p == nxt:
                at, nxt = p, p + r.randint(case["doc_lo"], case["doc_hi"])
            if p >= s:
                first.append(at)
    return starts, ns, prefix, first


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ inputs
def _i32(values, dev="cuda"):
    return torch.tensor(values, dtype=torch.int32).to(dev)


def _tables(lens, bs, g, spare=3):
    """Block tables over a permuted pool, -1 past each sequence's last block; (tables, pool blocks)."""
    used = [_ceil(n, bs) for n in lens]
    pool = sum(used) + spare
    perm = torch.randperm(pool, generator=g)
    table = torch.full((len(lens), max(max(used), 1)), -1, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u].to(torch.int32)
        at += u
    return table.cuda(), pool


def _cache(case, pool, gd):
    """(cache, scales): values of unit size, whose blocks differ in magnitude where the cache holds codes."""
    shape = (pool, case["bs"], case["Hkv"], D)
    if case["cache"] == "16":
        return torch.randn(shape, generator=gd, device="cuda", dtype=_DTYPE[case["dtype"]]), None
    gain = torch.exp(0.5 * torch.randn((pool, 1, case["Hkv"], 1), generator=gd, device="cuda"))
    x = torch.randn(shape, generator=gd, device="cuda") * gain
    top = 448.0 if case["cache"] == "e4m3" else 127.0
    scale = x.abs().amax(dim=(1, 3)) / top
    x = x / scale[:, None, :, None]
    if case["cache"] == "e4m3":
        return x.to(torch.float8_e4m3fn).view(torch.uint8), scale
    return x.round().clamp(-127, 127).to(torch.int8), scale


def _attention_inputs(case, lens, rows, g, seed):
    gd = torch.Generator(device="cuda").manual_seed(seed)
    tables, pool = _tables(lens, case["bs"], g)
    k, ks = _cache(case, pool, gd)
    v, vs = _cache(case, pool, gd)
    # queries three times unit size: scores of a few units, where the cap and the softmax both act
    q = (3 * torch.randn((rows, case["Hq"], D), generator=gd, device="cuda")).to(_DTYPE[case["dtype"]])
    slopes = None
    if case["alibi"]:
        h = torch.arange(1, case["Hq"] + 1, dtype=torch.float64)
        slopes = torch.exp2(-8 * h / case["Hq"]).to(torch.float32).cuda()
    return {"q": q, "k": k, "v": v, "k_scale": ks, "v_scale": vs, "tables": tables, "slopes": slopes,
            "scale": 1 / math.sqrt(D), "softcap": case["softcap"], "op": case["op"], "bs": case["bs"]}


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    if case["op"] == "tables":
        bs = case["bs"]
        starts, ends = _tables_lens(case)
        held = [_ceil(s, bs) for s in starts]
        grown = [_ceil(e, bs) for e in ends]
        perm = torch.randperm(case["blocks"], generator=g)
        ref = torch.zeros(case["blocks"], dtype=torch.int32)
        table = torch.full((case["B"], max(grown)), -1, dtype=torch.int32)
        at = 0
        for b, u in enumerate(held):
            table[b, :u] = perm[at:at + u].to(torch.int32)
            at += u
        ref[perm[:at]] = 1
        others = (case["blocks"] - at - sum(grown) + sum(held)) // 2  # blocks of sequences outside this batch
        if others > 0:
            ref[perm[at:at + others]] = 1
        total = sum(e - s for s, e in zip(starts, ends))
        return {"op": "tables", "tables": table.cuda(), "ref": ref.cuda(), "starts": _i32(starts), "ends": _i32(ends),
                "bs": bs, "tokens": total}
    if case["op"] == "decode":
        ctx, first = _decode_lens(case)
        st = _attention_inputs(case, ctx, case["B"], g, seed)
        st.update(ctx=_i32(ctx), first=_i32(first) if case["window"] else None, max_ctx=case["ctx_hi"])
        return st
    starts, ns, prefix, first = _prefill_lens(case)
    st = _attention_inputs(case, [s + n for s, n in zip(starts, ns)], sum(ns), g, seed)
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    st.update(starts=_i32(starts), cu=_i32(cu), max_q=max(ns), prefix=_i32(prefix) if case["prefix"] else None,
              first=_i32(first) if case["doc_hi"] else None)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "tables":
        return _plain_tables(state)
    if state["op"] == "decode":
        return _plain_decode(state)
    return _plain_prefill(state)


def _run_own(st):
    import pagedattention_decode_pkv_gb300 as pkv

    if st["op"] == "tables":
        cu, slots = pkv.pkv_grow_block_tables(st["tables"], st["starts"], st["ends"], st["ref"], st["bs"],
                                              num_new_tokens=st["tokens"])
        pkv.pkv_shrink_block_tables(st["tables"], st["starts"], st["ends"], st["ref"], st["bs"])
        return cu, slots, st["tables"], st["ref"]
    mods = dict(softcap=st["softcap"], alibi_slopes=st["slopes"], key_starts=st["first"], k_scale=st["k_scale"],
                v_scale=st["v_scale"])
    if st["op"] == "decode":
        return pkv.pkv_paged_attention_decode_mod(st["q"], st["k"], st["v"], st["tables"], st["ctx"], st["scale"],
                                                  st["max_ctx"], **mods)
    return pkv.pkv_paged_attention_prefill_mod(st["q"], st["k"], st["v"], st["tables"], st["starts"], st["cu"],
                                               st["scale"], st["max_q"], prefix_lens=st["prefix"], **mods)


def _plain_tables(st):
    bs, table, ref = st["bs"], st["tables"], st["ref"]
    starts, ends = st["starts"].long(), st["ends"].long()
    held, grown = (starts + bs - 1) // bs, (ends + bs - 1) // bs
    need = grown - held
    upto = torch.cumsum(need, 0)
    free = ref == 0
    rank = torch.cumsum(free, 0) - 1
    granted = (need == 0) | (upto <= free.sum())
    ids = torch.arange(ref.numel(), device=ref.device)
    by_rank = torch.zeros(ref.numel() + 1, dtype=torch.int64, device=ref.device)
    by_rank.scatter_(0, torch.where(free, rank, ref.numel()), ids)  # the lowest free block first
    ref += (free & (rank < (need * granted).sum())).to(torch.int32)
    j = torch.arange(table.shape[1], device=ref.device)[None]
    fresh = (j >= held[:, None]) & (j < grown[:, None])
    at = (upto - need)[:, None] + j - held[:, None]
    new = torch.where(granted[:, None], by_rank[at.clamp(0, ref.numel() - 1)], -1)
    table.copy_(torch.where(fresh, new.to(torch.int32), table))
    cu = torch.zeros(starts.numel() + 1, dtype=torch.int32, device=ref.device)
    cu[1:] = torch.cumsum(ends - starts, 0)
    k = torch.arange(st["tokens"], device=ref.device)
    b = torch.searchsorted(cu[1:].long(), k, right=True)
    p = starts[b] + k - cu[b]
    slots = torch.where(granted[b], table[b, p // bs].long() * bs + p % bs, -1).to(torch.int32)
    # give the new blocks back
    gone = fresh & (table >= 0)
    ref.index_add_(0, torch.where(gone, table, 0).flatten(), -gone.flatten().to(torch.int32))
    table.masked_fill_(fresh, -1)
    return cu, slots, table, ref


def _rows(cache, scale, tables):
    """Every table entry's rows in order: [B, entries * bs, Hkv, d] in 32 bits (missing blocks read block 0)."""
    ids = tables.long().clamp(min=0)
    x = cache[ids]
    if cache.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn)
    x = x.float()
    if scale is not None:
        x = x * scale[ids][:, :, None, :, None]
    return x.flatten(1, 2)


def _plain_attention(st, q, pos, visible):
    """q [B, n, Hq, d], pos [B, n], visible [B, n, T] -> [B, n, Hq, d]; rows that see nothing are zero."""
    k, v = _rows(st["k"], st["k_scale"], st["tables"]), _rows(st["v"], st["v_scale"], st["tables"])
    B, n, Hq, _ = q.shape
    T, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    qg = q.float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    s = qg @ k.permute(0, 2, 3, 1)
    s *= st["scale"]
    if st["softcap"]:
        s = st["softcap"] * torch.tanh_(s.div_(st["softcap"]))
    s = s.view(B, Hkv, G, n, T)
    if st["slopes"] is not None:
        far = (torch.arange(T, device=q.device)[None, None] - pos[:, :, None]).abs().float()
        s -= st["slopes"].view(1, Hkv, G, 1, 1) * far[:, None, None]
    s.masked_fill_(~visible[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, G * n, T) @ v.permute(0, 2, 1, 3)
    o = o.view(B, Hkv, G, n, D) / torch.where(total > 0, total, 1)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).to(q.dtype)


def _plain_decode(st):
    ctx = st["ctx"].long()
    t = torch.arange(st["tables"].shape[1] * st["bs"], device=ctx.device)[None, None]
    seen = t < ctx[:, None, None]
    if st["first"] is not None:
        seen = seen & (t >= st["first"][:, None, None])
    return _plain_attention(st, st["q"][:, None], ctx[:, None] - 1, seen)[:, 0]


def _plain_prefill(st):
    starts, cu = st["starts"].long(), st["cu"].long()
    rows = st["q"].shape[0]
    i = torch.arange(st["max_q"], device=cu.device)[None]
    at = (cu[:-1, None] + i).clamp(max=rows - 1)  # a padded batch of rows; what is past a sequence is not taken back
    pos = starts[:, None] + i
    t = torch.arange(st["tables"].shape[1] * st["bs"], device=cu.device)[None, None]
    seen = t <= pos[:, :, None]
    if st["prefix"] is not None:
        seen = seen | (t < st["prefix"][:, None, None])
    seen = seen & (t < (starts + cu[1:] - cu[:-1])[:, None, None])
    if st["first"] is not None:
        seen = seen & (t >= st["first"][at][:, :, None])
    o = _plain_attention(st, st["q"][at], pos, seen)
    r = torch.arange(rows, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), r, right=True)
    return o[b, r - cu[b]]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "tables":
        starts, ends = _tables_lens(case)
        new = sum(_ceil(e, case["bs"]) - _ceil(s, case["bs"]) for s, e in zip(starts, ends))
        tokens = sum(e - s for s, e in zip(starts, ends))
        # counts read; per new block its count and table entry written, then both again; lengths, offsets, slots
        return {"bytes": 4 * case["blocks"] + 4 * 4 * new + 3 * 4 * case["B"] + 4 * tokens, "flops": 0}
    es = 2 if case["cache"] == "16" else 1
    if case["op"] == "decode":
        ctx, first = _decode_lens(case)
        spans = list(zip(first, ctx))
        rows, pairs = case["B"], sum(c - f for f, c in spans)
    else:
        starts, ns, prefix, first = _prefill_lens(case)
        spans, pairs, at = [], 0, 0
        for s, n, x in zip(starts, ns, prefix):
            lo = s + n
            for p in range(s, s + n):
                f, e = first[at], max(p + 1, x)
                pairs += max(0, e - f)
                lo = min(lo, f)
                at += 1
            spans.append((lo, s + n))
        rows = sum(ns)
    row_bytes = 2 * case["Hkv"] * D * es
    blocks = sum(_ceil(e, case["bs"]) - f // case["bs"] for f, e in spans)
    size = sum(e - f for f, e in spans) * row_bytes + blocks * (4 + (0 if es == 2 else 8 * case["Hkv"]))
    size += 2 * rows * case["Hq"] * D * 2 + 4 * rows
    return {"bytes": size, "flops": 4 * D * case["Hq"] * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    if case["op"] == "tables":
        return None
    st = prepare(case, seed)
    if case["op"] == "decode":
        ctx, first = _decode_lens(case)
        queries = [(c, c, [f], 0, slice(b, b + 1)) for b, (c, f) in enumerate(zip(ctx, first))]
    else:
        starts, ns, prefix, first = _prefill_lens(case)
        queries, at = [], 0
        for s, n, x in zip(starts, ns, prefix):
            queries.append((s + 1, s + n, first[at:at + n], x, slice(at, at + n)))
            at += n
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    G = case["Hq"] // case["Hkv"]
    e4m3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().cuda()
    for b, (seen0, T, lows, prefix_len, rows) in enumerate(queries):  # seen0: keys up to the first query's own
        blocks = st["tables"][b, :_ceil(T, case["bs"])].long()
        low = torch.tensor(lows, device="cuda")[:, None]
        here = torch.arange(seen0 - 1, T, device="cuda")[:, None]
        key = torch.arange(T, device="cuda")[None]
        hidden = (key < low) | ((key > here) & (key >= prefix_len))
        for h in range(case["Hkv"]):
            kv = []
            for cache, scale in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
                x = cache[blocks, :, h]
                x = e4m3[x.long()] if case["cache"] == "e4m3" else x.double()
                if scale is not None:
                    x = x * scale[blocks, h].double()[:, None, None]
                kv.append(x.reshape(-1, D)[:T])
            for hq in range(h * G, h * G + G):
                s = (st["q"][rows, hq].double() * st["scale"]) @ kv[0].T
                if case["softcap"]:
                    s = torch.tanh(s / case["softcap"]) * case["softcap"]
                if case["alibi"]:
                    s -= st["slopes"][hq].double() * (key - here).abs()
                s[hidden] = -math.inf
                w = torch.softmax(s, dim=-1)
                out[rows, hq] = torch.where(hidden.all(1, keepdim=True), 0.0, w @ kv[1])
    return out
