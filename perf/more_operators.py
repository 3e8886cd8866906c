"""Measured cases of the rotary and 4-bit cache operators of a serving step.

Five kinds of pass, each the calls that a serving loop makes:
  rope     rotary positions of the step's queries and keys, keys and values written
           into the paged cache of their own type
  quant    the same into a cache of 4-bit codes, quantised as it is written (or
           quantised as it stands), and the cache read back
  load     rows of a 4-bit cache read back through a slot map
  decode   one query token per sequence over the 4-bit paged cache
  prefill  new tokens of every sequence over the 4-bit paged cache

`run` computes them in plain torch operations, in 32 bits, and in 64 where a value's
side of a rounding border, or a far position's angle, would be lost; with `own` set it
calls the library.  `exact` is the definition in 64 bits.

A 4-bit cache holds, for every (block, KV head, token), head_dim / 2 bytes of codes and
one float16 scale per 32 dims.  A nibble u stands for scale * (u - 8).  The eight dims
of four bytes are in the order 0 2, 4 6, 1 3, 5 7 (low nibble first).
"""
import math
import random

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROUP = 32           # dims that share a scale
TOP_SCALE = 9344.0   # 7 times it is the largest such value that float16 holds


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of the 64-sequence multi-head layer: a token each.
        {"name": "rope-step-64", "op": "rope", "dtype": "fp16", "Hq": 32, "Hkv": 32, "d": 128, "bs": 16, "N": 64,
         "pool": 20000, "pos_hi": 4096, "rot": 128, "interleaved": False, "scaling": "none", "factor": 1.0, "pad": 0,
         "lens": 1},
        # Prompts of a long-context layer, a quarter of each head rotated, pairs side by side.
        {"name": "rope-prompts-16k", "op": "rope", "dtype": "bf16", "Hq": 32, "Hkv": 8, "d": 128, "bs": 16, "N": 16381,
         "pool": 1100, "pos_hi": 131072, "rot": 32, "interleaved": True, "scaling": "yarn", "factor": 32.0, "pad": 5,
         "lens": 2},
        # One decode step of the 128-sequence grouped-query layer into a 4-bit cache.
        {"name": "quant-step-128", "op": "quant", "dtype": "bf16", "Hq": 16, "Hkv": 8, "d": 128, "bs": 16, "N": 128,
         "pool": 128, "pos_hi": 8192, "rot": 128, "interleaved": False, "scaling": "linear", "factor": 4.0, "pad": 0,
         "lens": 3},
        # Prompts of the long-context layer written as 4-bit codes.
        {"name": "quant-prompts-32k", "op": "quant", "dtype": "bf16", "Hq": 32, "Hkv": 8, "d": 128, "bs": 16, "N": 32700,
         "pool": 2048, "pos_hi": 32768, "rot": 128, "interleaved": False, "scaling": "ntk", "factor": 8.0, "pad": 11,
         "lens": 4},
        # Rows whose positions are applied already (or that have none), multi-head.
        {"name": "quant-rows-5k", "op": "quant", "dtype": "fp16", "Hq": 0, "Hkv": 32, "d": 128, "bs": 16, "N": 5003,
         "pool": 320, "pos_hi": 0, "rot": 0, "interleaved": False, "scaling": "none", "factor": 1.0, "pad": 3, "lens": 5},
        # One short context read back.
        {"name": "load-300", "op": "load", "dtype": "fp16", "Hkv": 8, "d": 128, "bs": 256, "N": 300, "pool": 16, "pad": 0,
         "lens": 6},
        # The contexts of a batch read back in order, to hand them on in 16 bits.
        {"name": "load-131k", "op": "load", "dtype": "bf16", "Hkv": 8, "d": 128, "bs": 16, "N": 131001, "pool": 10000,
         "pad": 77, "lens": 7},
        # A handful of short chats: latency of one decode call.
        {"name": "decode-short", "op": "decode", "dtype": "bf16", "Hq": 16, "Hkv": 8, "d": 128, "bs": 256, "B": 4,
         "ctx_lo": 1, "ctx_hi": 500, "softcap": 0.0, "alibi": False, "window": 0, "lens": 8},
        # The 64-sequence multi-head layer.
        {"name": "decode-b64", "op": "decode", "dtype": "fp16", "Hq": 32, "Hkv": 32, "d": 128, "bs": 16, "B": 64,
         "ctx_lo": 1, "ctx_hi": 4096, "softcap": 0.0, "alibi": False, "window": 0, "lens": 9},
        # Eight long contexts of the grouped-query layer.
        {"name": "decode-8x32k", "op": "decode", "dtype": "bf16", "Hq": 32, "Hkv": 8, "d": 128, "bs": 16, "B": 8,
         "ctx_lo": 32768, "ctx_hi": 32768, "softcap": 0.0, "alibi": False, "window": 0, "lens": 10},
        # Chunked prefill: the last 512 positions of long contexts.
        {"name": "prefill-chunk", "op": "prefill", "dtype": "bf16", "Hq": 32, "Hkv": 8, "d": 128, "bs": 16, "B": 8,
         "start_lo": 3000, "start_hi": 7680, "n_lo": 512, "n_hi": 512, "softcap": 0.0, "alibi": False, "doc_lo": 0,
         "doc_hi": 0, "prefix": 0.0, "lens": 11},
        # Whole prompts: the largest case.
        {"name": "prefill-8x4k", "op": "prefill", "dtype": "fp16", "Hq": 32, "Hkv": 8, "d": 128, "bs": 16, "B": 8,
         "start_lo": 0, "start_hi": 0, "n_lo": 3700, "n_hi": 4096, "softcap": 0.0, "alibi": False, "doc_lo": 0,
         "doc_hi": 0, "prefix": 0.0, "lens": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "quant", "load", "decode", "decode", "prefill"])
    lens = rng.randrange(1 << 30)
    Hq, Hkv = rng.choice([(8, 8), (16, 8), (32, 8), (64, 8), (32, 32), (16, 16), (4, 1), (12, 2)])
    bs = rng.choice([16, 32, 64, 256])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("rope", "quant", "load"):
        d = rng.choice([64, 96, 128, 128, 256])
        N = _log_int(rng, 1, 40_000_000 // ((Hq + 2 * Hkv) * d))
        case = {"op": op, "dtype": dtype if op == "quant" else rng.choice(["bf16", "fp16", "fp32"]), "Hkv": Hkv, "d": d,
                "bs": bs, "N": N, "pool": -(-N // bs) + _log_int(rng, 1, 200), "pad": rng.choice([0, 0, 1 + N // 50]),
                "lens": lens}
        if op == "load":
            return case
        bare = op == "quant" and rng.random() < 0.25
        scaling = "none" if bare else rng.choice(["none", "linear", "ntk", "yarn"])
        return {**case, "Hq": 0 if bare else Hq, "pos_hi": 0 if bare else _log_int(rng, 64, 1_000_000),
                "rot": 0 if bare else rng.choice([d, d, d // 2, d // 4, 20, 2]), "interleaved": rng.random() < 0.5,
                "scaling": scaling, "factor": 1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0])}
    case = {"op": op, "dtype": dtype, "Hq": Hq, "Hkv": Hkv, "bs": bs, "softcap": rng.choice([0.0, 0.0, 30.0]),
            "alibi": rng.random() < 0.25, "lens": lens}
    if op == "decode":
        hi = _log_int(rng, 16, 32768)
        B = _log_int(rng, 1, max(1, min(700, 250000 // hi)))
        return {**case, "d": rng.choice([64, 128, 128, 256]), "B": B, "ctx_lo": max(1, hi // rng.choice([1, 2, 100])),
                "ctx_hi": hi, "window": rng.choice([0, 0, _log_int(rng, 1, 5000)])}
    Hq, Hkv = rng.choice([(8, 8), (16, 8), (32, 8), (64, 8), (32, 32), (4, 1)])
    n = _log_int(rng, 1, 4096)
    start = rng.choice([0, _log_int(rng, 1, 8192)])
    # the padded score matrix of the plain form stays below the largest listed case's
    B = _log_int(rng, 1, max(1, min(64, 3_500_000_000 // (Hq * n * (start + n)))))
    doc = rng.choice([0, 0, _log_int(rng, 2, 3000)])
    return {**case, "Hq": Hq, "Hkv": Hkv, "d": 128, "B": B, "start_lo": start // 2, "start_hi": start,
            "n_lo": max(1, n // rng.choice([1, 2, 50])), "n_hi": n, "doc_lo": max(1, doc // 20) if doc else 0,
            "doc_hi": doc, "prefix": rng.choice([0.0, 0.0, 0.5])}


# ------------------------------------------------------------------ lengths: by the case alone
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


# ------------------------------------------------------------------ the 4-bit format
def _scales(x):
    """float16 scales of x [..., d] in 64 bits: the largest of 32 dims over 7, 8 significant bits, ties to even."""
    top = x.unflatten(-1, (-1, GROUP)).abs().amax(-1) / 7
    m, e = torch.frexp(top)
    return torch.ldexp(torch.round(m * 256), e - 8).clamp(max=TOP_SCALE).to(torch.float16)


def _codes(x, scales):
    """Nibbles 1 .. 15 of x [..., d] in 64 bits."""
    s = scales.double()[..., None]
    c = torch.round(x.unflatten(-1, (-1, GROUP)) / torch.where(s > 0, s, 1.0)).clamp(-7, 7)
    return (torch.where(s > 0, c, 0.0) + 8).to(torch.uint8).flatten(-2)


def _pack(u):
    u = u.unflatten(-1, (-1, 8))
    lo, hi = u[..., [0, 4, 1, 5]], u[..., [2, 6, 3, 7]]
    return (lo | hi << 4).flatten(-2)


def _values(codes, scales, dtype=torch.float32):
    """What codes [..., d / 2] and scales [..., d / 32] stand for, [..., d]."""
    b = codes.unflatten(-1, (-1, 4))
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2)  # dims 0 2 4 6 1 3 5 7
    c = n[..., [0, 4, 1, 5, 2, 6, 3, 7]].flatten(-2).to(dtype) - 8
    return (c.unflatten(-1, (-1, GROUP)) * scales.to(dtype)[..., None]).flatten(-2)


def _random_cache(pool, Hkv, bs, d, gd):
    """Codes and scales of values whose dims differ in magnitude, as keys' do."""
    gain = torch.exp(0.5 * torch.randn((1, Hkv, 1, d), generator=gd, device="cuda"))
    codes, scales = [], []
    step = max(1, (1 << 26) // (Hkv * bs * d))
    for at in range(0, pool, step):
        x = torch.randn((min(step, pool - at), Hkv, bs, d), generator=gd, device="cuda") * gain
        s = _scales(x.double())
        u = torch.round(x.unflatten(-1, (-1, GROUP)) / s.float()[..., None]).clamp(-7, 7) + 8
        codes.append(_pack(u.to(torch.uint8).flatten(-2)))
        scales.append(s)
    return torch.cat(codes), torch.cat(scales)


# ------------------------------------------------------------------ rotary frequencies
BASE, ORIGINAL = 10000.0, 4096


def _frequencies(case):
    """(float64 angle per position of each pair, amplitude)."""
    r = case["rot"]
    i = torch.arange(r // 2, dtype=torch.float64)
    base, factor, kind = BASE, case["factor"], case["scaling"]
    if kind == "ntk" and r > 2:
        base = base * factor ** (r / (r - 2))
    f = base ** (-2 * i / r)
    if kind == "linear":
        f = f / factor
    if kind == "yarn":  # pairs that turn 32 times and more over the original length stay, those below once are stretched
        keep = ((ORIGINAL * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        return f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


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


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    op, d, bs, Hkv, dtype = case["op"], case["d"], case["bs"], case["Hkv"], _DTYPE[case["dtype"]]
    st = {"op": op, "bs": bs, "dtype": dtype}
    if op in ("rope", "quant", "load"):
        N, pool = case["N"], case["pool"]
        slots = torch.randperm(pool * bs, generator=g)[:N].to(torch.int32)
        if case["pad"]:  # rows of a padded batch that are not written
            slots[N - case["pad"]:] = -1
        st["slots"] = slots.cuda()
        if op == "rope":
            st["k"] = torch.randn((pool, bs, Hkv, d), generator=gd, device="cuda", dtype=dtype)
            st["v"] = torch.randn((pool, bs, Hkv, d), generator=gd, device="cuda", dtype=dtype)
        else:
            st["k"], st["ks"] = _random_cache(pool, Hkv, bs, d, gd)
            st["v"], st["vs"] = _random_cache(pool, Hkv, bs, d, gd)
        if op == "load":
            return st
        # one projection's output: a token's query, key and value heads side by side
        Hq = case["Hq"]
        qkv = torch.randn((N, Hq + 2 * Hkv, d), generator=gd, device="cuda")
        qkv[:, Hq:Hq + Hkv] *= torch.exp(0.5 * torch.randn((Hkv, d), generator=gd, device="cuda"))
        qkv = qkv.to(dtype)
        st["q"], st["key"], st["value"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st["rot"], st["interleaved"] = case["rot"], case["interleaved"]
        st["all"] = torch.arange(pool * bs, dtype=torch.int32, device="cuda")
        if case["rot"]:
            st["pos"] = torch.randint(0, case["pos_hi"], (N,), generator=g, dtype=torch.int32).cuda()
            f, st["amplitude"] = _frequencies(case)
            st["freq"] = f.cuda()
            if own:
                import pagedattention_decode_pkv_gb300 as pkv

                st["rope"] = pkv.pkv_rope_frequencies(
                    case["rot"], BASE, scaling=None if case["scaling"] == "none" else case["scaling"],
                    factor=case["factor"], original_len=ORIGINAL, device="cuda")
        return st
    if op == "decode":
        ctx, first = _decode_lens(case)
        rows, lens = case["B"], ctx
        st.update(ctx=_i32(ctx), first=_i32(first) if case["window"] else None, max_ctx=case["ctx_hi"], prefix=None)
    else:
        starts, ns, prefix, first = _prefill_lens(case)
        rows, lens = sum(ns), [s + n for s, n in zip(starts, ns)]
        cu = [0]
        for n in ns:
            cu.append(cu[-1] + n)
        st.update(starts=_i32(starts), cu=_i32(cu), max_q=max(ns), prefix=_i32(prefix) if case["prefix"] else None,
                  first=_i32(first) if case["doc_hi"] else None)
    st["tables"], pool = _tables(lens, bs, g)
    st["k"], st["ks"] = _random_cache(pool, Hkv, bs, d, gd)
    st["v"], st["vs"] = _random_cache(pool, Hkv, bs, d, gd)
    # queries three times unit size: scores of a few units, where the cap and the softmax both act
    st["q"] = (3 * torch.randn((rows, case["Hq"], d), generator=gd, device="cuda")).to(dtype)
    st["slopes"] = None
    if case["alibi"]:
        h = torch.arange(1, case["Hq"] + 1, dtype=torch.float64)
        st["slopes"] = torch.exp2(-8 * h / case["Hq"]).to(torch.float32).cuda()
    st.update(scale=1 / math.sqrt(d), softcap=case["softcap"])
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope_store, "quant": _plain_quant, "load": _plain_load, "decode": _plain_decode,
            "prefill": _plain_prefill}[state["op"]](state)


def _run_own(st):
    import pagedattention_decode_pkv_gb300 as pkv

    op = st["op"]
    if op == "rope":
        q = pkv.pkv_rope_store_kvcache(st["q"], st["key"], st["value"], st["pos"], st["rope"], st["k"], st["v"], st["slots"],
                                       interleaved=st["interleaved"])
        return q, st["k"], st["v"]
    cache = (st["k"], st["v"], st["ks"], st["vs"])
    if op == "load":
        return pkv.pkv_load_kvcache_int4(*cache, st["slots"], st["dtype"])
    if op == "quant":
        if st["rot"]:
            q = pkv.pkv_rope_store_kvcache_int4(st["q"], st["key"], st["value"], st["pos"], st["rope"], *cache, st["slots"],
                                                interleaved=st["interleaved"])
            return q, *pkv.pkv_load_kvcache_int4(*cache, st["all"], st["dtype"])
        pkv.pkv_store_kvcache_int4(st["key"], st["value"], *cache, st["slots"])
        return pkv.pkv_load_kvcache_int4(*cache, st["all"], st["dtype"])
    mods = dict(softcap=st["softcap"], alibi_slopes=st["slopes"], key_starts=st["first"])
    if op == "decode":
        return pkv.pkv_paged_attention_decode_int4(st["q"], *cache, st["tables"], st["ctx"], st["scale"], st["max_ctx"], **mods)
    return pkv.pkv_paged_attention_prefill_int4(st["q"], *cache, st["tables"], st["starts"], st["cu"], st["scale"],
                                                st["max_q"], prefix_lens=st["prefix"], **mods)


def _plain_rotate(st, x, dtype):
    """Rotates the first dims of x [N, H, d] in `dtype`; angles and their sines in 64 bits."""
    r = st["rot"]
    angle = st["pos"].double()[:, None] * st["freq"]
    cos, sin = (angle.cos() * st["amplitude"]).to(dtype)[:, None], (angle.sin() * st["amplitude"]).to(dtype)[:, None]
    y = x.to(dtype)
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if st["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([ra, rb], -1).flatten(-2) if st["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([turned, y[..., r:]], -1)


def _plain_rope_store(st):
    q = _plain_rotate(st, st["q"], torch.float32).to(st["dtype"])
    key = _plain_rotate(st, st["key"], torch.float32).to(st["dtype"])
    live = st["slots"] >= 0
    at = st["slots"][live].long()
    st["k"].flatten(0, 1)[at] = key[live]
    st["v"].flatten(0, 1)[at] = st["value"][live]
    return q, st["k"], st["v"]


def _plain_rows(st, slots):
    """Rows of the 4-bit caches in the passes' type; slots of -1 read as zero."""
    at = slots.long().clamp(min=0)
    b, o = at // st["bs"], at % st["bs"]
    live = (slots >= 0)[:, None, None]
    return tuple(torch.where(live, _values(c[b, :, o], s[b, :, o]), 0.0).to(st["dtype"])
                 for c, s in ((st["k"], st["ks"]), (st["v"], st["vs"])))


def _plain_quant(st):
    out = ()
    key, value = st["key"].double(), st["value"].double()
    if st["rot"]:
        out = (_plain_rotate(st, st["q"], torch.float32).to(st["dtype"]),)
        key = _plain_rotate(st, st["key"], torch.float64)  # a value's side of a rounding border
    live = st["slots"] >= 0
    at = st["slots"][live].long()
    b, o = at // st["bs"], at % st["bs"]
    for x, c, s in ((key, st["k"], st["ks"]), (value, st["v"], st["vs"])):
        scales = _scales(x[live])
        c[b, :, o] = _pack(_codes(x[live], scales))
        s[b, :, o] = scales
    return out + _plain_rows(st, st["all"])


def _plain_load(st):
    return _plain_rows(st, st["slots"])


def _plain_attention(st, q, pos, visible):
    """q [B, n, Hq, d], pos [B, n], visible [B, n, T] -> [B, n, Hq, d]; rows that see nothing are zero."""
    ids = st["tables"].long().clamp(min=0)
    k, v = (_values(c[ids], s[ids]).transpose(1, 2).flatten(2, 3) for c, s in ((st["k"], st["ks"]), (st["v"], st["vs"])))
    B, n, Hq, d = q.shape
    Hkv, T = k.shape[1], k.shape[2]
    G = Hq // Hkv
    qg = q.float().view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    s = qg @ k.transpose(2, 3)
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
    o = p.view(B, Hkv, G * n, T) @ v
    o = o.view(B, Hkv, G, n, d) / torch.where(total > 0, total, 1)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, d).to(q.dtype)


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
    op, d, Hkv, es = case["op"], case["d"], case["Hkv"], torch.finfo(_DTYPE[case["dtype"]]).bits // 8
    code_row = Hkv * (d // 2 + d // 16)  # a token's codes and scales, of K or of V
    if op in ("rope", "quant", "load"):
        N, live = case["N"], case["N"] - case["pad"]
        if op == "load":
            return {"bytes": 4 * N + 2 * live * code_row + 2 * N * Hkv * d * es, "flops": 2 * live * Hkv * d}
        Hq = case["Hq"]
        size = 2 * N * Hq * d * es + 2 * live * Hkv * d * es + (8 if case["rot"] else 4) * N
        flops = 3 * case["rot"] * (N * Hq + live * Hkv)
        if op == "rope":
            return {"bytes": size + 2 * live * Hkv * d * es, "flops": flops}
        rows = case["pool"] * case["bs"]
        size += 2 * live * code_row + 4 * rows + 2 * rows * (code_row + Hkv * d * es)
        return {"bytes": size, "flops": flops + 4 * live * Hkv * d + 2 * rows * Hkv * d}
    if op == "decode":
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
    blocks = sum(_ceil(e, case["bs"]) - f // case["bs"] for f, e in spans)
    size = sum(e - f for f, e in spans) * 2 * code_row + 4 * blocks
    size += 2 * rows * case["Hq"] * d * es + 4 * rows
    return {"bytes": size, "flops": 4 * d * case["Hq"] * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
_NIBBLE_OF_DIM = [0, 4, 1, 5, 2, 6, 3, 7]  # where dim j of eight stands in their 32-bit word


def _exact_values(codes, scales):
    """float64 [rows, d] of codes [rows, d / 2] and scales [rows, d / 32]."""
    words = codes.contiguous().view(torch.int32).long() & 0xffffffff
    u = torch.stack([words >> (4 * n) & 15 for n in _NIBBLE_OF_DIM], dim=-1).reshape(codes.shape[0], -1)
    return (u - 8).double() * scales.double().repeat_interleave(GROUP, dim=1)


def _exact_rotated(case, st, x):
    """One head's rows [N, d] in 64 bits: every pair as a complex number times e^(i angle)."""
    f, amplitude = _frequencies(case)
    r = case["rot"]
    angle = torch.outer(st["pos"].double(), f.to("cuda"))
    y = x.double().clone()
    first = slice(0, r, 2) if case["interleaved"] else slice(0, r // 2)
    second = slice(1, r, 2) if case["interleaved"] else slice(r // 2, r)
    z = torch.complex(y[:, first], y[:, second]) * torch.polar(torch.full_like(angle, amplitude), angle)
    y[:, first], y[:, second] = z.real, z.imag
    return y


def _exact_quantised(x):
    """What a row of 32-dim groups is stored as, in 64 bits."""
    groups = x.reshape(-1, GROUP)
    s = groups.abs().max(dim=1, keepdim=True).values / 7
    exponent = torch.floor(torch.log2(torch.where(s > 0, s, 1.0)))
    grid = torch.exp2((exponent - 7).clamp(min=-24))  # 8 significant bits, float16's smallest step at least
    s = torch.minimum(torch.round(s / grid) * grid, torch.tensor(TOP_SCALE, dtype=torch.float64, device=x.device))
    c = torch.round(groups / torch.where(s > 0, s, 1.0)).clamp(min=-7, max=7)
    return (c * s).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op, bs, Hkv, d = case["op"], case["bs"], case["Hkv"], case["d"]
    if op in ("rope", "quant", "load"):
        slots = st["slots"].long()
        live = torch.nonzero(slots >= 0)[:, 0]
        written = slots[live]
        results = []
        if op != "load" and case["Hq"]:
            q = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
            for h in range(case["Hq"]):
                q[:, h] = _exact_rotated(case, st, st["q"][:, h])
            results.append(q)
        for name, fresh in (("k", st.get("key")), ("v", st.get("value"))):
            cache = st[name]
            if op == "rope":
                rows = cache.double()
                flat = rows.view(-1, Hkv, d)
            elif op == "quant":
                flat = torch.empty((case["pool"] * bs, Hkv, d), dtype=torch.float64, device="cuda")
            else:
                flat = torch.zeros((case["N"], Hkv, d), dtype=torch.float64, device="cuda")
            for h in range(Hkv):
                if op != "rope":
                    stored = cache[:, h].reshape(-1, d // 2), st[name + "s"][:, h].reshape(-1, d // GROUP)
                if op == "load":
                    flat[live, h] = _exact_values(stored[0][written], stored[1][written])
                    continue
                x = fresh[:, h]
                x = _exact_rotated(case, st, x) if name == "k" and case["rot"] else x.double()
                if op == "quant":
                    flat[:, h] = _exact_values(*stored)
                    x = _exact_quantised(x)
                flat[written, h] = x[live]
            results.append(rows if op == "rope" else flat)
        return tuple(results)
    if op == "decode":
        ctx, first = _decode_lens(case)
        queries = [(c, c, [f], 0, slice(b, b + 1)) for b, (c, f) in enumerate(zip(ctx, first))]
    else:
        starts, ns, prefix, first = _prefill_lens(case)
        queries, at = [], 0
        for s, n, x in zip(starts, ns, prefix):
            queries.append((s + 1, s + n, first[at:at + n], x, slice(at, at + n)))
            at += n
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    G = case["Hq"] // Hkv
    for b, (seen0, T, lows, prefix_len, rows) in enumerate(queries):  # seen0: keys up to the first query's own
        blocks = st["tables"][b, :_ceil(T, bs)].long()
        low = torch.tensor(lows, device="cuda")[:, None]
        here = torch.arange(seen0 - 1, T, device="cuda")[:, None]
        key = torch.arange(T, device="cuda")[None]
        hidden = (key < low) | ((key > here) & (key >= prefix_len))
        for h in range(Hkv):
            kv = [_exact_values(st[n][blocks, h].reshape(-1, d // 2), st[n + "s"][blocks, h].reshape(-1, d // GROUP))[:T]
                  for n in ("k", "v")]
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
