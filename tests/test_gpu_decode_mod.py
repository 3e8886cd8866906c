"""Decode attention with score rules over every cache format, against the
definition in binary64 (tests/score_reference.py, which derives the tolerance)."""
import pytest
import torch

import pkv_workloads as wl
import score_reference as sr

pytestmark = pytest.mark.gpu

CTX = [1, 15, 16, 17, 64, 200, 333, 1000, 2047, 0, 700]


def _batch(dtype, Hq, Hkv, d, bs, ctx, seed, dev, q_gain=2.0):
    cfg = wl.DecodeConfig("t", dtype, Hq, Hkv, d, bs, len(ctx), 1, max(ctx), None)
    return wl.decode_batch(cfg, seed=seed, device=dev, ctx_override=ctx, nan_tails=True, nan_unused=True, q_gain=q_gain)


def _codes(pkv, fmt, batch, dev):
    nb, _, H, _ = batch.k_cache.shape
    g = torch.Generator().manual_seed(4)
    res = []
    for c in (batch.k_cache, batch.v_cache):
        gain = torch.exp(0.7 * torch.randn(nb, 1, H, 1, generator=g)).to(dev)
        res.append(getattr(pkv, "pkv_quantize_kvcache_" + fmt)((torch.nan_to_num(c.float()) * gain).to(c.dtype)))
    return res


def _rules(name, ctx, Hq, dev):
    slopes = torch.exp2(-8 * torch.arange(1, Hq + 1) / Hq).float().to(dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    window = i32([max(-3, c - 100) for c in ctx])
    far = i32([c - 1 if i % 2 else c + 5 for i, c in enumerate(ctx)])  # one key, or none
    odd = i32([(37 * i + 11) % max(c, 1) for i, c in enumerate(ctx)])
    return {"plain": {}, "cap": {"softcap": 6.0}, "alibi": {"alibi_slopes": slopes},
            "window": {"key_starts": window}, "all": {"softcap": 9.0, "alibi_slopes": slopes, "key_starts": odd},
            "blind": {"key_starts": far, "softcap": 20.0}}[name]


def _reference(q, kc, vc, tables, ctx, scale, rules):
    parts = []
    ks = rules.get("key_starts")
    for b, c in enumerate(ctx):
        lo = torch.tensor([0 if ks is None else int(ks[b])])
        slopes = rules.get("alibi_slopes")
        parts.append(sr.attention(q[b:b + 1].cpu(), sr.rows_of(kc, tables[b], c), sr.rows_of(vc, tables[b], c),
                                  torch.tensor([c - 1]), lo, torch.tensor([c]), scale, rules.get("softcap", 0.0),
                                  None if slopes is None else slopes.cpu()))
    return tuple(torch.cat(x) for x in zip(*parts))


def _check(pkv, batch, ctx, rules, caches=None, max_ctx=None):
    kc, ks, vc, vs = batch.k_cache, None, batch.v_cache, None
    if caches is not None:
        (kc, ks), (vc, vs) = caches
    err = torch.zeros(1, dtype=torch.int32, device=batch.q.device)
    out = torch.full_like(batch.q, float("nan"))
    pkv.pkv_paged_attention_decode_mod(batch.q, kc, vc, batch.block_tables, batch.context_lens, batch.scale,
                                       max_ctx or max(ctx), k_scale=ks, v_scale=vs, out=out, err_flag=err, **rules)
    ref = _reference(batch.q, sr.dequantize(kc, ks), sr.dequantize(vc, vs), batch.block_tables, ctx, batch.scale, rules)
    assert int(err.item()) == 0
    sr.assert_within(out, ref, vc, vs)
    return out


RULES = ["plain", "cap", "alibi", "window", "all", "blind"]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hkv,bs", [(8, 8, 16), (16, 8, 256), (32, 8, 48), (6, 2, 32), (8, 1, 16)])
def test_rules(pkv, cuda_dev, dtype, Hq, Hkv, bs, rule):
    _check(pkv, _batch(dtype, Hq, Hkv, 128, bs, CTX, Hq + bs, cuda_dev), CTX, _rules(rule, CTX, Hq, cuda_dev))


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("dtype,Hq,Hkv,bs", [(torch.bfloat16, 16, 8, 16), (torch.float16, 8, 2, 256), (torch.bfloat16, 7, 1, 48)])
def test_codes(pkv, cuda_dev, fmt, dtype, Hq, Hkv, bs, rule):
    batch = _batch(dtype, Hq, Hkv, 128, bs, CTX, Hq + bs, cuda_dev)
    _check(pkv, batch, CTX, _rules(rule, CTX, Hq, cuda_dev), _codes(pkv, fmt, batch, cuda_dev))


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype,Hq,Hkv,d,bs", [(torch.float32, 8, 2, 64, 4), (torch.bfloat16, 4, 4, 96, 7),
                                               (torch.float16, 32, 2, 128, 16), (torch.float32, 4, 1, 256, 16)])
def test_other_shapes(pkv, cuda_dev, dtype, Hq, Hkv, d, bs, rule):
    """fp32, other head sizes, block sizes and group sizes: the CUDA-core kernel."""
    _check(pkv, _batch(dtype, Hq, Hkv, d, bs, CTX, d + bs, cuda_dev), CTX, _rules(rule, CTX, Hq, cuda_dev))


@pytest.mark.parametrize("softcap", [1e-30, 0.01, 300.0, 1e30])
@pytest.mark.parametrize("dtype,d,bs", [(torch.bfloat16, 128, 16), (torch.float16, 128, 16), (torch.float32, 64, 4)])
def test_caps_of_any_size(pkv, cuda_dev, softcap, dtype, d, bs):
    ctx = [1, 100, 700]
    _check(pkv, _batch(dtype, 8, 8, d, bs, ctx, 12, cuda_dev), ctx, {"softcap": softcap})


@pytest.mark.parametrize("ctx", [[4096] * 8, [3000, 9, 8192, 1], [16384]])
@pytest.mark.parametrize("rule", ["plain", "cap", "window", "all"])
def test_long_contexts(pkv, cuda_dev, ctx, rule):
    """Equal lengths (the schedule guessed ahead), ragged ones, and one sequence over all SMs."""
    _check(pkv, _batch(torch.bfloat16, 16, 8, 128, 16, ctx, 3, cuda_dev), ctx, _rules(rule, ctx, 16, cuda_dev))


@pytest.mark.parametrize("fmt", [None, "int8"])
def test_more_than_512_sequences(pkv, cuda_dev, fmt):
    ctx = [(13 * i) % 90 for i in range(1100)]
    batch = _batch(torch.bfloat16, 4, 2, 128, 16, ctx, 5, cuda_dev)
    _check(pkv, batch, ctx, _rules("all", ctx, 4, cuda_dev), _codes(pkv, fmt, batch, cuda_dev) if fmt else None)


@pytest.mark.parametrize("fmt", [None, "fp8"])
def test_append(pkv, cuda_dev, fmt):
    """With key / value the caches end as after the store, and the row counts in the attention."""
    ctx = [5, 16, 17, 900, 333]
    batch = _batch(torch.bfloat16, 16, 8, 128, 16, ctx, 6, cuda_dev)
    rules = _rules("window", ctx, 16, cuda_dev)
    rules["softcap"] = 12.0
    kc, ks, vc, vs = batch.k_cache, None, batch.v_cache, None
    if fmt:
        (kc, ks), (vc, vs) = _codes(pkv, fmt, batch, cuda_dev)
    k2, v2 = kc.clone(), vc.clone()
    key, value = (torch.randn(len(ctx), 8, 128, device=cuda_dev).to(torch.bfloat16) for _ in range(2))
    out = pkv.pkv_paged_attention_decode_mod(batch.q, kc, vc, batch.block_tables, batch.context_lens, batch.scale, 900,
                                             key=key, value=value, k_scale=ks, v_scale=vs, **rules)
    slots = torch.tensor([int(batch.block_tables[b, (c - 1) // 16]) * 16 + (c - 1) % 16 for b, c in enumerate(ctx)],
                         dtype=torch.int32, device=cuda_dev)
    if fmt:
        pkv.pkv_store_kvcache_fp8(key, value, k2, v2, ks, vs, slots)
    else:
        pkv.pkv_store_kvcache(key, value, k2, v2, slots)
    as_bits = (lambda x: x) if fmt else (lambda x: x.view(torch.int16))
    assert torch.equal(as_bits(kc), as_bits(k2)) and torch.equal(as_bits(vc), as_bits(v2))
    ref = _reference(batch.q, sr.dequantize(kc, ks), sr.dequantize(vc, vs), batch.block_tables, ctx, batch.scale, rules)
    sr.assert_within(out, ref, vc, vs)


@pytest.mark.parametrize("fmt", [None, "fp8", "int8"])
def test_append_where_nothing_is_visible(pkv, cuda_dev, fmt):
    """A window that ends before the new token: the row is stored all the same, the output row is zero."""
    ctx = [5, 16, 17, 900, 1, 64]
    batch = _batch(torch.float16, 16, 8, 128, 16, ctx, 6, cuda_dev)
    first = torch.tensor([5, 100, 3, 900, 1, 64], dtype=torch.int32, device=cuda_dev)
    kc, ks, vc, vs = batch.k_cache, None, batch.v_cache, None
    if fmt:
        (kc, ks), (vc, vs) = _codes(pkv, fmt, batch, cuda_dev)
    k2, v2 = kc.clone(), vc.clone()
    key, value = (torch.randn(len(ctx), 8, 128, device=cuda_dev).half() for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = pkv.pkv_paged_attention_decode_mod(batch.q, kc, vc, batch.block_tables, batch.context_lens, batch.scale, 900,
                                             key=key, value=value, k_scale=ks, v_scale=vs, key_starts=first,
                                             err_flag=err)
    slots = torch.tensor([int(batch.block_tables[b, (c - 1) // 16]) * 16 + (c - 1) % 16 for b, c in enumerate(ctx)],
                         dtype=torch.int32, device=cuda_dev)
    if fmt:
        getattr(pkv, "pkv_store_kvcache_" + fmt)(key, value, k2, v2, ks, vs, slots)
    else:
        pkv.pkv_store_kvcache(key, value, k2, v2, slots)
    as_bits = (lambda x: x) if fmt else (lambda x: x.view(torch.int16))
    assert torch.equal(as_bits(kc), as_bits(k2)) and torch.equal(as_bits(vc), as_bits(v2))
    ref = _reference(batch.q, sr.dequantize(kc, ks), sr.dequantize(vc, vs), batch.block_tables, ctx, batch.scale,
                     {"key_starts": first})
    sr.assert_within(out, ref, vc, vs)
    assert int(err.item()) == 0 and torch.count_nonzero(out[[0, 1, 3, 4, 5]]) == 0


def test_plain_rule_gives_the_plain_call(pkv, cuda_dev):
    """Without a rule the kernel does the arithmetic of the plain call: the same bits."""
    batch = _batch(torch.bfloat16, 16, 8, 128, 16, CTX, 7, cuda_dev)
    args = (batch.q, batch.k_cache, batch.v_cache, batch.block_tables, batch.context_lens, batch.scale, max(CTX))
    assert torch.equal(pkv.pkv_paged_attention_decode_mod(*args), pkv.pkv_paged_attention_decode(*args))


@pytest.mark.parametrize("fmt", [None, "fp8"])
def test_nonfinite_in_front_of_the_window(pkv, cuda_dev, fmt):
    ctx = [300, 77, 2000]
    batch = _batch(torch.bfloat16, 16, 8, 128, 16, ctx, 8, cuda_dev)
    caches = _codes(pkv, fmt, batch, cuda_dev) if fmt else None
    first = [250, 70, 1001]
    for b, f in enumerate(first):
        for t in range(f):
            for c in [batch.k_cache, batch.v_cache] if caches is None else [x for x, _ in caches]:
                c[int(batch.block_tables[b, t // 16]), t % 16] = 0x7F if fmt else float("nan")
    ks = torch.tensor(first, dtype=torch.int32, device=cuda_dev)
    _check(pkv, batch, ctx, {"key_starts": ks, "softcap": 7.0}, caches)


def test_errors(pkv, cuda_dev):
    ctx = [100, 50, 30]
    batch = _batch(torch.bfloat16, 8, 8, 128, 16, ctx, 9, cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    lens = batch.context_lens.clone()
    lens[1] = 1000  # longer than declared
    ks = torch.tensor([3, 4, 29], dtype=torch.int32, device=cuda_dev)
    out = pkv.pkv_paged_attention_decode_mod(batch.q, batch.k_cache, batch.v_cache, batch.block_tables, lens,
                                             batch.scale, 100, key_starts=ks, err_flag=err)
    assert int(err.item()) == pkv.ERRBIT_CONTEXT and torch.count_nonzero(out[1]) == 0
    bt = batch.block_tables.clone()
    bt[0, 2] = -1  # positions 32 .. 47 are dropped
    err.zero_()
    out = pkv.pkv_paged_attention_decode_mod(batch.q, batch.k_cache, batch.v_cache, bt, batch.context_lens,
                                             batch.scale, 100, softcap=30.0, err_flag=err)
    assert int(err.item()) == pkv.ERRBIT_BLOCK_RANGE
    kc, vc = sr.dequantize(batch.k_cache, None), sr.dequantize(batch.v_cache, None)
    keep = [t for t in range(100) if not 32 <= t < 48]
    ref = sr.attention(batch.q[:1].cpu(), sr.rows_of(kc, batch.block_tables[0], 100)[keep],
                       sr.rows_of(vc, batch.block_tables[0], 100)[keep], torch.tensor([99]), torch.tensor([0]),
                       torch.tensor([84]), batch.scale, 30.0)
    sr.assert_within(out[:1], ref, batch.v_cache)


def test_captured(pkv, cuda_dev):
    ctx = [3000, 9, 512]
    batch = _batch(torch.bfloat16, 16, 8, 128, 16, ctx, 10, cuda_dev)
    args = (batch.q, batch.k_cache, batch.v_cache, batch.block_tables, batch.context_lens, batch.scale, max(ctx))
    rules = _rules("all", ctx, 16, cuda_dev)
    want = pkv.pkv_paged_attention_decode_mod(*args, **rules)
    torch.cuda.synchronize()
    ws = torch.empty(pkv.pkv_paged_attention_decode_workspace_size(3, 16, 8, 128, 16, max(ctx), torch.bfloat16),
                     dtype=torch.uint8, device=cuda_dev)
    out = torch.empty_like(batch.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.pkv_paged_attention_decode_mod(*args, **rules, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        # chunks of the tail go to whichever CTA asks first, but each piece is the same and is merged in order
        assert torch.equal(out, want)
