"""Prefill attention with score rules and over 8-bit caches, against the
definition in binary64 (tests/score_reference.py, which derives the tolerance)."""
import pytest
import torch

import pkv_workloads as wl
import score_reference as sr

pytestmark = pytest.mark.gpu

SPANS = [(0, 100), (37, 64), (512, 16), (5, 1), (0, 1), (300, 200), (127, 130), (128, 128), (0, 257)]


def _case(dtype, Hq, Hkv, bs, spans, seed, dev, q_gain=2.0):
    totals = [s + n for s, n in spans]
    cfg = wl.DecodeConfig("t", dtype, Hq, Hkv, 128, bs, len(spans), 1, max(totals), None)
    batch = wl.decode_batch(cfg, seed=seed, device=dev, ctx_override=totals, nan_tails=True, nan_unused=True)
    g = torch.Generator().manual_seed(seed + 1)
    ns = [n for _, n in spans]
    q = (torch.randn(sum(ns), Hq, 128, generator=g) * q_gain).to(dtype).to(dev)
    starts = torch.tensor([s for s, _ in spans], dtype=torch.int32, device=dev)
    cu = torch.zeros(len(spans) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(ns), 0)
    return batch, q, starts, cu.to(dev), ns


def _codes(pkv, fmt, batch, gain_seed, dev):
    """8-bit copies of the batch's caches whose blocks differ in magnitude."""
    nb, _, H, _ = batch.k_cache.shape
    g = torch.Generator().manual_seed(gain_seed)
    res = []
    for c in (batch.k_cache, batch.v_cache):
        gain = torch.exp(0.7 * torch.randn(nb, 1, H, 1, generator=g)).to(dev)
        quant = getattr(pkv, "pkv_quantize_kvcache_" + fmt)
        res.append(quant((torch.nan_to_num(c.float()) * gain).to(c.dtype)))
    return res


def _slopes(Hq, dev):
    return torch.exp2(-8 * torch.arange(1, Hq + 1) / Hq).float().to(dev)


def _rules(name, spans, Hq, dev, seed=9):
    g = torch.Generator().manual_seed(seed)
    docs = []
    for s, n in spans:
        at, nxt = 0, 0
        for p in range(s + n):
            if p == nxt:
                at, nxt = p, p + int(torch.randint(1, 150, (1,), generator=g))
            if p >= s:
                docs.append(at)
    window = [max(-5, p - 69) for s, n in spans for p in range(s, s + n)]
    blind = [d if i % 7 else 10 ** 6 for i, d in enumerate(docs)]  # every seventh row sees nothing
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    prefix = [int(torch.randint(0, s + n + 40, (1,), generator=g)) for s, n in spans]
    return {"plain": {}, "cap": {"softcap": 8.0}, "alibi": {"alibi_slopes": _slopes(Hq, dev)},
            "cap-alibi": {"softcap": 5.0, "alibi_slopes": _slopes(Hq, dev)}, "documents": {"key_starts": i32(docs)},
            "window-cap": {"key_starts": i32(window), "softcap": 20.0}, "prefix": {"prefix_lens": i32(prefix)},
            "prefix-alibi": {"prefix_lens": i32(prefix), "alibi_slopes": _slopes(Hq, dev)},
            "blind": {"key_starts": i32(blind), "prefix_lens": i32(prefix), "softcap": 10.0}}[name]


RULES = ["plain", "cap", "alibi", "cap-alibi", "documents", "window-cap", "prefix", "prefix-alibi", "blind"]


def _check(pkv, batch, q, starts, cu, ns, spans, rules, scale, caches=None, max_q=None, err_bits=0):
    err = torch.zeros(1, dtype=torch.int32, device=q.device)
    if caches is None:
        kc, ks, vc, vs = batch.k_cache, None, batch.v_cache, None
    else:
        (kc, ks), (vc, vs) = caches
    out = torch.full_like(q, float("nan"))
    pkv.pkv_paged_attention_prefill_mod(q, kc, vc, batch.block_tables, starts, cu, scale, max_q or max(ns), k_scale=ks,
                                        v_scale=vs, out=out, err_flag=err, **rules)
    ref = sr.prefill(q, sr.dequantize(kc, ks), sr.dequantize(vc, vs), batch.block_tables,
                          [s for s, _ in spans], ns, scale, rules.get("softcap", 0.0), rules.get("alibi_slopes"),
                          rules.get("key_starts"), rules.get("prefix_lens"))
    assert int(err.item()) == err_bits
    sr.assert_within(out, ref, vc, vs)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hkv,bs", [(8, 8, 16), (16, 8, 256), (32, 8, 48), (64, 8, 16), (4, 1, 64)])
def test_rules(pkv, cuda_dev, dtype, Hq, Hkv, bs, rule):
    batch, q, starts, cu, ns = _case(dtype, Hq, Hkv, bs, SPANS, Hq + bs, cuda_dev)
    _check(pkv, batch, q, starts, cu, ns, SPANS, _rules(rule, SPANS, Hq, cuda_dev), batch.scale)


@pytest.mark.parametrize("rule", ["plain", "cap", "cap-alibi", "blind", "prefix-alibi"])
@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("dtype,Hq,Hkv,bs", [(torch.bfloat16, 8, 8, 16), (torch.float16, 16, 8, 256),
                                             (torch.bfloat16, 32, 8, 48), (torch.float16, 8, 1, 16)])
def test_codes(pkv, cuda_dev, fmt, dtype, Hq, Hkv, bs, rule):
    batch, q, starts, cu, ns = _case(dtype, Hq, Hkv, bs, SPANS, Hq + bs, cuda_dev)
    _check(pkv, batch, q, starts, cu, ns, SPANS, _rules(rule, SPANS, Hq, cuda_dev), batch.scale,
           _codes(pkv, fmt, batch, 3, cuda_dev))


@pytest.mark.parametrize("scale", [-0.06, 0.0, 1e-35])
@pytest.mark.parametrize("fmt", [None, "int8"])
@pytest.mark.parametrize("rule", ["plain", "cap", "prefix"])
def test_other_scales(pkv, cuda_dev, scale, fmt, rule):
    spans = [(0, 100), (300, 70), (17, 1)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 16, 8, 16, spans, 74, cuda_dev)
    _check(pkv, batch, q, starts, cu, ns, spans, _rules(rule, spans, 16, cuda_dev), scale,
           _codes(pkv, fmt, batch, 3, cuda_dev) if fmt else None)


@pytest.mark.parametrize("rule", ["plain", "cap", "alibi", "window-cap", "prefix"])
@pytest.mark.parametrize("fmt", [None, "fp8"])
@pytest.mark.parametrize("spans", [[(2000, 1)], [(1500, 40), (3, 2)], [(4000, 33)], [(0, 700)]])
def test_split_keys(pkv, cuda_dev, rule, fmt, spans):
    """Few rows over long contexts: the key blocks are cut over several CTAs and joined."""
    Hq, Hkv, bs = 8, 2, 16
    batch, q, starts, cu, ns = _case(torch.bfloat16, Hq, Hkv, bs, spans, 5, cuda_dev)
    assert pkv.pkv_paged_attention_prefill_mod_workspace_size(len(spans), Hq, Hkv, 128, bs, max(ns),
                                                              batch.block_tables.shape[1]) > 0
    _check(pkv, batch, q, starts, cu, ns, spans, _rules(rule, spans, Hq, cuda_dev), batch.scale,
           _codes(pkv, fmt, batch, 8, cuda_dev) if fmt else None)
    # a generous bound on the new tokens gives other splits of the same rows
    _check(pkv, batch, q, starts, cu, ns, spans, _rules(rule, spans, Hq, cuda_dev), batch.scale,
           _codes(pkv, fmt, batch, 8, cuda_dev) if fmt else None, max_q=max(ns) + 300)


@pytest.mark.parametrize("softcap", [1e-30, 0.01, 3.0, 50.5, 51.0, 300.0, 1e30])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("q_gain", [0.1, 30.0])
def test_caps_of_any_size(pkv, cuda_dev, softcap, dtype, q_gain):
    """Scores far below and far above the cap (up to where tanh is 1), caps on both sides of the
    bound up to which P needs no reference maximum, whole rows of scores at minus the cap."""
    spans = [(0, 150), (700, 20)]
    batch, q, starts, cu, ns = _case(dtype, 8, 8, 16, spans, 11, cuda_dev, q_gain)
    q[::7] = -q_gain * batch.k_cache[batch.block_tables[0, 0].item(), 0].to(dtype)  # against key 0
    _check(pkv, batch, q, starts, cu, ns, spans, {"softcap": softcap}, batch.scale)


@pytest.mark.parametrize("fmt", [None, "fp8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_small_scores_beside_large_ones(pkv, cuda_dev, dtype, fmt):
    """Rows whose scores pass a large cap do not cost the rows beside them their precision."""
    spans = [(200, 120)]
    batch, q, starts, cu, ns = _case(dtype, 8, 8, 16, spans, 31, cuda_dev)
    q[::2] *= 3e3  # scores of 6000 in standard deviation
    rules = {"softcap": 2e4}
    caches = _codes(pkv, fmt, batch, 3, cuda_dev) if fmt else None
    (kc, ks), (vc, vs) = caches or ((batch.k_cache, None), (batch.v_cache, None))
    out = pkv.pkv_paged_attention_prefill_mod(q, kc, vc, batch.block_tables, starts, cu, batch.scale, 120, k_scale=ks,
                                              v_scale=vs, **rules)
    ref = sr.prefill(q, sr.dequantize(kc, ks), sr.dequantize(vc, vs), batch.block_tables, [200], ns, batch.scale, 2e4)
    assert torch.isfinite(out).all()
    sr.assert_within(out[1::2], tuple(x[1::2] for x in ref), vc, vs)


def test_plain_rule_equals_the_plain_call(pkv, cuda_dev):
    """Both kernels round P the same way; their reference maxima move alike, so only the summing order differs."""
    batch, q, starts, cu, ns = _case(torch.bfloat16, 16, 8, 16, SPANS, 6, cuda_dev)
    a = pkv.pkv_paged_attention_prefill_mod(q, batch.k_cache, batch.v_cache, batch.block_tables, starts, cu,
                                            batch.scale, max(ns))
    b = pkv.pkv_paged_attention_prefill(q, batch.k_cache, batch.v_cache, batch.block_tables, starts, cu, batch.scale,
                                        max(ns))
    ref = sr.prefill(q, sr.dequantize(batch.k_cache, None), sr.dequantize(batch.v_cache, None),
                          batch.block_tables, [s for s, _ in SPANS], ns, batch.scale)
    for x in (a, b):
        sr.assert_within(x, ref, batch.v_cache)


@pytest.mark.parametrize("fmt", [None, "fp8"])
def test_nonfinite_in_masked_places(pkv, cuda_dev, fmt):
    """NaN and infinities in K of masked keys and in V rows that nobody in the tile sees leave no trace."""
    spans = [(0, 200), (250, 30)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 16, 8, 16, spans, 8, cuda_dev)
    # keys below 130 / 256 are seen by no row
    ks = torch.tensor([130] * 200 + [256] * 30, dtype=torch.int32, device=cuda_dev)
    caches = _codes(pkv, fmt, batch, 3, cuda_dev) if fmt else None
    target = [batch.k_cache, batch.v_cache] if caches is None else [c for c, _ in caches]
    for b, upto in ((0, 130), (1, 256)):
        for t in range(upto):
            blk, row = int(batch.block_tables[b, t // 16]), t % 16
            for c in target:
                c[blk, row] = 0x7F if fmt else (float("nan") if t % 2 else float("inf"))
    _check(pkv, batch, q, starts, cu, ns, spans, {"key_starts": ks}, batch.scale, caches)


@pytest.mark.parametrize("fmt", [None, "int8"])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_tiles_that_see_nothing(pkv, cuda_dev, fmt, softcap):
    """No row of whole query tiles sees a key: zero rows, nothing read for them, no error."""
    spans = [(0, 400), (600, 70), (30, 20)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 16, 8, 16, spans, 21, cuda_dev)
    ks = torch.tensor([2 ** 31 - 1] * 300 + [310] * 100 + [2 ** 31 - 1] * 70 + [50] * 20, dtype=torch.int32, device=cuda_dev)
    _check(pkv, batch, q, starts, cu, ns, spans, {"key_starts": ks, "softcap": softcap}, batch.scale,
           _codes(pkv, fmt, batch, 3, cuda_dev) if fmt else None)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("gain", [1e-30, 1.0, 1e15])
def test_extreme_scales(pkv, cuda_dev, fmt, gain):
    """V scales of any magnitude, blocks of zeros (scale 0), and blocks 2^40 apart."""
    spans = [(100, 60)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 8, 8, 16, spans, 8, cuda_dev)
    caches = _codes(pkv, fmt, batch, 3, cuda_dev)
    (kc, ks), (vc, vs) = caches
    vs *= gain
    used = batch.block_tables[0].tolist()
    vs[used[1]] *= 2.0 ** 40
    vs[used[2]] *= 2.0 ** -40
    for c, s in caches:  # a block of zeros in each cache
        c[used[4]] = 0
        s[used[4]] = 0
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = pkv.pkv_paged_attention_prefill_mod(q, kc, vc, batch.block_tables, starts, cu, batch.scale, 60, k_scale=ks,
                                              v_scale=vs, err_flag=err)
    ref = sr.prefill(q, sr.dequantize(kc, ks), sr.dequantize(vc, vs), batch.block_tables, [100], ns, batch.scale)
    sr.assert_within(out, ref, vc, vs)


@pytest.mark.parametrize("gain", [1e-36, 3e-5, 1e6, 1e30])
def test_bf16_queries_of_any_magnitude_over_codes(pkv, cuda_dev, gain):
    """bf16 queries outside f16's range: scaled exactly by a power of two per row."""
    spans = [(50, 70)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 8, 8, 16, spans, 8, cuda_dev)
    q = (q.float() * gain).to(torch.bfloat16)
    _check(pkv, batch, q, starts, cu, ns, spans, {}, batch.scale / gain, _codes(pkv, "fp8", batch, 3, cuda_dev))


def test_errors(pkv, cuda_dev):
    spans = [(100, 50), (0, 40)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 16, 8, 16, spans, 72, cuda_dev)
    args = (q, batch.k_cache, batch.v_cache)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    bt = batch.block_tables.clone()
    bt[0, 2] = 10_000  # positions 32 .. 47 of sequence 0 are dropped
    out = pkv.pkv_paged_attention_prefill_mod(*args, bt, starts, cu, batch.scale, 50, softcap=20.0, err_flag=err)
    assert int(err.item()) == pkv.ERRBIT_BLOCK_RANGE
    kc, vc = sr.dequantize(batch.k_cache, None), sr.dequantize(batch.v_cache, None)
    k0, v0 = sr.rows_of(kc, batch.block_tables[0], 150), sr.rows_of(vc, batch.block_tables[0], 150)
    keep = [t for t in range(150) if not 32 <= t < 48]
    pos = torch.arange(100, 150)
    ref = sr.attention(q[:50].cpu(), k0[keep], v0[keep], pos, torch.zeros(50), pos + 1 - 16, batch.scale, 20.0)
    sr.assert_within(out[:50], ref, batch.v_cache)
    bad = starts.clone()
    bad[1] = -3  # zero rows
    err.zero_()
    out = pkv.pkv_paged_attention_prefill_mod(*args, batch.block_tables, bad, cu, batch.scale, 50, err_flag=err)
    assert int(err.item()) == pkv.ERRBIT_CONTEXT and torch.count_nonzero(out[50:]) == 0
    err.zero_()
    out = torch.full_like(q, 7.0)  # more new tokens than declared: that sequence's rows stay
    pkv.pkv_paged_attention_prefill_mod(*args, batch.block_tables, starts, cu, batch.scale, 45, out=out, err_flag=err)
    assert int(err.item()) == pkv.ERRBIT_CONTEXT
    assert bool((out[:50] == 7).all()) and not bool((out[50:] == 7).all())


def test_rows_behind_the_last_sequence_stay(pkv, cuda_dev):
    spans = [(0, 30), (20, 20)]
    batch, q, starts, cu, ns = _case(torch.float16, 8, 8, 16, spans, 3, cuda_dev)
    padded = torch.cat([q, torch.zeros(9, 8, 128, dtype=q.dtype, device=cuda_dev)])
    out = torch.full_like(padded, 5.0)
    pkv.pkv_paged_attention_prefill_mod(padded, batch.k_cache, batch.v_cache, batch.block_tables, starts, cu,
                                        batch.scale, 30, out=out)
    assert bool((out[50:] == 5).all())


def test_captured_and_on_another_stream(pkv, cuda_dev):
    """A graph replay, and a call on a side stream with its own workspace, give the eager call's bits."""
    spans = [(1500, 40)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 8, 2, 16, spans, 5, cuda_dev)
    args = (q, batch.k_cache, batch.v_cache, batch.block_tables, starts, cu, batch.scale, 40)
    rules = {"softcap": 15.0, "alibi_slopes": _slopes(8, cuda_dev)}
    want = pkv.pkv_paged_attention_prefill_mod(*args, **rules)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = pkv.pkv_paged_attention_prefill_mod(*args, **rules)
    side.synchronize()
    assert torch.equal(got, want)
    n = pkv.pkv_paged_attention_prefill_mod_workspace_size(1, 8, 2, 128, 16, 40, batch.block_tables.shape[1])
    ws = torch.empty(n, dtype=torch.uint8, device=cuda_dev)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.pkv_paged_attention_prefill_mod(*args, **rules, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
