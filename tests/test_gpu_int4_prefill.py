"""Prefill attention over the 4-bit cache with score rules, against the definition in binary64
over the values that the codes stand for (tests/score_reference.py derives the tolerance: K and
V are exact in float16, P is rounded to it)."""
import pytest
import torch

import int4_reference as ref
import score_reference as sr
from test_gpu_int4_decode import batch
from test_gpu_prefill_mod import RULES, SPANS, _rules

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def case(Hq, Hkv, bs, spans, dtype, seed):
    _, caches, tables = batch(Hq, Hkv, 128, bs, [s + n for s, n in spans], dtype, seed)
    ns = [n for _, n in spans]
    g = torch.Generator().manual_seed(seed + 1)
    q = (2 * torch.randn(sum(ns), Hq, 128, generator=g)).to(dtype).cuda()
    starts = torch.tensor([s for s, _ in spans], dtype=torch.int32).cuda()
    cu = torch.zeros(len(spans) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(ns), 0)
    return q, caches, tables, starts, cu.cuda(), ns


def check(pkv, q, caches, tables, starts, cu, ns, spans, rules, scale, max_q=None, tables_of_reference=None):
    err = torch.zeros(1, dtype=torch.int32, device=q.device)
    out = torch.full_like(q, float("nan"))
    pkv.pkv_paged_attention_prefill_int4(q, *caches, tables, starts, cu, scale, max_q or max(ns), out=out, err_flag=err, **rules)
    assert int(err) == 0
    k, v = (ref.token_major(caches[i], caches[2 + i]) for i in (0, 1))
    want = sr.prefill(q, k, v, tables, [s for s, _ in spans], ns, scale, rules.get("softcap", 0.0), rules.get("alibi_slopes"),
                      rules.get("key_starts"), rules.get("prefix_lens"))
    v_max = 8 * float(torch.nan_to_num(caches[3].float()).abs().max())
    tol = sr.tolerance(want, q.dtype, F16, v_max)
    e = (out.cpu().double() - want[0]).abs()
    assert torch.isfinite(out).all()
    assert bool((e <= tol).all()), f"worst error / tolerance {(e / tol).max().item():.3g}"
    return out


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype,Hq,Hkv,bs", [(BF16, 8, 8, 16), (F16, 16, 8, 256), (BF16, 32, 8, 48), (F16, 8, 1, 16), (BF16, 4, 1, 64)])
def test_rules(pkv, cuda_dev, dtype, Hq, Hkv, bs, rule):
    q, caches, tables, starts, cu, ns = case(Hq, Hkv, bs, SPANS, dtype, Hq + bs)
    check(pkv, q, caches, tables, starts, cu, ns, SPANS, _rules(rule, SPANS, Hq, cuda_dev), 128 ** -0.5)


@pytest.mark.parametrize("spans", [[(0, 1)], [(3000, 1), (2000, 5)], [(1000, 64)], [(0, 1500)]], ids=str)
def test_spans(pkv, cuda_dev, spans):
    """Single tokens, drafted tokens and chunks over long contexts (whose keys are split), long prompts."""
    q, caches, tables, starts, cu, ns = case(8, 2, 16, spans, BF16, 4)
    check(pkv, q, caches, tables, starts, cu, ns, spans, {}, 128 ** -0.5)
    check(pkv, q, caches, tables, starts, cu, ns, spans, {"softcap": 20.0}, 128 ** -0.5, max_q=max(ns) + 200)


LONG = [(0, 900), (37, 771), (512, 16), (5, 1), (3000, 900), (127, 130), (0, 800)]


@pytest.mark.parametrize("rule", ["plain", "cap-alibi", "window-cap", "blind", "prefix-alibi"])
@pytest.mark.parametrize("dtype,Hq,Hkv,bs", [(BF16, 8, 2, 16), (F16, 4, 2, 256), (BF16, 8, 1, 48)])
def test_widened_rules(pkv, cuda_dev, dtype, Hq, Hkv, bs, rule):
    """Calls of many rows, whose blocks are widened into the workspace first."""
    q, caches, tables, starts, cu, ns = case(Hq, Hkv, bs, LONG, dtype, Hq + bs)
    size = pkv.pkv_paged_attention_prefill_int4_workspace_size(len(LONG), Hq, Hkv, 128, bs, 900, tables.shape[1])
    assert size > 2 * len(LONG) * 3900 * Hkv * 128 * 2
    check(pkv, q, caches, tables, starts, cu, ns, LONG, _rules(rule, LONG, Hq, cuda_dev), 128 ** -0.5)


def test_widened_equals_fused(pkv, cuda_dev):
    """The same keys, the same products: a bound on the positions that changes the way changes no more than the order of sums."""
    spans = [(100, 800)]
    q, caches, tables, starts, cu, ns = case(8, 2, 16, spans, F16, 3)
    wide = torch.full((1, 70000), -1, dtype=torch.int32, device=cuda_dev)  # a table for a million tokens: fused
    wide[:, :tables.shape[1]] = tables
    size = pkv.pkv_paged_attention_prefill_int4_workspace_size
    # fused: the splits' workspace alone, as the 16-bit call's; widened: a pool of 57 blocks of K and of V too
    assert size(1, 8, 2, 128, 16, 800, 70000) == pkv.pkv_paged_attention_prefill_mod_workspace_size(1, 8, 2, 128, 16, 800, 70000)
    assert size(1, 8, 2, 128, 16, 800, 70000, 900) >= 2 * 57 * 16 * 2 * 128 * 2
    a = check(pkv, q, caches, wide, starts, cu, ns, spans, {}, 0.1)
    out = pkv.pkv_paged_attention_prefill_int4(q, *caches, wide, starts, cu, 0.1, 800, max_total_len=900)
    assert bool(((a.float() - out.float()).abs() <= 2.0 ** -9 * a.float().abs() + 2.0 ** -10).all())
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = pkv.pkv_paged_attention_prefill_int4(q, *caches, wide, starts, cu, 0.1, 800, max_total_len=880, err_flag=err)
    assert int(err) == pkv.ERRBIT_CONTEXT and not bool(out.any())


def test_widened_errors_and_two_graphs(pkv, cuda_dev):
    spans = [(0, 800), (16, 790), (0, 800)]
    q, caches, tables, starts, cu, ns = case(4, 2, 16, spans, BF16, 6)
    want = check(pkv, q, caches, tables, starts, cu, ns, spans, {}, 0.1)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    bad = starts.clone()
    bad[1] = -3
    out = pkv.pkv_paged_attention_prefill_int4(q, *caches, tables, bad, cu, 0.1, 800, err_flag=err)
    assert int(err) == pkv.ERRBIT_CONTEXT and not bool(out[800:1590].any())
    assert torch.equal(out[:800], want[:800]) and torch.equal(out[1590:], want[1590:])
    holes = tables.clone()
    holes[2, 0], holes[0, 3] = -1, 10 ** 8
    err.zero_()
    out = pkv.pkv_paged_attention_prefill_int4(q, *caches, holes, starts, cu, 0.1, 800, err_flag=err)
    assert int(err) == pkv.ERRBIT_BLOCK_RANGE and torch.isfinite(out).all() and not bool(out[1590:1606].any())
    assert torch.equal(out[:48], want[:48]) and torch.equal(out[800:1590], want[800:1590])
    # two graphs with a workspace each, replayed in turn
    graphs, outs = [], []
    for k in range(2):
        g, o = torch.cuda.CUDAGraph(), torch.empty_like(q)
        with torch.cuda.graph(g):
            pkv.pkv_paged_attention_prefill_int4(q, *caches, tables if k == 0 else holes, starts, cu, 0.1, 800, out=o)
        graphs.append(g)
        outs.append(o)
    for k in (0, 1, 0):
        graphs[k].replay()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], out)


def test_negative_scale_and_magnitudes(pkv, cuda_dev):
    spans = [(20, 70)]
    q, caches, tables, starts, cu, ns = case(8, 2, 16, spans, BF16, 5)
    check(pkv, q, caches, tables, starts, cu, ns, spans, {}, -(128 ** -0.5))
    for gain in (2.0 ** -30, 3e4):
        check(pkv, (q.float() * gain).to(BF16), caches, tables, starts, cu, ns, spans, {}, 128 ** -0.5 / gain)


def test_errors(pkv, cuda_dev):
    spans = [(0, 40), (16, 40), (0, 40)]
    q, caches, tables, starts, cu, ns = case(4, 2, 16, spans, F16, 6)
    want = check(pkv, q, caches, tables, starts, cu, ns, spans, {}, 0.1)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    bad = starts.clone()
    bad[1] = 10 ** 6
    out = pkv.pkv_paged_attention_prefill_int4(q, *caches, tables, bad, cu, 0.1, 40, err_flag=err)
    assert int(err) == pkv.ERRBIT_CONTEXT and not bool(out[40:80].any())
    assert torch.equal(out[:40], want[:40]) and torch.equal(out[80:], want[80:])
    holes = tables.clone()
    holes[2, 0] = -1  # keys 0 .. 15: rows that see nothing else are zero
    err.zero_()
    out = pkv.pkv_paged_attention_prefill_int4(q, *caches, holes, starts, cu, 0.1, 40, err_flag=err)
    assert int(err) == pkv.ERRBIT_BLOCK_RANGE
    assert torch.equal(out[:80], want[:80]) and not bool(out[80:96].any()) and torch.isfinite(out).all()


def test_a_step_of_the_serving_loop(pkv, cuda_dev):
    """Tables grown, keys rotated and written as 4-bit codes, prefill, then decode steps: each call's
    output is what the plain calls give over the cache read back in 16 bits."""
    Hq, Hkv, d, bs, nb = 16, 4, 128, 16, 300
    g = torch.Generator().manual_seed(11)
    lens = [70, 1, 333]
    B = len(lens)
    caches = ref.empty_cache(nb, Hkv, bs, d, 1, cuda_dev)
    tables = torch.full((B, 40), -1, dtype=torch.int32, device=cuda_dev)
    counts = torch.zeros(nb, dtype=torch.int32, device=cuda_dev)
    rope = pkv.pkv_rope_frequencies(d, scaling="yarn", factor=4.0, original_len=256)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    at = [0] * B
    for step in range(4):
        new = lens if step == 0 else [1] * B if step != 2 else [3, 1, 4]  # a prompt, tokens, drafts
        ends = [a + n for a, n in zip(at, new)]
        n = sum(new)
        cu, slots = pkv.pkv_grow_block_tables(tables, i32(at), i32(ends), counts, bs, num_new_tokens=n)
        qkv = torch.randn(n, Hq + 2 * Hkv, d, generator=g).to(BF16).cuda()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = i32([p for a, e in zip(at, ends) for p in range(a, e)])
        q = pkv.pkv_rope_store_kvcache_int4(q, k, v, pos, rope, *caches, slots)
        every = torch.arange(nb * bs, dtype=torch.int32, device=cuda_dev)
        wide = [x.view(nb, bs, Hkv, d) for x in pkv.pkv_load_kvcache_int4(*caches, every, F16)]
        if max(new) > 1:
            got = pkv.pkv_paged_attention_prefill_int4(q, *caches, tables, i32(at), cu, d ** -0.5, max(new))
            want = pkv.pkv_paged_attention_prefill_mod(q.half(), *wide, tables, i32(at), cu, d ** -0.5, max(new))
        else:
            got = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, i32(ends), d ** -0.5, max(ends))
            want = pkv.pkv_paged_attention_decode(q.half(), *wide, tables, i32(ends), d ** -0.5, max(ends))
        # both within score_reference's bounds of the definition, over values of magnitude below 8
        assert bool(((got.float() - want.float()).abs() <= 2.0 ** -8 * want.float().abs() + 0.02).all())
        at = ends
