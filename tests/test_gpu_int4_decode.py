"""Decode attention over the 4-bit cache, against the definition in binary64 over the values
that the codes stand for.

Tolerance: score_reference.py's, with P in float16, and a larger score error.  K's codes enter
their products as u and 16 u (under q / 16) in units of 2^-24, their offset taken back by the start
of the f32 accumulator.  A group of 32 dims is two instructions; each may cut its sum to 2^-22
of its largest term or partial sum, at most (15 + 8) sum |q| over the group: together 2 x 23 x
2^-22 < 2^-16 sum |q|, in code steps.  With scales up to s the score is off by at most
scale s 2^-16 sum |q| more.
P is rounded to float16 twice, by itself and times V's scale, and not in the row sum: the same
two half steps.  Below float16's normal range p s is off by 2^-25 and its codes are up to 7: that
term is 2^-25 keys max(8, |V|), with p at least 1 for the key that set the reference (it is 2^11
there where V's scales are below 1, and less by their binades else: the term shrinks with it).
"""
import pytest
import torch

import int4_reference as ref
import score_reference as sr

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
CTX = [1, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 100, 255, 256, 300, 511, 700, 1025]


def batch(Hq, Hkv, d, bs, ctx, dtype, seed, spare=2, hole=None):
    """(q, caches, tables): a permuted pool whose unused rows hold NaN scales."""
    g = torch.Generator().manual_seed(seed)
    used = [sr.cdiv(c, bs) for c in ctx]
    nb = sum(used) + spare
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    x = torch.randn(2, nb, Hkv, bs, d, generator=g).double() * torch.exp(0.5 * torch.randn(Hkv, 1, d, generator=g)).double()
    s = ref.scales(x)
    codes = ref.pack(ref.codes(x, s))
    width = max(max(used), 1) + 1
    tables = torch.full((len(ctx), width), -1, dtype=torch.int32)
    seen = torch.zeros(nb, bs, dtype=torch.bool)
    at = 0
    for b, (u, c) in enumerate(zip(used, ctx)):
        tables[b, :u] = perm[at:at + u]
        for j in range(u):
            seen[perm[at + j], :min(bs, c - j * bs)] = True
        at += u
    s = torch.where(seen[None, :, None, :, None], s, float("nan"))
    q = torch.randn(len(ctx), Hq, d, generator=g).to(dtype).cuda()
    return q, (codes[0].cuda(), codes[1].cuda(), s[0].contiguous().cuda(), s[1].contiguous().cuda()), tables.cuda()


def check(got, q, caches, want, scale):
    s_max = float(torch.nan_to_num(caches[2].float()).abs().max())
    score = sr.SCORE + scale * s_max * 2.0 ** -16 * q.double().abs().sum(-1).max().item()
    out, mag, keys = want
    v_max = 8 * max(1.0, float(torch.nan_to_num(caches[3].float()).abs().max()))
    tol = sr.tolerance(want, got.dtype, F16, v_max) + 2 * (score - sr.SCORE) * mag
    err = (got.cpu().double() - out).abs()
    assert torch.isfinite(got).all()
    assert bool((err <= tol).all()), f"worst error / tolerance {(err / tol).max().item():.3g}, max abs {err.max().item():.3g}"


def reference(q, caches, tables, ctx, scale, softcap=0.0, slopes=None, key_starts=None):
    k, v = ref.token_major(caches[0], caches[2]), ref.token_major(caches[1], caches[3])
    some = [b for b, c in enumerate(ctx) if c > 0]
    starts = None if key_starts is None else key_starts[some]
    parts = sr.prefill(q[some], k, v, tables[some], [ctx[b] - 1 for b in some], [1] * len(some), scale, softcap, slopes, starts)
    whole = [torch.zeros(len(ctx), *p.shape[1:], dtype=torch.float64) for p in parts]
    for w, p in zip(whole, parts):
        w[some] = p
    return tuple(whole)


def rules(name, ctx, Hq):
    first = torch.tensor([max(-3, c - 70) if i % 5 else c + 3 for i, c in enumerate(ctx)], dtype=torch.int32).cuda()
    slopes = torch.exp2(-8 * torch.arange(1, Hq + 1) / Hq).float().cuda()
    return {"plain": {}, "cap": {"softcap": 3.0}, "alibi": {"alibi_slopes": slopes}, "window": {"key_starts": first},
            "all": {"softcap": 30.0, "alibi_slopes": slopes, "key_starts": first}}[name]


@pytest.mark.parametrize("rule", ["plain", "cap", "alibi", "window", "all"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,d,bs", [(8, 8, 128, 16), (16, 8, 128, 256), (32, 8, 128, 48), (64, 8, 128, 16), (4, 1, 128, 64),
                                         (6, 2, 64, 16), (8, 2, 256, 32), (12, 1, 128, 16), (40, 2, 64, 32), (9, 1, 256, 16)])
def test_decode(pkv, cuda_dev, Hq, Hkv, d, bs, dtype, rule):
    q, caches, tables = batch(Hq, Hkv, d, bs, CTX, dtype, Hq + d + bs)
    kw = rules(rule, CTX, Hq)
    scale = d ** -0.5
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = torch.full_like(q, float("nan"))
    ctx = torch.tensor(CTX, dtype=torch.int32, device=cuda_dev)
    pkv.pkv_paged_attention_decode_int4(q, *caches, tables, ctx, scale, max(CTX), out=out, err_flag=err, **kw)
    assert int(err) == 0
    check(out, q, caches, reference(q, caches, tables, CTX, scale, kw.get("softcap", 0.0), kw.get("alibi_slopes"),
                                    kw.get("key_starts")), scale)


def cdiv16(n):
    return sr.cdiv(n, 16)


SHORT = [1, 16, 33, 0, 64, 65, 300, 511, 700, 1000]


@pytest.mark.parametrize("rule", ["plain", "all", "window"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,Hkv,d,bs", [(8, 8, 128, 16), (32, 8, 128, 48), (12, 1, 128, 256), (6, 2, 64, 16), (9, 1, 256, 16)])
def test_few_short_contexts(pkv, cuda_dev, Hq, Hkv, d, bs, dtype, rule):
    """A CTA per unit: no workspace, the warps' parts joined in shared memory."""
    assert pkv.pkv_paged_attention_decode_int4_workspace_size(len(SHORT), Hq, Hkv, d, max(SHORT)) == 0
    q, caches, tables = batch(Hq, Hkv, d, bs, SHORT, dtype, Hq + d + bs)
    kw = rules(rule, SHORT, Hq)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = torch.full_like(q, float("nan"))
    ctx = torch.tensor(SHORT, dtype=torch.int32, device=cuda_dev)
    pkv.pkv_paged_attention_decode_int4(q, *caches, tables, ctx, d ** -0.5, max(SHORT), out=out, err_flag=err, **kw)
    assert int(err) == 0
    want = reference(q, caches, tables, SHORT, d ** -0.5, kw.get("softcap", 0.0), kw.get("alibi_slopes"), kw.get("key_starts"))
    check(out, q, caches, want, d ** -0.5)
    # the same batch under a bound that makes it slices and a join: two orders of the same sums
    long = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, ctx, d ** -0.5, 1025, **kw)
    check(long, q, caches, want, d ** -0.5)


@pytest.mark.parametrize("bound", [1025, 1 << 16])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 4, 64), (8, 1, 256)])
def test_small_values(pkv, cuda_dev, Hq, Hkv, d, bound):
    """Scales of V that are 2^11 times smaller (still normal in float16) are as exact, relative to them:
    P makes use of float16's whole range, so p s leaves the normal range 2^11 later than the tolerance has it."""
    ctx = [900, 1025, 77]
    q, caches, tables = batch(Hq, Hkv, d, 16, ctx, BF16, 21 + d)
    caches = (*caches[:3], caches[3].clamp(min=0.25))
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    small = (*caches[:3], caches[3] / 2048)
    out = pkv.pkv_paged_attention_decode_int4(q, *small, tables, lens, 0.3 * d ** -0.5, bound)
    check(out * 2048, q, caches, reference(q, caches, tables, ctx, 0.3 * d ** -0.5), 0.3 * d ** -0.5)


@pytest.mark.parametrize("bound", [900, 40000])
def test_many_small_weights_of_small_values(pkv, cuda_dev, bound):
    """One key far above the others, which together weigh more: p s of each is 2^-25 where p is 1 for that key.

    The outputs are rounded by 2^-9 of them; p and p s by 2^-11 each of a magnitude that is below 2 times the
    output; the one key's score is off by at most 2^-16 0.13 64, which moves the output by less than half of that.
    Together 2^-9 + 2^-9 + 2^-13.9 < 2^-7.9."""
    n, d = bound, 64
    top = 12.0 if n > 5000 else 7.0  # binades
    kc = torch.zeros(cdiv16(n), 1, 16, d)
    kc[0, 0, 5] = 1
    vc = torch.full_like(kc, 7)
    vc[0, 0, 5] = -7
    ks = torch.full((cdiv16(n), 1, 16, d // 32), top * 0.6931 / 64).to(F16)
    vs = torch.full_like(ks, 2.0 ** (-13 if n > 5000 else -18))
    caches = tuple(x.cuda() for x in (ref.pack(kc), ref.pack(vc), ks, vs))
    q = torch.ones(1, 1, d, dtype=BF16).cuda()
    tables = torch.arange(cdiv16(n), dtype=torch.int32).cuda()[None]
    out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, torch.tensor([n], dtype=torch.int32).cuda(), 1.0, bound)
    want = reference(q, caches, tables, [n], 1.0)[0]
    assert bool(((out.cpu().double() - want).abs() <= 2.0 ** -7.9 * want.abs()).all()), (out[0, 0, 0], want[0, 0, 0])


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 4, 64), (8, 1, 256)])
def test_scales_that_change_along_the_context(pkv, cuda_dev, Hq, Hkv, d, order):
    """V's scales from 2^-8 to 2^8 and back down, so that the room of P moves within a unit."""
    ctx = [1025, 600, 3000]
    q, caches, tables = batch(Hq, Hkv, d, 16, ctx, BF16, 31 + d)
    vs = caches[3].clone()
    for b, c in enumerate(ctx):
        for j in range(sr.cdiv(c, 16)):
            e = round(8 * order * torch.tensor(j / 11.0).sin().item())
            vs[tables[b, j].item()] = (vs[tables[b, j].item()].clamp(0.25, 4) * 2.0 ** e).to(F16)
    caches = (*caches[:3], vs)
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    for bound in (3000, 1 << 20):
        out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, d ** -0.5, bound)
        check(out, q, caches, reference(q, caches, tables, ctx, d ** -0.5), d ** -0.5)


def test_two_streams_at_once(pkv, cuda_dev):
    """Calls that overlap, each with the workspace of its own stream."""
    ctx = [3000] * 8
    q, caches, tables = batch(32, 8, 128, 16, ctx, BF16, 12)
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    want = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, 0.09, 3000)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, 0.09, 3000, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_nan_stays_in_its_sequence_and_head(pkv, cuda_dev):
    ctx = [300, 70, 1500]
    q, caches, tables = batch(8, 2, 128, 16, ctx, F16, 13)
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    for bound in (1500, 1 << 20):
        want = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, 0.09, bound)
        hurt = q.clone()
        hurt[1, 3, 5], hurt[2, 0, 0] = float("nan"), float("inf")
        got = pkv.pkv_paged_attention_decode_int4(hurt, *caches, tables, lens, 0.09, bound)
        assert bool(torch.isnan(got[1, 3]).all())
        rest = torch.ones(3, 8, dtype=torch.bool, device=cuda_dev)
        rest[1, 3] = rest[2, 0] = False
        assert bool(torch.isnan(pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, float("nan"), bound)).all())
        assert torch.isfinite(got[rest]).all() and bool(((got - want)[rest].abs() <= 2.0 ** -9 * (want[rest].abs() + 1)).all())


@pytest.mark.parametrize("ctx", [[1], [40000], [3] * 600, [17000, 1, 0, 9]], ids=["one", "long", "many", "mixed"])
def test_lengths(pkv, cuda_dev, ctx):
    q, caches, tables = batch(8, 2, 128, 16, ctx, BF16, 5)
    out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, torch.tensor(ctx, dtype=torch.int32).cuda(), 128 ** -0.5, max(ctx))
    check(out, q, caches, reference(q, caches, tables, ctx, 128 ** -0.5), 128 ** -0.5)


@pytest.mark.parametrize("rule", ["window", "all"])
def test_groups_of_sequences_with_rules(pkv, cuda_dev, rule):
    ctx = [(7 * i) % 90 for i in range(1100)]  # three launches over one workspace
    q, caches, tables = batch(4, 2, 64, 16, ctx, F16, 8)
    kw = rules(rule, ctx, 4)
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, 0.125, max(ctx), **kw)
    check(out, q, caches, reference(q, caches, tables, ctx, 0.125, kw.get("softcap", 0.0), kw.get("alibi_slopes"),
                                    kw.get("key_starts")), 0.125)


def test_errors_and_holes(pkv, cuda_dev):
    """Bad lengths give zero rows, missing blocks count as masked; both set their bits."""
    ctx = [100, 100, 100, 64]
    q, caches, tables = batch(4, 2, 128, 16, ctx, F16, 6)
    want = reference(q, caches, tables, ctx, 0.1)
    given = torch.tensor([100, -4, 300, 64], dtype=torch.int32).cuda()
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, given, 0.1, 128, err_flag=err)
    assert int(err) == pkv.ERRBIT_CONTEXT and not bool(out[1:3].any())
    check(out[[0, 3]], q[[0, 3]], caches, tuple(w[[0, 3]] for w in want), 0.1)
    # blocks 0 and 2 of sequence 0 missing: the rest alone, blocks in front of the window never looked at
    holes = tables.clone()
    holes[0, 0], holes[0, 2] = -1, 10 ** 6
    given = torch.tensor(ctx, dtype=torch.int32).cuda()
    err.zero_()
    out = pkv.pkv_paged_attention_decode_int4(q, *caches, holes, given, 0.1, 128, err_flag=err)
    assert int(err) == pkv.ERRBIT_BLOCK_RANGE
    k, v = (ref.token_major(caches[i], caches[2 + i]) for i in (0, 1))
    rows = [torch.cat([x[tables[0, j].item()] for j in (1, 3, 4, 5, 6)])[:68] for x in (k, v)]
    pos = torch.tensor([67])
    alone = sr.attention(q[:1].cpu(), rows[0], rows[1], pos, torch.tensor([0]), torch.tensor([68]), 0.1)
    check(out[:1], q[:1], caches, alone, 0.1)
    err.zero_()
    first = torch.tensor([48, 0, 0, 0], dtype=torch.int32).cuda()
    pkv.pkv_paged_attention_decode_int4(q, *caches, holes, given, 0.1, 128, key_starts=first, err_flag=err)
    assert int(err) == 0


@pytest.mark.parametrize("gain", [2.0 ** -100, 2.0 ** -30, 1e-3, 1.0, 3e4, 2.0 ** 90, 2.0 ** 110])
def test_magnitudes(pkv, cuda_dev, gain):
    """Queries far from unit size: the scores, not the queries, decide (the scale makes up for it)."""
    ctx = [200, 33]
    q, caches, tables = batch(8, 2, 128, 16, ctx, BF16, 8)
    q = (q.float() * gain).to(BF16)
    scale = 128 ** -0.5 / gain
    out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, torch.tensor(ctx, dtype=torch.int32).cuda(), scale, 200)
    check(out, q, caches, reference(q, caches, tables, ctx, scale), scale)


@pytest.mark.parametrize("top", [30.0, 3000.0, 65408.0])
def test_large_values(pkv, cuda_dev, top):
    """V up to the largest that the format holds: P times its scale stays in float16's range."""
    n, Hkv, d = 150, 2, 128
    g = torch.Generator().manual_seed(4)
    key, value = torch.randn(n, Hkv, d, generator=g), torch.rand(n, Hkv, d, generator=g) * 2 - 1
    value[:, :, ::32] = 1.0
    caches = ref.empty_cache(10, Hkv, 16, d, 4, cuda_dev)
    slots = torch.arange(n, dtype=torch.int32).cuda()
    pkv.pkv_store_kvcache_int4(key.cuda(), (value * top).cuda(), *caches, slots)
    # rising scores: every later key may exceed the reference
    q = (key[-1].repeat_interleave(4, 0)[None] * 2).to(BF16).cuda()
    tables = torch.arange(10, dtype=torch.int32).cuda()[None]
    out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, torch.tensor([n], dtype=torch.int32).cuda(), d ** -0.5, n)
    check(out, q, caches, reference(q, caches, tables, [n], d ** -0.5), d ** -0.5)


def test_empty_batch(pkv, cuda_dev):
    q, caches, tables = batch(8, 2, 128, 16, [5], BF16, 8)
    out = pkv.pkv_paged_attention_decode_int4(q[:0], *caches, tables[:0], torch.empty(0, dtype=torch.int32, device=cuda_dev), 0.1, 5)
    assert out.shape == (0, 8, 128)


def test_captured_and_on_another_stream(pkv, cuda_dev):
    ctx = [700, 33, 2000]
    q, caches, tables = batch(16, 4, 128, 16, ctx, BF16, 9)
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    want = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, 0.09, 2000)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, 0.09, 2000, stream=other)
    other.synchronize()
    assert torch.equal(got, want)  # pieces are joined in order: the same bits
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, 0.09, 2000)
    for step in range(2):
        q.mul_(-1)
        lens.sub_(step)
        graph.replay()
        assert torch.equal(out, pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, 0.09, 2000))


def test_offsets_past_32_bits(pkv, cuda_dev):
    nb, Hkv, bs, d = 20000, 8, 256, 128
    kc = torch.zeros(nb, Hkv, bs, d // 2, dtype=torch.uint8, device=cuda_dev)
    ks = torch.zeros(nb, Hkv, bs, d // 32, dtype=F16, device=cuda_dev)
    caches = (kc, kc.clone(), ks, ks.clone())
    ctx, ids = 300, [nb - 1, 12345]
    g = torch.Generator().manual_seed(3)
    key, value = (torch.randn(ctx, Hkv, d, generator=g).to(BF16).cuda() for _ in range(2))
    slots = torch.tensor([ids[p // bs] * bs + p % bs for p in range(ctx)], dtype=torch.int32).cuda()
    pkv.pkv_store_kvcache_int4(key, value, *caches, slots)
    q = torch.randn(1, 32, d, generator=g).to(BF16).cuda()
    tables = torch.tensor([ids], dtype=torch.int32).cuda()
    out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, torch.tensor([ctx], dtype=torch.int32).cuda(), d ** -0.5, ctx)
    near = tuple(c[ids].contiguous() for c in caches)
    check(out, q, near, reference(q, near, torch.tensor([[0, 1]]), [ctx], d ** -0.5), d ** -0.5)
