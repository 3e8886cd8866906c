"""The score-rule prefill at its limits: what rows that a query does not see may hold,
blocks that are missing, unused table entries, values at the ends of their ranges."""
import pytest
import torch

import score_reference as sr
from test_gpu_prefill_mod import _case, _codes, _slopes

pytestmark = pytest.mark.gpu

RULES = {"plain": {}, "bounded": {"softcap": 8.0}, "cap": {"softcap": 60.0}, "alibi": {"alibi_slopes": True},
         "cap-alibi": {"softcap": 5.0, "alibi_slopes": True}}


def _rules(name, Hq, dev):
    return {k: _slopes(Hq, dev) if v is True else v for k, v in RULES[name].items()}


def _caches(pkv, fmt, batch, dev):
    return _codes(pkv, fmt, batch, 3, dev) if fmt else ((batch.k_cache, None), (batch.v_cache, None))


def _call(pkv, q, caches, tables, starts, cu, scale, max_q, rules, **kw):
    (kc, ks), (vc, vs) = caches
    err = torch.zeros(1, dtype=torch.int32, device=q.device)
    out = pkv.pkv_paged_attention_prefill_mod(q, kc, vc, tables, starts, cu, scale, max_q, k_scale=ks, v_scale=vs,
                                              err_flag=err, **rules, **kw)
    return out, int(err.item())


def _reference(q, caches, tables, starts, ns, scale, rules):
    (kc, ks), (vc, vs) = caches
    return sr.prefill(q, sr.dequantize(kc, ks), sr.dequantize(vc, vs), tables, starts, ns, scale,
                      rules.get("softcap", 0.0), rules.get("alibi_slopes"), rules.get("key_starts"))


def _dropping(q, caches, table, start, n, gone, scale, rules):
    """The definition with the scores of the keys in the 16-token blocks `gone` at minus infinity."""
    Hq, G = q.shape[1], q.shape[1] // caches[0][0].shape[2]
    total = start + n
    k, v = (sr.rows_of(sr.dequantize(c, x), table, total) for c, x in caches)
    pos, t = torch.arange(start, total), torch.arange(total)
    seen = (t <= pos[:, None]) & ~torch.isin(t // 16, torch.tensor(gone))
    want, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for h in range(Hq):
        x = scale * (q[:, h].cpu().double() @ k[:, h // G].T)
        if "softcap" in rules:
            x = rules["softcap"] * torch.tanh(x / rules["softcap"])
        if "alibi_slopes" in rules:
            x = x - rules["alibi_slopes"][h].cpu().double() * (pos[:, None] - t)
        w = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
        want[:, h], mag[:, h] = w @ v[:, h // G], w @ v[:, h // G].abs()
    return want, mag, seen.sum(1).double()[:, None, None]


@pytest.mark.parametrize("rule", ["plain", "bounded", "cap", "cap-alibi"])
@pytest.mark.parametrize("fmt", [None, "fp8"])
@pytest.mark.parametrize("start", [10, 1034])
@pytest.mark.parametrize("at", [32, 96, 160])
def test_nonfinite_in_later_tokens(pkv, cuda_dev, fmt, rule, start, at):
    """NaN and infinities in tokens from row `at` on, where a pair of query tiles begins (64 rows a
    pair here, counted from the last one down; a key half block ends inside it), leave no trace in
    the rows before: one pair's values do not reach another's.  start 1034: the keys are split."""
    spans = [(start, 200)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 16, 4, 16, spans, 8, cuda_dev)
    caches = _caches(pkv, fmt, batch, cuda_dev)
    rules = _rules(rule, 16, cuda_dev)
    ref = _reference(q[:at], caches, batch.block_tables, [start], [at], batch.scale, rules)
    clean = caches[1][0].clone()
    for t in range(start + at, start + 200):
        for c, _ in caches:
            c[int(batch.block_tables[0, t // 16]), t % 16] = 0x7F if fmt else (float("nan") if t % 2 else float("inf"))
    out, err = _call(pkv, q, caches, batch.block_tables, starts, cu, batch.scale, 200, rules)
    assert err == 0
    sr.assert_within(out[:at], ref, clean, caches[1][1])


@pytest.mark.parametrize("fmt", [None, "fp8", "int8"])
@pytest.mark.parametrize("rule", ["plain", "bounded", "alibi"])
@pytest.mark.parametrize("bs", [16, 48, 256])
def test_entries_that_nobody_sees(pkv, cuda_dev, fmt, rule, bs):
    """Table entries in front of every row's window, or behind the last row that sees anything, are not
    used: they may be missing or wrong without an error, and their blocks' scales are not read."""
    spans = [(300, 60), (0, 90), (700, 20)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 16, 8, bs, spans, 8, cuda_dev)
    caches = _caches(pkv, fmt, batch, cuda_dev)
    ks = [p - 69 for p in range(300, 360)] + [0 if p < 70 else 10 ** 6 for p in range(90)] + [690] * 20
    rules = {**_rules(rule, 16, cuda_dev), "key_starts": torch.tensor(ks, dtype=torch.int32, device=cuda_dev)}
    ref = _reference(q, caches, batch.block_tables, [300, 0, 700], ns, batch.scale, rules)
    tables = batch.block_tables.clone()
    unused = [(0, j) for j in range(231 // bs)] + [(1, j) for j in range(sr.cdiv(70, bs), sr.cdiv(90, bs))]
    unused += [(2, j) for j in range(690 // bs)]
    for i, (b, j) in enumerate(unused):
        tables[b, j] = -1 if i % 2 else 77_777
    out, err = _call(pkv, q, caches, tables, starts, cu, batch.scale, 60 + 30, rules)
    assert err == 0
    sr.assert_within(out, ref, caches[1][0], caches[1][1])
    if fmt:
        scales = caches[1][1].clone()
        for b, j in unused:
            for _, s in caches:
                s[batch.block_tables[b, j]] = float("nan") if b else float("inf")
        out, err = _call(pkv, q, caches, batch.block_tables, starts, cu, batch.scale, 60 + 30, rules)
        assert err == 0
        sr.assert_within(out, ref, caches[1][0], scales)


@pytest.mark.parametrize("fmt", [None, "fp8", "int8"])
@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("spans", [[(100, 90), (0, 40)], [(1500, 40)]])
def test_missing_blocks(pkv, cuda_dev, fmt, rule, dtype, spans):
    """Table entries out of range among the used ones: their tokens are dropped, whether they are a
    part of a 64-key step or all of it, in a span whose keys are split too."""
    batch, q, starts, cu, ns = _case(dtype, 16, 8, 16, spans, 72, cuda_dev)
    caches = _caches(pkv, fmt, batch, cuda_dev)
    rules = _rules(rule, 16, cuda_dev)
    tables = batch.block_tables.clone()
    gone = [1] + list(range(4, 8))  # positions 16 .. 31 and 64 .. 127
    for j in gone:
        tables[0, j] = -1 if j % 2 else 10_000
    out, err = _call(pkv, q, caches, tables, starts, cu, batch.scale, max(ns), rules)
    assert err == pkv.ERRBIT_BLOCK_RANGE
    s, n = spans[0]
    ref = _dropping(q[:n], caches, batch.block_tables[0], s, n, gone, batch.scale, rules)
    sr.assert_within(out[:n], ref, caches[1][0], caches[1][1])
    if len(spans) > 1:  # the other sequence is whole
        ref = _reference(q[n:], caches, batch.block_tables[1:], [0], ns[1:], batch.scale, rules)
        sr.assert_within(out[n:], ref, caches[1][0], caches[1][1])


@pytest.mark.parametrize("fmt", [None, "fp8", "int8"])
@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_missing_blocks_of_a_decode_step(pkv, cuda_dev, fmt, rule, dtype):
    """The same for a decode call: whole stages of 16 tokens are dropped, one of them the last."""
    batch, q, _, _, _ = _case(dtype, 16, 8, 16, [(199, 1), (77, 1)], 72, cuda_dev)
    caches = _caches(pkv, fmt, batch, cuda_dev)
    rules = _rules(rule, 16, cuda_dev)
    tables = batch.block_tables.clone()
    gone = [1] + list(range(4, 8)) + [12]
    for j in gone:
        tables[0, j] = -1 if j % 2 else 10_000
    (kc, ks), (vc, vs) = caches
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    ctx = torch.tensor([200, 78], dtype=torch.int32, device=cuda_dev)
    out = pkv.pkv_paged_attention_decode_mod(q, kc, vc, tables, ctx, batch.scale, 200, k_scale=ks, v_scale=vs,
                                             err_flag=err, **rules)
    assert int(err.item()) == pkv.ERRBIT_BLOCK_RANGE
    ref = _dropping(q[:1], caches, batch.block_tables[0], 199, 1, gone, batch.scale, rules)
    sr.assert_within(out[:1], ref, vc, vs)
    ref = _reference(q[1:], caches, batch.block_tables[1:], [77], [1], batch.scale, rules)
    sr.assert_within(out[1:], ref, vc, vs)


@pytest.mark.parametrize("softcap", [8.0, 50.0, 60.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", [None, "fp8"])
def test_rows_do_not_depend_on_their_neighbours(pkv, cuda_dev, softcap, dtype, fmt):
    """A row's bits are the same whatever the scores of the rows beside it and of keys that it does not see."""
    spans = [(200, 120)]
    batch, q, starts, cu, ns = _case(dtype, 8, 8, 16, spans, 31, cuda_dev)
    caches = _caches(pkv, fmt, batch, cuda_dev)
    args = (batch.block_tables, starts, cu, batch.scale, 120, {"softcap": softcap})
    want, _ = _call(pkv, q, caches, *args)
    loud = q.clone()
    loud[::2] *= 100
    got, _ = _call(pkv, loud, caches, *args)
    assert torch.equal(got[1::2], want[1::2])
    if not fmt:
        for t in range(316, 320):
            batch.k_cache[int(batch.block_tables[0, t // 16]), t % 16] *= 1000
        got, _ = _call(pkv, q, caches, *args)
        assert torch.equal(got[:116], want[:116])


@pytest.mark.parametrize("fmt", [None, "fp8"])
@pytest.mark.parametrize("rule", ["plain", "cap", "alibi"])
@pytest.mark.parametrize("upto", [256, 2001])
def test_nan_in_visible_keys(pkv, cuda_dev, fmt, rule, upto):
    """Visible NaN keys make the row NaN, also where they are all that one CTA of a split span sees."""
    spans = [(2000, 1)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 8, 2, 16, spans, 5, cuda_dev)
    caches = _caches(pkv, fmt, batch, cuda_dev)
    for t in range(upto):
        caches[0][0][int(batch.block_tables[0, t // 16]), t % 16] = 0x7F if fmt else float("nan")
    assert pkv.pkv_paged_attention_prefill_mod_workspace_size(1, 8, 2, 128, 16, 1, batch.block_tables.shape[1]) > 0
    out, _ = _call(pkv, q, caches, batch.block_tables, starts, cu, batch.scale, 1, _rules(rule, 8, cuda_dev))
    assert bool(out.isnan().all())


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("softcap", [0.0, 10.0])
def test_smallest_scales(pkv, cuda_dev, fmt, softcap):
    """V scales from 2^-100 to 2^-97 everywhere, and zero blocks: no bits are lost.  The comparison is at
    2^100 times the values, exact in bf16 and in the reference."""
    spans = [(100, 60), (0, 300)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 8, 8, 16, spans, 8, cuda_dev)
    (kc, ks), (vc, vs) = _codes(pkv, fmt, batch, 3, cuda_dev)
    g = torch.Generator().manual_seed(2)
    vs.copy_((1 + 7 * torch.rand(vs.shape, generator=g)).to(cuda_dev) * 2.0 ** -100)
    for b in range(2):
        i = int(batch.block_tables[b, 2])
        vc[i], vs[i] = 0, 0
    rules = {"softcap": softcap}
    out, err = _call(pkv, q, ((kc, ks), (vc, vs)), batch.block_tables, starts, cu, batch.scale, 300, rules)
    up = vs * 2.0 ** 100
    ref = _reference(q, ((kc, ks), (vc, up)), batch.block_tables, [100, 0], ns, batch.scale, rules)
    assert err == 0
    sr.assert_within(out * 2.0 ** 100, ref, vc, up)


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("gain", [2.0 ** -44, 2.0 ** 42])
def test_bounded_cap_with_values_of_extreme_size(pkv, cuda_dev, sign, gain):
    """Every score at one end of a cap of 50, where P is 2^-72 or 2^72 without a reference maximum, times V
    whose values are near the ends of what stays in f32's range (below 2^54 / keys; above 2^-53)."""
    spans = [(0, 300)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 8, 8, 16, spans, 8, cuda_dev)
    g = torch.Generator().manual_seed(4)
    base = torch.randn(128, generator=g)
    base *= 128 ** 0.5 / base.norm()
    rows = torch.randn(batch.k_cache.shape, generator=g)
    batch.k_cache.copy_((base + 0.05 * rows).to(torch.bfloat16))
    q.copy_((sign * 40 * base).to(torch.bfloat16).expand_as(q))  # scores near +-450
    batch.v_cache.mul_(gain)
    caches, rules = ((batch.k_cache, None), (batch.v_cache, None)), {"softcap": 50.0}
    out, err = _call(pkv, q, caches, batch.block_tables, starts, cu, batch.scale, 300, rules)
    assert err == 0
    sr.assert_within(out, _reference(q, caches, batch.block_tables, [0], ns, batch.scale, rules), batch.v_cache)


@pytest.mark.parametrize("fmt", [None, "int8"])
def test_generous_bound_on_the_rows(pkv, cuda_dev, fmt):
    """A bound so far above the rows that a sequence's tile pairs take several grids."""
    spans = [(37, 64), (0, 1), (127, 130)]
    batch, q, starts, cu, ns = _case(torch.bfloat16, 8, 1, 16, spans, 8, cuda_dev)
    caches = _caches(pkv, fmt, batch, cuda_dev)
    rules = _rules("cap-alibi", 8, cuda_dev)
    out, err = _call(pkv, q, caches, batch.block_tables, starts, cu, batch.scale, 1 << 21, rules)
    assert err == 0  # 16 positions a tile: 65536 pairs
    ref = _reference(q, caches, batch.block_tables, [s for s, _ in spans], ns, batch.scale, rules)
    sr.assert_within(out, ref, caches[1][0], caches[1][1])


@pytest.mark.parametrize("fmt", [None, "fp8", "int8"])
@pytest.mark.parametrize("bs", [16, 48, 256])
@pytest.mark.parametrize("append", [False, True])
def test_entries_in_front_of_a_decode_window(pkv, cuda_dev, fmt, bs, append):
    """Released blocks in front of the window: no error, and their scales are not read."""
    ctx, first = [400, 78, 700, 64], [231, 70, 699, 64]
    batch, q, _, _, _ = _case(torch.bfloat16, 16, 8, bs, [(c - 1, 1) for c in ctx], 8, cuda_dev)
    caches = _caches(pkv, fmt, batch, cuda_dev)
    (kc, ks), (vc, vs) = caches
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    rules = {"softcap": 20.0, "key_starts": i32(first)}
    row = {}
    if append:
        key, value = (torch.randn(4, 8, 128, device=cuda_dev).to(torch.bfloat16) for _ in range(2))
        pkv.pkv_paged_attention_decode_mod(q, kc, vc, batch.block_tables, i32(ctx), batch.scale, 700, key=key, value=value,
                                           k_scale=ks, v_scale=vs, **rules)  # the same row twice: the caches as they will be
        row = {"key": key, "value": value}
    ref = _reference(q, caches, batch.block_tables, [c - 1 for c in ctx], [1] * 4, batch.scale, rules)
    tables, scales = batch.block_tables.clone(), None if vs is None else vs.clone()
    for b, (c, f) in enumerate(zip(ctx, first)):
        for j in range(min(f // bs, (c - 1) // bs)):
            tables[b, j] = -1 if j % 2 else 77_777
            for s in (ks, vs):
                if s is not None:
                    s[batch.block_tables[b, j]] = float("nan")
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    for entries in (tables, batch.block_tables):
        out = pkv.pkv_paged_attention_decode_mod(q, kc, vc, entries, i32(ctx), batch.scale, 700, k_scale=ks, v_scale=vs,
                                                 err_flag=err, **row, **rules)
        assert int(err.item()) == 0
        sr.assert_within(out, ref, vc, scales)
