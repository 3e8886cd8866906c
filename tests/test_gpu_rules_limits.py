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
