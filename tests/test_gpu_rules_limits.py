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
