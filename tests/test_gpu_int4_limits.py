"""The 4-bit cache at the ends of its inputs' ranges.  Stored codes and scales are equal to the
definition's in binary64, bit for bit, in the vector kernels ("apart") and the scalar one ("odd");
attention is within the tolerance of its own tests."""
import pytest
import torch

import int4_reference as ref
from test_gpu_int4_cache import _same
from test_gpu_int4_decode import batch, check as decode_check, reference
from test_gpu_int4_prefill import case as prefill_case, check as prefill_check
from test_gpu_rope import BF16, F16, F32, rope_of

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def _laid_out(x, layout):
    """x [n, H, d] on the device, its rows aligned for vectors or not."""
    n, H, d = x.shape
    if layout == "apart":
        return x.cuda()
    buf = torch.zeros(n, H * d + 1, dtype=x.dtype, device="cuda")
    key = buf[:, 1:].unflatten(1, (H, d))
    key.copy_(x)
    return key


def _store_and_compare(pkv, x, pos, rope, freq, amp, inter, layout):
    """Stores x [n, H, d] as keys, rotated, and as values; compares both caches."""
    n, H, d = x.shape
    nb = -(-n // 16)
    slots = torch.arange(n, dtype=torch.int32)
    caches = ref.empty_cache(nb, H, 16, d, 4, "cuda")
    want = ref.stored(caches, ref.rotate(x, pos, freq, amp, inter)[0], x.double(), slots)
    key = _laid_out(x, layout)
    pkv.pkv_rope_store_kvcache_int4(key, key, key, pos.cuda(), rope, *caches, slots.cuda(), interleaved=inter)
    _same(caches, want)


@pytest.mark.parametrize("scaling", [None, "yarn"])
@pytest.mark.parametrize("layout", ["apart", "odd"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_rotated_keys_beyond_the_range(pkv, cuda_dev, dtype, inter, layout, scaling):
    """Infinities, NaN and values whose rotation leaves float32: what is beyond 65408 saturates, and the
    rest of its group is stored under the largest scale.  No sine or cosine here is near 0 but at position 0."""
    d = 128
    plants = [{3: INF}, {70: -INF}, {3: INF, 67: INF}, {3: -INF, 67: INF}, {8: INF, 9: -INF}, {9: NAN, 40: INF}, {5: NAN}]
    if dtype != F16:
        plants += [{5: 3.3e38, 69: 3.3e38}, {4: 3.3e38, 5: -3.3e38}, {20: 3.0e38, 21: 3.3e38, 84: -3.0e38, 85: 3.3e38},
                   {j: 3.3e38 * (-1) ** (j // 3) for j in range(d)}]
    positions = [0, 1, 7, 12345]
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(len(plants) * len(positions), 2, d, generator=g) * 20000).clamp(-60000, 60000)
    for i in range(x.shape[0]):
        for j, v in plants[i % len(plants)].items():
            x[i, 0, j] = v
    pos = torch.tensor(positions, dtype=torch.int32).repeat_interleave(len(plants))
    rope, (freq, amp) = rope_of(pkv, d, scaling)
    _store_and_compare(pkv, x.to(dtype), pos, rope, freq, amp, inter, layout)


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("layout", ["apart", "odd"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_largest_value_of_seven_and_a_half_steps(pkv, cuda_dev, dtype, inter, layout, turned):
    """Small scales are multiples k of 2^-24, so that a group's largest value may be 7.5 of them, a tie whose
    even side, 8, is no code; so may 70080 under the largest scale.  Each in all places of a group, both signs; in
    float32 their neighbours too.  At position 0, where a turn is exact, and as they stand."""
    tops = [7.5 * k * 2.0 ** -24 for k in range(1, 8)]
    if dtype == F32:
        tops.append(70080.0)
        tops += [torch.nextafter(torch.tensor(t), torch.tensor(to)).item() for t in tops for to in (0.0, INF)]
    tops = [t for t in tops if torch.tensor(t).to(dtype).double() == t]
    assert len(tops) >= 3
    g = torch.Generator().manual_seed(6)
    groups = []
    for t in tops:
        for sign in (1, -1):
            for place in range(32):
                x = t * torch.randint(-7, 8, (32,), generator=g) / 7.5
                x[place] = sign * t
                groups.append(x)
    x = torch.stack(groups).reshape(-1, 1, 128).to(dtype)
    pos = torch.zeros(x.shape[0], dtype=torch.int32)
    r = 128 if turned else 0
    rope, (freq, amp) = rope_of(pkv, r, None)
    _store_and_compare(pkv, x, pos, rope, freq, amp, inter, layout)


@pytest.mark.parametrize("layout", ["apart", "odd"])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_pairs_that_cancel(pkv, cuda_dev, dtype, layout):
    """A group of small values turned from large ones, which float32 has wrong by many codes: angles of some
    1e-9 (so far below float32's of a turn), and pairs whose rotation is a remainder of 2^-24 of them."""
    n, d, half = 64, 128, 64
    g = torch.Generator().manual_seed(7)
    size = 10000 + 50000 * torch.rand(n, 1, half, generator=g)
    big = (size * (1 - 2 * torch.randint(0, 2, size.shape, generator=g))).to(dtype)
    pos = torch.randint(1, 4, (n,), generator=g, dtype=torch.int32)
    freq = [(0.5 + i / half) * 1e-9 for i in range(half)]
    _store_and_compare(pkv, torch.cat([torch.zeros_like(big), big], -1), pos, pkv.pkv_rope_turns(freq), freq, 1.0, False, layout)
    if dtype == F32:
        freq = [0.3 + i / half for i in range(half)]
        t = ref.angles(pos, freq)[:, None]
        first = big.double() * torch.tan(t)  # first cos - big sin = 0 but for its rounding
        _store_and_compare(pkv, torch.cat([first.float(), big], -1), pos, pkv.pkv_rope_turns(freq), freq, 1.0, False, layout)


@pytest.mark.parametrize("gain", [2.0 ** -119, 2.0 ** -105, 2.0 ** 120])
def test_decode_of_queries_and_scales_far_from_one(pkv, cuda_dev, gain):
    """The factor of the scores leaves float32 below: they are all 0, and every key counts alike.  Where it leaves it above,
    scores of 0 stay 0."""
    ctx = [200, 33, 1]
    q, caches, tables = batch(8, 2, 128, 16, ctx, BF16, 8)
    scale = 1e-12
    if gain > 1:
        q, scale = torch.zeros_like(q), 1e20
        q[..., 5] = gain
        caches[0][:, :, :, 0:4] = 0x88  # dims 0 .. 7 of K: zeros
    else:
        q = (q.float() * gain).to(BF16)
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    for bound in (200, 5000):
        out = pkv.pkv_paged_attention_decode_int4(q, *caches, tables, lens, scale, bound)
        decode_check(out, q, caches, reference(q, caches, tables, ctx, scale), 0.0 if gain > 1 else scale)


@pytest.mark.parametrize("rule", ["plain", "cap", "alibi"])
@pytest.mark.parametrize("gain", [2.0 ** -119, 2.0 ** -105, 2.0 ** 120])
@pytest.mark.parametrize("spans", [[(0, 70), (130, 5)], [(0, 1100), (30, 200)]], ids=["fused", "widened"])
def test_prefill_of_queries_and_scales_far_from_one(pkv, cuda_dev, spans, gain, rule):
    q, caches, tables, starts, cu, ns = prefill_case(8, 2, 16, spans, BF16, 9)
    rules = {"plain": {}, "cap": {"softcap": 20.0}, "alibi": {"alibi_slopes": torch.exp2(-torch.arange(1.0, 9.0)).cuda()}}[rule]
    scale = 1e-12
    if gain > 1:
        q, scale = torch.zeros_like(q), 1e20
        q[..., 5] = gain
        caches[0][:, :, :, 0:4] = 0x88
    else:
        q = (q.float() * gain).to(BF16)
    prefill_check(pkv, q, caches, tables, starts, cu, ns, spans, rules, scale)
