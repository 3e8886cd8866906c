"""Rotary positions with the cache write, against the definition in binary64.

Tolerance.  The kernels turn a pair in f32: the angle within 2^-25 of a turn's eighth and
rounded once, a sine and cosine within 2 ulp, the amplitude, two products and a sum each
rounded once: together below 7 x 2^-24 (|x_a| + |x_b|) amplitude.  The result is rounded to
its type, half a step: eps / 2 of it, or 2^-25 below float16's normal range.
"""
import pytest
import torch

import int4_reference as ref

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _within(got, want, mag):
    u = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 0.0
    tol = 7 * 2.0 ** -24 * mag + u * (want.abs() + 7 * 2.0 ** -24 * mag) + (2.0 ** -25 if got.dtype == F16 else 0.0)
    tol = torch.where(mag > 0, tol, 0.0)  # what is not rotated stays
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), f"worst error / tolerance {(err / tol.clamp(min=1e-30)).max().item():.3g}"


def inputs(n, Hq, Hkv, d, dtype, seed, layout="fused", slots=None, num_slots=512, pos_hi=20000):
    """(q, key, value, positions, slots) on the CPU side of the device's tensors."""
    g = torch.Generator().manual_seed(seed)
    heads = Hq + 2 * Hkv
    if layout == "fused":  # one projection's output
        x = torch.randn(n, heads, d, generator=g).to(dtype).cuda()
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    elif layout == "odd":  # strides and bases that no vector fits
        x = torch.randn(n, heads * d + 1, generator=g).to(dtype).cuda()[:, 1:]
        q, k, v = (x[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, heads)))
    else:
        q, k, v = (torch.randn(n, h, d, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    pos = torch.randint(0, pos_hi, (n,), generator=g, dtype=torch.int32)
    if slots is None:
        slots = torch.randperm(num_slots, generator=g)[:n].to(torch.int32)
        slots[n // 2:n // 2 + n // 5] = -1
    return q, k, v, pos.cuda(), slots.cuda()


def rope_of(pkv, r, scaling):
    kw = {None: {}, "linear": dict(factor=4.0), "ntk": dict(factor=8.0),
          "yarn": dict(factor=16.0, original_len=2048)}[scaling]
    return pkv.pkv_rope_frequencies(r, scaling=scaling, **kw), ref.frequencies(r, scaling=scaling, **kw)


SHAPES = [  # Hq, Hkv, d, rotary_dim, interleaved, layout
    (8, 2, 128, 128, False, "fused"), (8, 2, 128, 128, True, "fused"), (4, 4, 128, 64, False, "apart"),
    (6, 3, 128, 32, True, "fused"), (4, 1, 64, 64, False, "fused"), (5, 5, 96, 96, False, "fused"), (3, 3, 80, 48, True, "apart"),
    (2, 2, 256, 256, False, "fused"), (2, 1, 512, 512, True, "fused"), (4, 2, 128, 20, False, "fused"),
    (4, 2, 128, 2, True, "apart"), (4, 2, 128, 128, False, "odd"), (3, 1, 40, 10, True, "apart"), (1, 1, 1024, 1024, False, "fused"),
    (0, 4, 128, 128, False, "apart"), (8, 2, 128, 0, False, "fused"), (33, 7, 128, 128, False, "fused")]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,n,scaling", [(BF16, 37, "yarn"), (F16, 1, None), (F32, 130, "ntk"), (BF16, 300, "linear")])
def test_rope_store(pkv, cuda_dev, shape, dtype, n, scaling):
    Hq, Hkv, d, r, inter, layout = shape
    nb, bs = 32, 16
    q, k, v, pos, slots = inputs(n, Hq, Hkv, d, dtype, n + d, layout)
    rope, (freq, amp) = rope_of(pkv, r, scaling)
    g = torch.Generator().manual_seed(5)
    kc, vc = (torch.randn(nb, bs, Hkv, d, generator=g).to(dtype).cuda() for _ in range(2))
    kc0, vc0 = kc.clone(), vc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, kc, vc, slots, interleaved=inter, err_flag=err)
    assert int(err) == 0 and out.shape == q.shape and out.is_contiguous()
    _within(out, *ref.rotate(q, pos, freq, amp, inter))
    want, mag = ref.rotate(k, pos, freq, amp, inter)
    live = slots >= 0
    at = slots[live].long()
    _within(kc.flatten(0, 1)[at], want[live.cpu()], mag[live.cpu()])
    assert torch.equal(vc.flatten(0, 1)[at], v[live])
    rest = torch.ones(nb * bs, dtype=torch.bool, device=cuda_dev)
    rest[at] = False
    for new, old in ((kc, kc0), (vc, vc0)):
        assert torch.equal(new.flatten(0, 1)[rest], old.flatten(0, 1)[rest])


def test_far_and_negative_positions(pkv, cuda_dev):
    """Angles of positions up to 2^31 either way are as exact as those of small ones."""
    pos = torch.tensor([0, 1, -1, 131072, 10 ** 6, -10 ** 6, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    n = pos.numel()
    g = torch.Generator().manual_seed(1)
    q = torch.randn(n, 2, 64, generator=g).cuda()
    k = torch.randn(n, 1, 64, generator=g).cuda()
    cache = torch.zeros(1, 16, 1, 64).cuda()
    rope = pkv.pkv_rope_frequencies(64)
    out = pkv.pkv_rope_store_kvcache(q, k, k, pos.cuda(), rope, cache, cache.clone(), torch.arange(n, dtype=torch.int32).cuda())
    freq, amp = ref.frequencies(64)
    want, mag = ref.rotate(q, pos, freq, amp, False)
    # the table's frequency is a binary64 quotient: off by 2^-53 of it, times the position
    slack = 2 * 3.15 * 2.0 ** -53 * pos.double().abs()[:, None, None] * mag
    err = (out.cpu().double() - want).abs()
    assert bool((err <= 7 * 2.0 ** -24 * mag + slack).all())


def test_turned_back(pkv, cuda_dev):
    q, k, v, pos, slots = inputs(50, 4, 2, 128, F32, 3)
    rope = pkv.pkv_rope_frequencies(128, scaling="yarn", factor=8.0, original_len=1024)
    cache = torch.zeros(32, 16, 2, 128, device=cuda_dev)
    there = pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, cache, cache.clone(), slots)
    back = pkv.pkv_rope_store_kvcache(there, k, v, pos, rope.inverse(), cache, cache.clone(), slots)
    # two turns of pairs whose |x_a| + |x_b| is at most sqrt(2) times the pair's norm, which stays
    mag = 4 * q.double().unflatten(-1, (2, 64)).norm(dim=-2, keepdim=True).expand(-1, -1, 2, -1).flatten(-2)
    assert bool(((back - q).abs().double() <= 7 * 2.0 ** -24 * mag).all())


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
@pytest.mark.parametrize("r", [0, 2, 64, 128])
def test_frequencies(pkv, cuda_dev, scaling, r):
    rope, (freq, amp) = rope_of(pkv, r, scaling)
    assert rope.rotary_dim == r and abs(rope.amplitude - amp) < 1e-15 and rope.turns.device.type == "cuda"
    given = pkv.pkv_rope_turns(freq, amplitude=amp)
    for got in (rope, given):
        t = (got.turns.cpu().double() / 2.0 ** 64) % 1.0
        want = torch.tensor(freq, dtype=torch.float64) / (2 * torch.pi)
        # pow and two operations, relative; and an entry is a whole multiple of 2^-64, cut off: below 2^-64
        assert bool(((t - want).abs() <= 8 * 2.0 ** -53 * want + 2.0 ** -64).all())


@pytest.mark.parametrize("layout", ["fused", "odd"])
def test_bad_slots_are_skipped(pkv, cuda_dev, layout):
    slots = torch.tensor([3, -1, 512, 7, -2, 511, 2 ** 31 - 1], dtype=torch.int32)
    q, k, v, pos, slots = inputs(7, 4, 2, 128, BF16, 9, layout, slots)
    rope, (freq, amp) = rope_of(pkv, 128, None)
    kc, vc = (torch.full((32, 16, 2, 128), 3.0, dtype=BF16, device=cuda_dev) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, kc, vc, slots, err_flag=err)
    assert int(err) == pkv.ERRBIT_SLOT_RANGE
    _within(out, *ref.rotate(q, pos, freq, amp, False))
    rows = vc.flatten(0, 1)
    assert torch.equal(rows[[3, 7, 511]], v[[0, 3, 5]])
    rows[[3, 7, 511]] = 3.0
    assert bool((vc == 3.0).all())


@pytest.mark.parametrize("d,r", [(128, 128), (40, 20)])  # the vector kernel, the scalar one
def test_in_place(pkv, cuda_dev, d, r):
    q, k, v, pos, slots = inputs(33, 8, 2, d, BF16, 4, "apart")
    rope, _ = rope_of(pkv, r, None)
    cache = torch.zeros(32, 16, 2, d, dtype=BF16, device=cuda_dev)
    want = pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, cache, cache.clone(), slots)
    got = pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, cache, cache.clone(), slots, out=q)
    assert got is q and torch.equal(got, want)


def test_large_rows_cross_32_bits(pkv, cuda_dev):
    """A pool and a batch whose offsets pass 2^31 elements."""
    nb, bs, H, d, n = 9000, 256, 8, 128, 5  # 2.36e9 elements
    kc = torch.zeros(nb, bs, H, d, dtype=F16, device=cuda_dev)
    vc = torch.zeros_like(kc)
    slots = torch.tensor([0, nb * bs - 1, 2 ** 21, 2 ** 21 + 1, nb * bs // 2], dtype=torch.int32)
    q, k, v, pos, slots = inputs(n, 8, H, d, F16, 2, "fused", slots)
    rope, (freq, amp) = rope_of(pkv, d, None)
    pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, kc, vc, slots)
    _within(kc.view(-1, H, d)[slots.long()], *ref.rotate(k, pos, freq, amp, False))
    assert torch.equal(vc.view(-1, H, d)[slots.long()], v)


def test_captured_and_on_another_stream(pkv, cuda_dev):
    q, k, v, pos, slots = inputs(64, 8, 2, 128, BF16, 6)
    rope, _ = rope_of(pkv, 128, None)
    kc, vc = (torch.zeros(32, 16, 2, 128, dtype=BF16, device=cuda_dev) for _ in range(2))
    want = pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, kc, vc, slots)
    want_k = kc.clone()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    kc.zero_()
    other.wait_stream(torch.cuda.current_stream())
    got = pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, kc, vc, slots, stream=other)
    other.synchronize()
    assert torch.equal(got, want) and torch.equal(kc, want_k)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, kc, vc, slots, out=out)
    for shift in (0, 5):
        pos.add_(shift)
        kc.zero_()
        graph.replay()
        want = pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, kc.clone(), vc.clone(), slots)
        assert torch.equal(out, want)
