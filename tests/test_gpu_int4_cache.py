"""The 4-bit cache written, with and without rotary positions, and read back: codes, scales
and values are equal to the definition's in binary64, bit for bit."""
import pytest
import torch

import int4_reference as ref
from test_gpu_rope import BF16, F16, F32, inputs, rope_of

pytestmark = pytest.mark.gpu


def _same(got, want):
    for a, b, name in zip(got, want, ("k codes", "v codes", "k scales", "v scales")):
        x = a.cpu()
        differ = (x.view(torch.int16) != b.view(torch.int16)) if x.dtype == F16 else x != b
        assert not bool(differ.any()), f"{name}: {int(differ.sum())} of {x.numel()} differ"


SHAPES = [  # Hq, Hkv, d, rotary_dim, interleaved, layout
    (8, 2, 128, 128, False, "fused"), (8, 2, 128, 128, True, "fused"), (4, 4, 128, 64, False, "apart"),
    (6, 3, 128, 32, True, "fused"), (6, 3, 128, 40, True, "fused"), (4, 2, 128, 32, False, "fused"), (4, 1, 64, 64, False, "fused"),
    (5, 5, 96, 96, True, "fused"), (5, 5, 96, 96, False, "fused"), (2, 2, 256, 256, False, "fused"), (2, 1, 512, 512, True, "fused"),
    (4, 2, 128, 20, False, "fused"), (4, 2, 32, 32, True, "fused"), (4, 2, 128, 128, False, "odd"), (33, 7, 128, 128, False, "fused")]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,n,scaling,bs", [(BF16, 37, "yarn", 16), (F16, 1, None, 256), (F32, 130, "ntk", 48),
                                                (F16, 300, "linear", 16)])
def test_rope_store_int4(pkv, cuda_dev, shape, dtype, n, scaling, bs):
    Hq, Hkv, d, r, inter, layout = shape
    nb = -(-512 // bs)
    q, k, v, pos, slots = inputs(n, Hq, Hkv, d, dtype, n + d, layout)
    rope, (freq, amp) = rope_of(pkv, r, scaling)
    caches = ref.empty_cache(nb, Hkv, bs, d, 3, cuda_dev)
    want = ref.stored(caches, ref.rotate(k, pos, freq, amp, inter)[0], v.cpu().double(), slots)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = pkv.pkv_rope_store_kvcache_int4(q, k, v, pos, rope, *caches, slots, interleaved=inter, err_flag=err)
    assert int(err) == 0
    _same(caches, want)
    plain = torch.zeros(nb, bs, Hkv, d, dtype=dtype, device=cuda_dev)
    assert torch.equal(out, pkv.pkv_rope_store_kvcache(q, k, v, pos, rope, plain, plain.clone(), slots, interleaved=inter))


def test_many_rotated_values(pkv, cuda_dev):
    """Two million rotated values, of which some lie within f32's error of a rounding border."""
    n, H, d = 2000, 8, 128
    q, k, v, pos, slots = inputs(n, 8, H, d, F16, 77, "fused", torch.arange(n, dtype=torch.int32))
    rope, (freq, amp) = rope_of(pkv, d, "yarn")
    caches = ref.empty_cache(n // 16, H, 16, d, 3, cuda_dev)
    pkv.pkv_rope_store_kvcache_int4(q, k, v, pos, rope, *caches, slots)
    y = ref.rotate(k, pos, freq, amp, False)[0]
    s = ref.scales(y)
    rows = caches[2].transpose(1, 2).flatten(0, 1).cpu()
    assert torch.equal(rows.view(torch.int16), s.view(torch.int16))
    assert torch.equal(caches[0].transpose(1, 2).flatten(0, 1).cpu(), ref.pack(ref.codes(y, s)))


@pytest.mark.parametrize("layout", ["apart", "odd"])
@pytest.mark.parametrize("turned", [False, True])
def test_borders(pkv, cuda_dev, layout, turned):
    """Ties, saturation, zeros, tiny and huge groups, infinities and NaN; also at position 0, where a turn is exact."""
    rows = []
    tie = torch.arange(32) * 0.5 - 7.5   # halves of the scale 1
    tie[0] = 7.0
    rows += [tie, tie * 3, tie * 2.0 ** -20, -tie * 2.0 ** 12]
    rows += [torch.zeros(32), torch.full((32,), 2.0 ** -24), torch.full((32,), 1e-7), torch.full((32,), 3.0 * 2.0 ** -23)]
    rows += [torch.linspace(-3e38, 3e38, 32), torch.linspace(-70000, 70000, 32), torch.linspace(-65408, 65408, 32)]
    rows += [torch.where(torch.arange(32) == k, v, tie) for k, v in ((3, float("nan")), (5, float("inf")), (9, -float("inf")))]
    rows += [torch.full((32,), float("nan")), tie * 7 * 1.00390625, tie + 2.0 ** -22, tie - 2.0 ** -22]
    # maxima around a midpoint of two scales: 7 x (1 + 2^-8), and its neighbours
    for m in (7 * (1 + 2.0 ** -8), 7 * (1 + 3 * 2.0 ** -8)):
        for step in (-1, 0, 1):
            top = torch.nextafter(torch.tensor(m), torch.tensor(float("inf") if step > 0 else 0.0)) if step else torch.tensor(m)
            rows.append(torch.cat([top[None], tie[1:]]))
    while len(rows) % 4:
        rows.append(tie)
    x = torch.stack(rows).float().reshape(-1, 1, 128)
    n = x.shape[0]
    buf = torch.zeros(2, n, 129, device=cuda_dev)
    key = buf[0, :, 1:].unflatten(1, (1, 128)) if layout == "odd" else buf.new_empty(n, 1, 128)
    key.copy_(x)
    slots = torch.arange(n, dtype=torch.int32).cuda()
    caches = ref.empty_cache(2, 1, 16, 128, 4, cuda_dev)
    want = ref.stored(caches, x.double(), x.double(), slots)
    if turned:  # the rows with NaN and infinities spread them over their pairs
        keep = torch.isfinite(x).all(-1)[:, 0]
        key, slots, n = key[keep.cuda()], slots[keep.cuda()], int(keep.sum())
        want = ref.stored(caches, x[keep].double(), x[keep].double(), slots)
        pos = torch.zeros(n, dtype=torch.int32, device=cuda_dev)
        pkv.pkv_rope_store_kvcache_int4(key, key, key, pos, pkv.pkv_rope_frequencies(128), *caches, slots)
    else:
        pkv.pkv_store_kvcache_int4(key, key, *caches, slots)
    _same(caches, want)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("H,d,bs", [(2, 128, 16), (1, 32, 16), (8, 64, 256), (3, 96, 48), (4, 256, 32)])
def test_load(pkv, cuda_dev, dtype, H, d, bs):
    nb = 20
    caches = ref.empty_cache(nb, H, bs, d, 8, cuda_dev)
    g = torch.Generator().manual_seed(1)
    slots = torch.randint(0, nb * bs, (211,), generator=g, dtype=torch.int32)  # with repeats
    slots[7:19] = -1
    got = pkv.pkv_load_kvcache_int4(*caches, slots.cuda(), dtype)
    for x, c, s in zip(got, caches[:2], caches[2:]):
        want = ref.token_major(c, s).flatten(0, 1)[slots.long().clamp(min=0)]
        want[slots < 0] = 0
        assert torch.equal(x.cpu(), want.to(dtype))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_load_under_any_scales(pkv, cuda_dev, dtype):
    """Scales of all eleven bits, subnormal ones and infinities among them: one rounding of the product."""
    caches = list(ref.empty_cache(8, 3, 16, 64, 9))
    g = torch.Generator().manual_seed(2)
    caches[2] = torch.randint(0, 0x7c01, caches[2].shape, generator=g).to(torch.int16).view(F16)
    caches[3][5, 1, 7, 0] = 1.0 + 2.0 ** -10  # alone among scales of eight bits
    slots = torch.arange(8 * 16, dtype=torch.int32)
    got = pkv.pkv_load_kvcache_int4(*[c.cuda() for c in caches], slots.cuda(), dtype)
    for x, c, s in zip(got, caches[:2], caches[2:]):
        want = ref.token_major(c, s).flatten(0, 1).float().to(dtype)  # (the product is exact in float32)
        assert torch.equal(x.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


def test_load_more_tokens_than_a_grid_holds(pkv, cuda_dev):
    caches = ref.empty_cache(30, 1, 16, 32, 10, cuda_dev)
    n = 2 ** 22 + 77
    slots = (torch.arange(n, dtype=torch.int64, device=cuda_dev) * 31 % 480).to(torch.int32)
    slots[-1] = 480
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    for x, c, s in zip(pkv.pkv_load_kvcache_int4(*caches, slots, F16, err_flag=err), caches[:2], caches[2:]):
        want = ref.token_major(c, s).flatten(0, 1).to(F16).to(cuda_dev)
        assert torch.equal(x[:-1], want[slots[:-1].long()]) and not bool(x[-1].any())
    assert int(err) == pkv.ERRBIT_SLOT_RANGE


def test_load_skips_bad_slots(pkv, cuda_dev):
    caches = ref.empty_cache(4, 2, 16, 128, 8, cuda_dev)
    slots = torch.tensor([0, 64, -1, 63, -7], dtype=torch.int32).cuda()
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    k, v = pkv.pkv_load_kvcache_int4(*caches, slots, F32, err_flag=err)
    assert int(err) == pkv.ERRBIT_SLOT_RANGE
    want = ref.token_major(caches[0], caches[2]).flatten(0, 1).float()
    assert torch.equal(k[[0, 3]].cpu(), want[[0, 63]]) and not bool(k[[1, 2, 4]].any()) and not bool(v[[1, 2, 4]].any())


def test_store_then_load_across_32_bits(pkv, cuda_dev):
    nb, H, bs, d = 20000, 8, 256, 128  # 2.6e9 bytes of codes
    kc = torch.zeros(nb, H, bs, d // 2, dtype=torch.uint8, device=cuda_dev)
    ks = torch.zeros(nb, H, bs, d // 32, dtype=F16, device=cuda_dev)
    caches = (kc, kc.clone(), ks, ks.clone())
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, H, d, generator=g).to(BF16)
    slots = torch.tensor([0, nb * bs - 1, 2 ** 21, 2 ** 22 + 5, 4_200_000, 77], dtype=torch.int32)
    pkv.pkv_store_kvcache_int4(x.cuda(), -x.cuda(), *caches, slots.cuda())
    k, v = pkv.pkv_load_kvcache_int4(*caches, slots.cuda(), F32)
    s = ref.scales(x.double())
    want = ref.codes(x.double(), s) * s.double().repeat_interleave(32, -1)
    assert torch.equal(k.cpu().double(), want) and torch.equal(v.cpu().double(), -want)


def test_no_tokens(pkv, cuda_dev):
    caches = ref.empty_cache(4, 2, 16, 128, 8, cuda_dev)
    none = torch.empty(0, dtype=torch.int32, device=cuda_dev)
    x = torch.empty(0, 2, 128, dtype=F16, device=cuda_dev)
    before = [c.clone() for c in caches]
    out = pkv.pkv_rope_store_kvcache_int4(x, x, x, none, pkv.pkv_rope_frequencies(128), *caches, none)
    pkv.pkv_store_kvcache_int4(x, x, *caches, none)
    assert out.shape == (0, 2, 128) and pkv.pkv_load_kvcache_int4(*caches, none)[0].shape == (0, 2, 128)
    assert all(torch.equal(a, b) for a, b in zip(caches, before))
