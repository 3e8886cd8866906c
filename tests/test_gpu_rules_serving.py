"""The table and score-rule operators as a serving loop runs them, and what such
a loop meets: long caches, other streams."""
import pytest
import torch

import score_reference as sr

pytestmark = pytest.mark.gpu

HQ, HKV, D = 8, 2, 128


def _slopes(dev):
    return torch.exp2(-torch.arange(1, HQ + 1, dtype=torch.float32)).to(dev)


@pytest.mark.parametrize("fmt", [None, "fp8", "int8"])
def test_serving_loop(pkv, cuda_dev, fmt):
    """grow -> store -> prefill in two chunks, three decode steps that append, then everything is
    given back: capped, biased scores in a window, over every cache format."""
    torch.manual_seed(5)
    dt, bs, nb, width = torch.bfloat16, 16, 60, 12
    B, scale, cap, window = 4, D ** -0.5, 30.0, 50
    rules = {"softcap": cap, "alibi_slopes": _slopes(cuda_dev)}
    if fmt is None:
        kc = torch.full((nb, bs, HKV, D), float("nan"), dtype=dt, device=cuda_dev)
        ks = vs = None
    else:
        kc = torch.full((nb, bs, HKV, D), 0x7F, dtype=torch.uint8 if fmt == "fp8" else torch.int8, device=cuda_dev)
        ks = torch.full((nb, HKV), 0.02 if fmt == "fp8" else 0.04, device=cuda_dev)
        vs = ks * 0.5
    vc = kc.clone()
    t = torch.full((B, width), -1, dtype=torch.int32, device=cuda_dev)
    ref_counts = torch.zeros(nb, dtype=torch.int32, device=cuda_dev)
    ref_counts[1::3] = 2  # someone else's
    before = ref_counts.clone()
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    rand = lambda n, h: torch.randn(n, h, D, device=cuda_dev).to(dt)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_dev)  # noqa: E731

    def reference(q, starts, ns, first):
        return sr.prefill(q, sr.dequantize(kc, ks), sr.dequantize(vc, vs), t, starts, ns, scale, cap, rules["alibi_slopes"], first)

    lens = [0] * B
    for chunk in ([37, 1, 90, 0], [20, 33, 0, 70]):
        ends = [a + n for a, n in zip(lens, chunk)]
        n = sum(chunk)
        cu, slots = pkv.pkv_grow_block_tables(t, i32(lens), i32(ends), ref_counts, bs, num_new_tokens=n, err_flag=err)
        store = pkv.pkv_store_kvcache if fmt is None else getattr(pkv, "pkv_store_kvcache_" + fmt)
        scales = () if fmt is None else (ks, vs)
        store(rand(n, HKV), rand(n, HKV), kc, vc, *scales, slots, err_flag=err)
        q = rand(n, HQ)
        first = i32([p - window + 1 for a, e in zip(lens, ends) for p in range(a, e)])
        out = pkv.pkv_paged_attention_prefill_mod(q, kc, vc, t, i32(lens), cu, scale, max(chunk), key_starts=first,
                                                  k_scale=ks, v_scale=vs, err_flag=err, **rules)
        sr.assert_within(out, reference(q, lens, chunk, first), vc, vs)
        lens = ends
    for _ in range(3):
        ends = [a + 1 for a in lens]
        pkv.pkv_grow_block_tables(t, i32(lens), i32(ends), ref_counts, bs, num_new_tokens=B, err_flag=err)
        q, key, value = rand(B, HQ), rand(B, HKV), rand(B, HKV)
        first = i32([a - window + 1 for a in lens])
        out = pkv.pkv_paged_attention_decode_mod(q, kc, vc, t, i32(ends), scale, width * bs, key=key, value=value,
                                                 key_starts=first, k_scale=ks, v_scale=vs, err_flag=err, **rules)
        sr.assert_within(out, reference(q, lens, [1] * B, first), vc, vs)
        lens = ends
    pkv.pkv_shrink_block_tables(t, i32([0] * B), i32(lens), ref_counts, bs, err_flag=err)
    assert torch.equal(ref_counts, before) and bool((t == -1).all()) and int(err.item()) == 0


@pytest.mark.parametrize("fmt", [None, "int8"])
def test_offsets_past_32_bits(pkv, cuda_dev, fmt):
    """Blocks at the end of a pool of more than 2^32 bytes."""
    bs, dt = 256, torch.bfloat16
    nb = 2 ** 32 // (bs * HKV * D * (1 if fmt else 2)) + 40
    kc, vc = (torch.empty((nb, bs, HKV, D), dtype=dt if fmt is None else torch.int8, device=cuda_dev) for _ in range(2))
    ids = torch.tensor([[nb - 1, 0, nb - 7], [nb - 30, nb - 2, 3]], dtype=torch.int32, device=cuda_dev)
    g = torch.Generator().manual_seed(1)
    for c in (kc, vc):
        for i in ids.flatten().tolist():
            x = torch.randn(bs, HKV, D, generator=g)
            c[i] = (x.to(dt) if fmt is None else (40 * x).round().clamp(-127, 127).to(torch.int8)).to(cuda_dev)
    ks = vs = None
    if fmt:
        ks = torch.rand((nb, HKV), device=cuda_dev) * 0.01 + 0.02
        vs = torch.rand((nb, HKV), device=cuda_dev) * 0.01 + 0.02
    used = ids.flatten().long()
    small = [sr.dequantize(c[used], None if s is None else s[used]) for c, s in ((kc, ks), (vc, vs))]
    where = torch.arange(6, dtype=torch.int32).view(2, 3)  # the same blocks, gathered
    q = torch.randn(100, HQ, D, generator=g).to(dt).to(cuda_dev)
    starts, ns = [600, 500], [60, 40]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    out = pkv.pkv_paged_attention_prefill_mod(q, kc, vc, ids, i32(starts), i32([0, 60, 100]), D ** -0.5, 60, softcap=20.0,
                                              k_scale=ks, v_scale=vs)
    ref = sr.prefill(q, *small, where, starts, ns, D ** -0.5, 20.0)
    codes = vc[used]
    sr.assert_within(out, ref, codes, None if vs is None else vs[used])
    out = pkv.pkv_paged_attention_decode_mod(q[:2], kc, vc, ids, i32([660, 540]), D ** -0.5, 700, softcap=20.0, k_scale=ks,
                                             v_scale=vs)
    ref = sr.prefill(q[:2], *small, where, [659, 539], [1, 1], D ** -0.5, 20.0)
    sr.assert_within(out, ref, codes, None if vs is None else vs[used])


def test_buffers_belong_to_the_stream_given(pkv, cuda_dev, monkeypatch):
    """With stream=, what a call allocates is that stream's: a workspace freed on return is not handed
    to another stream under the running kernel."""
    side = torch.cuda.Stream()
    seen = []
    plain = torch.empty

    def spy(*a, **kw):
        seen.append(torch.cuda.current_stream() == side)
        return plain(*a, **kw)

    B, bs, nb = 2, 16, 200
    t = torch.arange(nb, dtype=torch.int32, device=cuda_dev).view(B, -1).contiguous()
    kc, vc = (torch.randn(nb, bs, HKV, D, device=cuda_dev).to(torch.float16) for _ in range(2))
    q = torch.randn(4, HQ, D, device=cuda_dev).to(torch.float16)
    lens = torch.tensor([1500, 900], dtype=torch.int32, device=cuda_dev)
    cu = torch.tensor([0, 1, 4], dtype=torch.int32, device=cuda_dev)
    ref_counts, grown = torch.zeros(nb, dtype=torch.int32, device=cuda_dev), torch.full_like(t, -1)
    zero = torch.zeros_like(lens)
    args = dict(softcap=20.0)
    want = (pkv.pkv_paged_attention_prefill_mod(q, kc, vc, t, lens, cu, 0.1, 3, **args),
            pkv.pkv_paged_attention_decode_mod(q[:2], kc, vc, t, lens, 0.1, 1600, **args))
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", spy)
    got = (pkv.pkv_paged_attention_prefill_mod(q, kc, vc, t, lens, cu, 0.1, 3, stream=side, **args),
           pkv.pkv_paged_attention_decode_mod(q[:2], kc, vc, t, lens, 0.1, 1600, stream=side, **args))
    pkv.pkv_grow_block_tables(grown, zero, lens, ref_counts, bs, num_new_tokens=20000, stream=side)
    monkeypatch.undo()
    side.synchronize()
    assert len(seen) == 7 and all(seen)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_error_flag_type(pkv, cuda_dev):
    i = torch.zeros(2, dtype=torch.int32, device=cuda_dev)
    t, r = torch.full((2, 3), -1, dtype=torch.int32, device=cuda_dev), torch.zeros(9, dtype=torch.int32, device=cuda_dev)
    byte = torch.zeros(1, dtype=torch.uint8, device=cuda_dev)
    with pytest.raises(TypeError):
        pkv.pkv_grow_block_tables(t, i, i, r, 16, num_new_tokens=0, err_flag=byte)
    with pytest.raises(TypeError):
        pkv.pkv_shrink_block_tables(t, i, i, r, 16, err_flag=byte)


def test_current_stream_without_the_raw_handle(pkv, cuda_dev, monkeypatch):
    """Where torch has no raw stream handle to give, the calls still run on the current stream."""
    t, lens = torch.full((2, 3), -1, dtype=torch.int32, device=cuda_dev), torch.tensor([5, 20], dtype=torch.int32, device=cuda_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    with torch.cuda.stream(side):
        assert pkv._raw_stream(cuda_dev, None) == side.cuda_stream
        ref_counts = torch.zeros(9, dtype=torch.int32, device=cuda_dev)
        cu, _ = pkv.pkv_grow_block_tables(t, torch.zeros_like(lens), lens, ref_counts, 16, num_new_tokens=25)
    side.synchronize()
    assert cu.tolist() == [0, 5, 25] and t.tolist() == [[0, -1, -1], [1, 2, -1]]
    assert pkv._raw_stream(cuda_dev, side) == side.cuda_stream
