"""Argument checks of the rotary and 4-bit cache operators: refused on the host, before anything
is enqueued (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import int4_reference as ref


def _p(x=1 << 20):
    return ctypes.c_void_p(x)


NAN, INF = float("nan"), float("inf")
ROPE = ["q_out", "q", "q_stride", "key", "key_stride", "value", "value_stride", "positions", "rope", "k_cache", "v_cache"]
SIZES = ["slots", "num_tokens", "Hq", "Hkv", "d"]


def _rope_struct(pkv, turns=1 << 20, amplitude=1.0, rotary_dim=64, interleaved=0):
    return ctypes.byref(pkv._Rope(turns, amplitude, rotary_dim, interleaved))


def _store(pkv, int4, rope=None, **kw):
    d = kw.get("d", 128)
    a = dict(q_out=_p(), q=_p(), q_stride=8 * d, key=_p(), key_stride=2 * d, value=_p(), value_stride=2 * d, positions=_p(),
             rope=_rope_struct(pkv, **(rope or {})), k_cache=_p(), v_cache=_p(), k_scale=_p(), v_scale=_p(), slots=_p(),
             num_tokens=3, Hq=8, Hkv=2, d=d, bs=16, num_blocks=10, num_slots=160, dtype=pkv.PKV_BF16, err=None, stream=None)
    a.update(kw)
    order = ROPE + (["k_scale", "v_scale"] if int4 else []) + SIZES + (["bs", "num_blocks"] if int4 else ["num_slots"]) + \
        ["dtype", "err", "stream"]
    fn = pkv._lib.pkv_rope_store_kvcache_int4 if int4 else pkv._lib.pkv_rope_store_kvcache
    return fn(*[a[n] for n in order])


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("bad,rope,status", [
    (dict(dtype=7), {}, "INVALID_ARG"), (dict(num_tokens=-1), {}, "INVALID_ARG"), (dict(Hq=-1), {}, "INVALID_ARG"),
    (dict(Hkv=0), {}, "INVALID_ARG"), (dict(d=0), {}, "INVALID_ARG"), (dict(q_stride=1023), {}, "INVALID_ARG"),
    (dict(key_stride=255), {}, "INVALID_ARG"), (dict(value_stride=0), {}, "INVALID_ARG"),
    (dict(q=None), {}, "INVALID_ARG"), (dict(q_out=None), {}, "INVALID_ARG"), (dict(key=None), {}, "INVALID_ARG"),
    (dict(value=None), {}, "INVALID_ARG"), (dict(positions=None), {}, "INVALID_ARG"), (dict(k_cache=None), {}, "INVALID_ARG"),
    (dict(v_cache=None), {}, "INVALID_ARG"), (dict(slots=None), {}, "INVALID_ARG"), (dict(key=_p((1 << 20) + 1)), {}, "INVALID_ARG"),
    (dict(slots=_p((1 << 20) + 2)), {}, "INVALID_ARG"), (dict(q_stride=2048, q_out=_p(), q=_p()), {}, "INVALID_ARG"),  # in place, strided
    ({}, dict(rotary_dim=-2), "INVALID_ARG"), ({}, dict(rotary_dim=7), "INVALID_ARG"), ({}, dict(rotary_dim=130), "INVALID_ARG"),
    ({}, dict(interleaved=2), "INVALID_ARG"), ({}, dict(amplitude=NAN), "INVALID_ARG"), ({}, dict(amplitude=INF), "INVALID_ARG"),
    ({}, dict(turns=None), "INVALID_ARG"), ({}, dict(turns=(1 << 20) + 4), "INVALID_ARG"),
    (dict(d=1056, q_stride=1 << 20, key_stride=1 << 20, value_stride=1 << 20), {}, "UNSUPPORTED")])
def test_rope_store_refuses(pkv, int4, bad, rope, status):
    assert _store(pkv, int4, rope, **bad) == getattr(pkv, "PKV_ERR_" + status)
    assert pkv._lib.pkv_last_error_string()


@pytest.mark.parametrize("bad,status", [
    (dict(bs=0), "INVALID_ARG"), (dict(num_blocks=-1), "INVALID_ARG"), (dict(num_blocks=1 << 28), "INVALID_ARG"),
    (dict(k_scale=None), "INVALID_ARG"), (dict(v_scale=_p((1 << 20) + 1)), "INVALID_ARG"), (dict(k_cache=_p((1 << 20) + 2)), "INVALID_ARG"),
    (dict(d=80), "UNSUPPORTED")])
def test_int4_store_refuses(pkv, bad, status):
    assert _store(pkv, True, **bad) == getattr(pkv, "PKV_ERR_" + status)


def test_nothing_to_store(pkv):
    for int4 in (False, True):
        assert _store(pkv, int4, num_tokens=0, key=None, q=None) == pkv.PKV_OK


LOAD = ["key", "value", "k_cache", "v_cache", "k_scale", "v_scale", "slots", "num_tokens", "Hkv", "d", "bs", "num_blocks", "dtype",
        "err", "stream"]


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=9), "INVALID_ARG"), (dict(num_tokens=-1), "INVALID_ARG"), (dict(Hkv=0), "INVALID_ARG"), (dict(d=-32), "INVALID_ARG"),
    (dict(bs=0), "INVALID_ARG"), (dict(num_blocks=1 << 28), "INVALID_ARG"), (dict(d=48), "UNSUPPORTED"),
    (dict(key=None), "INVALID_ARG"), (dict(value=_p((1 << 20) + 8)), "INVALID_ARG"), (dict(k_cache=None), "INVALID_ARG"),
    (dict(v_cache=_p((1 << 20) + 2)), "INVALID_ARG"), (dict(k_scale=None), "INVALID_ARG"), (dict(v_scale=None), "INVALID_ARG"),
    (dict(slots=None), "INVALID_ARG")])
def test_load_refuses(pkv, bad, status):
    a = dict(key=_p(), value=_p(), k_cache=_p(), v_cache=_p(), k_scale=_p(), v_scale=_p(), slots=_p(), num_tokens=5, Hkv=2, d=128,
             bs=16, num_blocks=10, dtype=pkv.PKV_F16, err=None, stream=None)
    a.update(bad)
    assert pkv._lib.pkv_load_kvcache_int4(*[a[n] for n in LOAD]) == getattr(pkv, "PKV_ERR_" + status)
    a.update(num_tokens=0, dtype=pkv.PKV_F16, **{k: v for k, v in dict(d=128, Hkv=2, bs=16, num_blocks=10).items()})
    assert pkv._lib.pkv_load_kvcache_int4(*[a[n] for n in LOAD]) == pkv.PKV_OK


DECODE = ["out", "q", "k_cache", "v_cache", "k_scale", "v_scale", "tables", "max_blocks", "lens", "B", "Hq", "Hkv", "d", "bs",
          "num_blocks", "max_ctx", "scale", "mod", "dtype", "ws", "ws_bytes", "err", "stream"]
PREFILL = ["out", "q", "k_cache", "v_cache", "k_scale", "v_scale", "tables", "max_blocks", "starts", "cu", "B", "max_q", "max_total",
           "Hq", "Hkv", "d", "bs", "num_blocks", "scale", "mod", "dtype", "ws", "ws_bytes", "err", "stream"]


def _attention(pkv, which, **kw):
    a = dict(out=_p(), q=_p(), k_cache=_p(), v_cache=_p(), k_scale=_p(), v_scale=_p(), tables=_p(), max_blocks=200, lens=_p(),
             starts=_p(), cu=_p(), B=2, max_q=64, max_total=0, Hq=8, Hkv=2, d=128, bs=16, num_blocks=500, max_ctx=3000, scale=0.1, mod=None,
             dtype=pkv.PKV_BF16, ws=_p(), ws_bytes=1 << 30, err=None, stream=None)
    cap = kw.pop("softcap", None)
    if cap is not None:
        a["mod"] = ctypes.byref(pkv._ScoreMod(cap, None, None, None))
    a.update(kw)
    fn = pkv._lib.pkv_paged_attention_decode_int4 if which == "decode" else pkv._lib.pkv_paged_attention_prefill_int4
    return fn(*[a[n] for n in (DECODE if which == "decode" else PREFILL)])


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), "INVALID_ARG"), (dict(B=-1), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"), (dict(Hkv=3), "INVALID_ARG"),
    (dict(bs=0), "INVALID_ARG"), (dict(num_blocks=1 << 28), "INVALID_ARG"), (dict(softcap=-1.0), "INVALID_ARG"),
    (dict(softcap=NAN), "INVALID_ARG"), (dict(softcap=1e-35), "INVALID_ARG"), (dict(dtype=0), "UNSUPPORTED"), (dict(d=96), "UNSUPPORTED"),
    (dict(bs=24), "UNSUPPORTED"), (dict(out=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(k_cache=None), "INVALID_ARG"),
    (dict(v_scale=None), "INVALID_ARG"), (dict(tables=None), "INVALID_ARG"), (dict(num_blocks=0), "INVALID_ARG"),
    (dict(q=_p((1 << 20) + 2)), "UNSUPPORTED"), (dict(k_cache=_p((1 << 20) + 8)), "UNSUPPORTED"),
    (dict(k_scale=_p((1 << 20) + 8)), "UNSUPPORTED"), (dict(ws=None), "WORKSPACE"), (dict(ws_bytes=100), "WORKSPACE"),
    (dict(ws=_p((1 << 20) + 16)), "WORKSPACE")])
def test_attention_refuses(pkv, which, bad, status):
    assert _attention(pkv, which, **bad) == getattr(pkv, "PKV_ERR_" + status)


@pytest.mark.parametrize("which,bad,status", [
    ("decode", dict(max_ctx=-1), "INVALID_ARG"), ("decode", dict(max_ctx=2 ** 31 - 10), "INVALID_ARG"),
    ("decode", dict(lens=None), "INVALID_ARG"), ("prefill", dict(starts=None), "INVALID_ARG"), ("prefill", dict(cu=None), "INVALID_ARG"),
    ("prefill", dict(max_q=-1), "INVALID_ARG"), ("prefill", dict(max_total=-1), "INVALID_ARG"), ("prefill", dict(Hq=6), "UNSUPPORTED"), ("prefill", dict(d=64), "UNSUPPORTED"),
    ("prefill", dict(B=70000), "UNSUPPORTED"),
    # too many tiles for a grid: refused before the blocks are widened into the workspace
    ("prefill", dict(B=600, max_q=2 ** 31 - 1, max_total=16, Hkv=1), "UNSUPPORTED")])
def test_one_attention_refuses(pkv, which, bad, status):
    assert _attention(pkv, which, **bad) == getattr(pkv, "PKV_ERR_" + status)


def test_empty_batches(pkv):
    assert _attention(pkv, "decode", B=0, q=None) == pkv.PKV_OK
    assert _attention(pkv, "prefill", B=0, q=None) == pkv.PKV_OK
    assert _attention(pkv, "prefill", max_q=0, q=None) == pkv.PKV_OK


def test_prefill_workspace(pkv):
    size, mod = pkv.pkv_paged_attention_prefill_int4_workspace_size, pkv.pkv_paged_attention_prefill_mod_workspace_size
    assert size(8, 32, 8, 128, 16, 16, 256) == mod(8, 32, 8, 128, 16, 16, 256)  # few rows: widened as they are read
    pool = 2 * 8 * 256 * 16 * 8 * 128 * 2
    assert size(8, 32, 8, 128, 16, 4096, 256) == pool + 8 * 256 * 4
    assert size(8, 32, 8, 128, 16, 4096, 256, 2048) == pool // 2 + 8 * 128 * 4  # a bound on the positions
    assert size(64, 32, 8, 128, 16, 4096, 2048) == mod(64, 32, 8, 128, 16, 4096, 2048) == 0  # too much: 8 GiB
    assert size(0, 32, 8, 128, 16, 4096, 256) == size(8, 32, 8, 64, 16, 4096, 256) == size(8, 32, 8, 128, 16, 4096, 256, -1) == 0


def test_decode_workspace(pkv):
    size = pkv.pkv_paged_attention_decode_int4_workspace_size
    assert size(4, 16, 8, 128, 500) == 0          # a CTA per unit
    assert size(4, 16, 8, 128, 5000) > 0 and size(500, 16, 8, 128, 500) > 0
    assert size(2000, 16, 8, 128, 5000) == size(512, 16, 8, 128, 5000)  # groups share it
    assert size(0, 16, 8, 128, 500) == size(4, 16, 8, 96, 5000) == size(4, 9, 8, 128, 5000) == 0


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=7), dict(rotary_dim=-2), dict(base=1.0), dict(base=NAN), dict(scaling=5), dict(scaling=1, factor=0.5),
    dict(scaling=2, factor=INF), dict(scaling=3, factor=2.0, original_len=0.0), dict(scaling=3, factor=2.0, beta_fast=1.0),
    dict(scaling=3, factor=2.0, beta_slow=-1.0), dict(turns=None), dict(amplitude=None)])
def test_frequencies_refuse(pkv, kw):
    turns, amp = torch.empty(64, dtype=torch.int64), ctypes.c_double()
    a = dict(rotary_dim=128, base=1e4, scaling=0, factor=1.0, original_len=2048.0, beta_fast=32.0, beta_slow=1.0,
             turns=ctypes.c_void_p(turns.data_ptr()), amplitude=ctypes.byref(amp))
    a.update(kw)
    assert pkv._lib.pkv_rope_frequencies(*a.values()) == pkv.PKV_ERR_INVALID_ARG


def test_frequencies_on_the_host(pkv):
    for scaling, kw in ((None, {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)), ("yarn", dict(factor=16.0, original_len=2048))):
        rope = pkv.pkv_rope_frequencies(64, scaling=scaling, device="cpu", **kw)
        freq, amp = ref.frequencies(64, scaling=scaling, **kw)
        t = (rope.turns.double() / 2.0 ** 64) % 1.0
        want = torch.tensor(freq, dtype=torch.float64) / (2 * math.pi)
        assert bool(((t - want).abs() <= 8 * 2.0 ** -53 * want + 2.0 ** -64).all()) and abs(rope.amplitude - amp) < 1e-15
    # fractions of a turn are exact, whole turns vanish, a negative frequency turns back
    quarter = pkv.pkv_rope_turns([math.pi / 2, 2 * math.pi, -math.pi / 2], device="cpu").turns.tolist()
    assert quarter == [1 << 62, 0, -(1 << 62)]
    with pytest.raises(pkv.PkvError):
        pkv.pkv_rope_turns([INF], device="cpu")
    with pytest.raises(ValueError):
        pkv.pkv_rope_frequencies(64, scaling="other", device="cpu")
    with pytest.raises(TypeError):
        pkv.RopeFrequencies(torch.zeros(4))


def test_bindings_refuse_shapes_and_cpu_tensors(pkv):
    x = torch.zeros(3, 2, 128, dtype=torch.float16)
    k, s = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16, 4, dtype=torch.float16)
    slots = torch.zeros(3, dtype=torch.int32)
    rope = pkv.pkv_rope_frequencies(128, device="cpu")
    wide = torch.zeros(4, 16, 2, 128, dtype=torch.float16)
    for call in (lambda: pkv.pkv_store_kvcache_int4(x, x, k, k, s, s, slots), lambda: pkv.pkv_load_kvcache_int4(k, k, s, s, slots),
                 lambda: pkv.pkv_rope_store_kvcache(x, x, x, slots, rope, wide, wide, slots),
                 lambda: pkv.pkv_paged_attention_decode_int4(x, k, k, s, s, slots[None], slots, 1.0, 4)):
        with pytest.raises(ValueError):  # no CPU path
            call()
    with pytest.raises(TypeError):
        pkv.pkv_store_kvcache_int4(x, x, k.to(torch.int8), k, s, s, slots)
    with pytest.raises(TypeError):
        pkv.pkv_store_kvcache_int4(x, x, k, k, s.float(), s, slots)
    with pytest.raises(TypeError):
        pkv.pkv_store_kvcache_int4(x, x.float(), k, k, s, s, slots)
    with pytest.raises(TypeError):
        pkv.pkv_rope_store_kvcache(x, x, x, slots, rope, wide.float(), wide, slots)
    with pytest.raises(ValueError):
        pkv.pkv_store_kvcache_int4(x, x, k, k, s[..., :2], s, slots)
    with pytest.raises(ValueError):
        pkv.pkv_store_kvcache_int4(x[:2], x, k, k, s, s, slots)


def test_format_reference():
    """The reference's own encoding: round trip, order of nibbles, ties, saturation."""
    x = torch.tensor([7.0, 6.5, 5.5, 0.5, -0.5, -1.5, -7.0, 0.49] * 4, dtype=torch.float64)[None]
    s = ref.scales(x)
    assert s.tolist() == [[1.0]]
    c = ref.codes(x, s)
    assert c[0, :8].tolist() == [7, 6, 6, 0, 0, -2, -7, 0]
    word = int.from_bytes(bytes(ref.pack(c)[0, :4].tolist()), "little")
    assert [word >> (4 * n) & 15 for n in range(8)] == [15, 14, 8, 1, 14, 8, 6, 8]  # dims 0 2 4 6 1 3 5 7
    assert torch.equal(ref.values(ref.pack(c), s), c)
    assert ref.scales(torch.full((1, 32), 1e9, dtype=torch.float64)).item() == 9344.0
    assert ref.scales(torch.full((1, 32), 1e-9, dtype=torch.float64)).item() == 0.0
