"""Argument checks of the table and score-rule operators: refused on the host,
before anything is enqueued (no GPU needed)."""
import ctypes

import pytest


def _p(x=1 << 20):
    return ctypes.c_void_p(x)


GROW = ["block_tables", "max_blocks", "starts", "ends", "num_seqs", "block_size", "ref_counts", "num_blocks", "cu_new",
        "slots", "num_new", "workspace", "ws_bytes", "err", "stream"]


def _grow(lib, **kw):
    a = dict(block_tables=_p(), max_blocks=4, starts=_p(), ends=_p(), num_seqs=3, block_size=16, ref_counts=_p(),
             num_blocks=10, cu_new=_p(), slots=_p(), num_new=5, workspace=_p(), ws_bytes=1 << 20, err=None,
             stream=None)
    a.update(kw)
    return lib.pkv_grow_block_tables(*[a[n] for n in GROW])


@pytest.mark.parametrize("bad,status", [
    (dict(max_blocks=-1), "INVALID_ARG"), (dict(num_seqs=-1), "INVALID_ARG"), (dict(block_size=0), "INVALID_ARG"),
    (dict(num_blocks=-1), "INVALID_ARG"), (dict(num_blocks=1 << 28), "INVALID_ARG"),
    (dict(num_new=-1), "INVALID_ARG"), (dict(num_seqs=65536), "UNSUPPORTED"), (dict(starts=None), "INVALID_ARG"),
    (dict(ends=None), "INVALID_ARG"), (dict(cu_new=None), "INVALID_ARG"), (dict(block_tables=None), "INVALID_ARG"),
    (dict(ref_counts=None), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"),
    (dict(num_blocks=40000, workspace=None), "WORKSPACE"), (dict(num_seqs=2000, ws_bytes=100), "WORKSPACE"),
    (dict(num_new=1 << 20, workspace=_p((1 << 20) + 16)), "WORKSPACE")])
def test_grow_refuses(pkv, bad, status):
    assert _grow(pkv._lib, **bad) == getattr(pkv, "PKV_ERR_" + status)
    assert b"grow" in pkv._lib.pkv_last_error_string()


def test_grow_of_nothing(pkv):
    assert _grow(pkv._lib, num_seqs=0, workspace=None, ws_bytes=0) == pkv.PKV_OK
    size = pkv._lib.pkv_grow_block_tables_workspace_size
    assert size(0, 10, 5) == 0 and size(3, 10, 5) == 0  # nothing, and one launch without a workspace
    assert min(size(2000, 10, 5), size(3, 40000, 5), size(3, 10, 1 << 20)) > 0


@pytest.mark.parametrize("bad,status", [
    (dict(max_blocks=-1), "INVALID_ARG"), (dict(num_seqs=-2), "INVALID_ARG"), (dict(block_size=-16), "INVALID_ARG"),
    (dict(num_blocks=1 << 28), "INVALID_ARG"), (dict(num_seqs=70000), "UNSUPPORTED"),
    (dict(keeps=None), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"), (dict(block_tables=None), "INVALID_ARG"),
    (dict(ref_counts=None), "INVALID_ARG")])
def test_shrink_refuses(pkv, bad, status):
    a = dict(block_tables=_p(), max_blocks=4, keeps=_p(), lens=_p(), num_seqs=3, block_size=16, ref_counts=_p(),
             num_blocks=10, err=None, stream=None)
    a.update(bad)
    order = ["block_tables", "max_blocks", "keeps", "lens", "num_seqs", "block_size", "ref_counts", "num_blocks",
             "err", "stream"]
    assert pkv._lib.pkv_shrink_block_tables(*[a[n] for n in order]) == getattr(pkv, "PKV_ERR_" + status)
    assert b"shrink" in pkv._lib.pkv_last_error_string()


def test_table_bindings_refuse_cpu_tensors(pkv):
    import torch

    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.pkv_grow_block_tables(torch.zeros(2, 3, dtype=torch.int32), i, i, torch.zeros(9, dtype=torch.int32), 16,
                                  num_new_tokens=0)
    with pytest.raises(ValueError):
        pkv.pkv_shrink_block_tables(torch.zeros(2, 3, dtype=torch.int32), i, i, torch.zeros(9, dtype=torch.int32), 16)


def _prefill(pkv, lib, **kw):
    mod = kw.pop("mod", None)
    a = dict(out=_p(), q=_p(), k=_p(), v=_p(), ks=None, vs=None, fmt=pkv.PKV_CACHE_DTYPE, tables=_p(), max_blocks=8,
             starts=_p(), cu=_p(), num_seqs=2, max_q=1000, Hq=16, Hkv=8, d=128, bs=16, nb=100, scale=0.1,
             mod=ctypes.byref(pkv._ScoreMod(*mod)) if mod else None, dtype=pkv.PKV_BF16, ws=_p(), ws_bytes=1 << 40,
             err=None, stream=None)
    a.update(kw)
    return lib.pkv_paged_attention_prefill_mod(*a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=7), "INVALID_ARG"), (dict(fmt=3), "INVALID_ARG"), (dict(num_seqs=-1), "INVALID_ARG"),
    (dict(max_q=-1), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"), (dict(Hq=12), "INVALID_ARG"),
    (dict(bs=0), "INVALID_ARG"), (dict(nb=1 << 28), "INVALID_ARG"), (dict(nb=0), "INVALID_ARG"),
    (dict(mod=(-1.0,)), "INVALID_ARG"), (dict(mod=(float("nan"),)), "INVALID_ARG"),
    (dict(mod=(float("inf"),)), "INVALID_ARG"), (dict(mod=(1e-33,)), "INVALID_ARG"), (dict(mod=(1e31,)), "INVALID_ARG"),
    (dict(num_seqs=65536), "UNSUPPORTED"), (dict(d=64), "UNSUPPORTED"),
    (dict(Hq=24), "UNSUPPORTED"), (dict(Hq=128), "UNSUPPORTED"), (dict(bs=24), "UNSUPPORTED"), (dict(dtype=0), "UNSUPPORTED"),
    (dict(out=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"),
    (dict(v=None), "INVALID_ARG"), (dict(tables=None), "INVALID_ARG"), (dict(starts=None), "INVALID_ARG"),
    (dict(cu=None), "INVALID_ARG"), (dict(q=_p((1 << 20) + 8)), "UNSUPPORTED"), (dict(k=_p((1 << 20) + 8)), "UNSUPPORTED"),
    (dict(fmt=1), "INVALID_ARG"), (dict(fmt=2, ks=_p()), "INVALID_ARG"),
    (dict(fmt=1, ks=_p(), vs=_p((1 << 20) + 2)), "INVALID_ARG"),
    (dict(max_q=20, max_blocks=800, ws=None), "WORKSPACE"), (dict(max_q=20, max_blocks=800, ws_bytes=64), "WORKSPACE"),
    (dict(max_q=20, max_blocks=800, ws=_p((1 << 20) + 16)), "WORKSPACE")])
def test_prefill_mod_refuses(pkv, bad, status):
    assert _prefill(pkv, pkv._lib, **bad) == getattr(pkv, "PKV_ERR_" + status)
    assert b"prefill" in pkv._lib.pkv_last_error_string()


def test_prefill_mod_of_nothing(pkv):
    assert _prefill(pkv, pkv._lib, num_seqs=0) == pkv.PKV_OK
    assert _prefill(pkv, pkv._lib, max_q=0) == pkv.PKV_OK


def test_prefill_mod_workspace(pkv):
    size = pkv.pkv_paged_attention_prefill_mod_workspace_size
    assert size(2, 16, 8, 128, 16, 20, 800) > 0      # few rows, long tables: split
    assert size(64, 16, 8, 128, 16, 4096, 800) == 0  # many CTAs
    assert size(2, 16, 8, 128, 16, 20, 8) == 0       # one block of keys
    assert size(0, 16, 8, 128, 16, 20, 800) == size(2, 16, 8, 64, 16, 20, 800) == 0


def _decode(pkv, lib, **kw):
    mod = kw.pop("mod", None)
    a = dict(out=_p(), q=_p(), key=None, value=None, k=_p(), v=_p(), ks=None, vs=None, fmt=pkv.PKV_CACHE_DTYPE,
             tables=_p(), max_blocks=8, ctx=_p(), num_seqs=2, Hq=16, Hkv=8, d=128, bs=16, nb=100, max_ctx=100,
             scale=0.1, mod=ctypes.byref(pkv._ScoreMod(*mod)) if mod else None, dtype=pkv.PKV_BF16, ws=_p(),
             ws_bytes=1 << 40, err=None, stream=None)
    a.update(kw)
    return lib.pkv_paged_attention_decode_mod(*a.values())


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=7), "INVALID_ARG"), (dict(fmt=-1), "INVALID_ARG"), (dict(num_seqs=-1), "INVALID_ARG"),
    (dict(Hq=12), "INVALID_ARG"), (dict(max_ctx=-1), "INVALID_ARG"), (dict(nb=1 << 28), "INVALID_ARG"),
    (dict(mod=(-0.5,)), "INVALID_ARG"), (dict(mod=(float("nan"),)), "INVALID_ARG"),
    (dict(mod=(float("inf"),)), "INVALID_ARG"), (dict(mod=(1e-33,)), "INVALID_ARG"), (dict(mod=(1e31,)), "INVALID_ARG"),
    (dict(key=_p()), "INVALID_ARG"), (dict(value=_p()), "INVALID_ARG"),
    (dict(out=None), "INVALID_ARG"), (dict(ctx=None), "INVALID_ARG"), (dict(fmt=1), "INVALID_ARG"),
    (dict(fmt=1, ks=_p(), vs=_p(), dtype=0), "UNSUPPORTED"), (dict(fmt=2, ks=_p(), vs=_p(), d=64), "UNSUPPORTED"),
    (dict(num_seqs=65536), "UNSUPPORTED"), (dict(d=2048), "UNSUPPORTED"), (dict(ws=None), "WORKSPACE"),
    (dict(ws_bytes=10), "WORKSPACE")])
def test_decode_mod_refuses(pkv, bad, status):
    assert _decode(pkv, pkv._lib, **bad) == getattr(pkv, "PKV_ERR_" + status)
    assert b"decode" in pkv._lib.pkv_last_error_string()


def test_decode_mod_of_nothing(pkv):
    assert _decode(pkv, pkv._lib, num_seqs=0) == pkv.PKV_OK
