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
    (dict(ref_counts=None), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"), (dict(workspace=None), "WORKSPACE"),
    (dict(ws_bytes=100), "WORKSPACE"), (dict(workspace=_p((1 << 20) + 16)), "WORKSPACE")])
def test_grow_refuses(pkv, bad, status):
    assert _grow(pkv._lib, **bad) == getattr(pkv, "PKV_ERR_" + status)
    assert b"grow" in pkv._lib.pkv_last_error_string()


def test_grow_of_nothing(pkv):
    assert _grow(pkv._lib, num_seqs=0, workspace=None, ws_bytes=0) == pkv.PKV_OK
    assert pkv._lib.pkv_grow_block_tables_workspace_size(0, 10) == 0
    assert pkv._lib.pkv_grow_block_tables_workspace_size(3, 10) > 0


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
