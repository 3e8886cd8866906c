"""Block tables and slot maps grown and shrunk on the GPU: exact equality with a
plain-Python model of the rule, and with the host allocator."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


def _cdiv(a, b):
    return -(-a // b)


def _model_grow(tables, starts, ends, ref, bs, cap):
    """(cu, slots, error bits); tables and ref (lists) change in place."""
    from pagedattention_decode_pkv_gb300 import ERRBIT_BLOCK_RANGE, ERRBIT_CONTEXT, ERRBIT_NO_BLOCKS, ERRBIT_SPAN

    free = [i for i, c in enumerate(ref) if c == 0]
    used, bits, cu, slots = 0, 0, [0], [-1] * cap
    want = 0
    for b, (s, e) in enumerate(zip(starts, ends)):
        count = max(0, e - s)
        row = tables[b]
        mapped = [-1] * count
        held, grown = _cdiv(s, bs), _cdiv(e, bs)
        if s < 0 or e < s or grown > len(row):
            bits |= ERRBIT_CONTEXT
        else:
            want += grown - held
            if grown == held or want <= len(free):
                if count and s < held * bs and not 0 <= row[s // bs] < len(ref):
                    bits |= ERRBIT_BLOCK_RANGE
                for j in range(held, grown):
                    row[j] = free[used]
                    ref[free[used]] = 1
                    used += 1
                mapped = [row[p // bs] * bs + p % bs if 0 <= row[p // bs] < len(ref) else -1 for p in range(s, e)]
            else:
                bits |= ERRBIT_NO_BLOCKS
                for j in range(held, grown):
                    row[j] = -1
        for i, x in enumerate(mapped):
            if cu[-1] + i < cap:
                slots[cu[-1] + i] = x
        if cu[-1] + count > cap:
            bits |= ERRBIT_SPAN
        cu.append(cu[-1] + count)
    return cu, slots, bits


def _grow(pkv, dev, tables, starts, ends, ref, bs, cap):
    t = torch.tensor(tables, dtype=torch.int32, device=dev)
    r = torch.tensor(ref, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    cu, slots = pkv.pkv_grow_block_tables(t, torch.tensor(starts, dtype=torch.int32, device=dev),
                                          torch.tensor(ends, dtype=torch.int32, device=dev), r, bs,
                                          num_new_tokens=cap, err_flag=err)
    return t.tolist(), r.tolist(), cu.tolist(), slots.tolist(), int(err.item())


def _state(rng, B, bs, nb, max_new, width, shared=False):
    """A pool with some blocks held by this batch and some by others."""
    ids = list(range(nb))
    rng.shuffle(ids)
    ref, tables, starts, ends = [0] * nb, [], [], []
    for _ in range(B):
        s = rng.randint(0, width * bs - max_new)
        row = [-1] * width
        for j in range(_cdiv(s, bs)):
            if not ids:
                s = min(s, j * bs)
                break
            row[j] = ids.pop()
            ref[row[j]] = 1
        tables.append(row)
        starts.append(s)
        ends.append(s + rng.randint(0, max_new))
    for i in ids[::3]:
        ref[i] = 2
    return tables, starts, ends, ref


@pytest.mark.parametrize("B,bs,nb,max_new,width", [
    (1, 1, 1, 1, 1), (1, 16, 7, 60, 6), (3, 4, 40, 9, 8), (64, 16, 20000, 1, 40), (65, 16, 1500, 300, 40),
    (513, 256, 4096, 700, 6), (700, 16, 9001, 33, 5), (17, 48, 300000, 2000, 90), (4500, 32, 30000, 40, 4),
    (2048, 16, 20000, 70, 7), (30, 16, 262144, 3000, 200), (9, 3, 1025, 500, 190)])
def test_grow_matches_model(pkv, cuda_dev, B, bs, nb, max_new, width):
    rng = random.Random(B + bs + nb)
    tables, starts, ends, ref = _state(rng, B, bs, nb, max_new, width)
    total = sum(e - s for s, e in zip(starts, ends))
    for cap in (total, total + 1000, total // 2):
        got = _grow(pkv, cuda_dev, tables, starts, ends, ref, bs, cap)
        t, r = [list(x) for x in tables], list(ref)
        cu, slots, bits = _model_grow(t, starts, ends, r, bs, cap)
        assert got == (t, r, cu, slots, bits)


@pytest.mark.parametrize("times", [20, 300])
@pytest.mark.parametrize("nb", [0, 1, 5, 12, 30, 600, 1100, 5000])
def test_grow_when_blocks_run_out(pkv, cuda_dev, nb, times):
    """Sequences are served in order until one does not fit; later ones that need no block still are."""
    bs = 4
    starts = [0, 3, 8, 2, 0, 5, 0] * times
    ends = [9, 20, 9, 4, 11, 8, 30] * times
    tables = [[0 if j < _cdiv(s, bs) and nb else -1 for j in range(8)] for s in starts]
    ref = [1 if i % 3 == 0 else 0 for i in range(nb)]
    cap = sum(e - s for s, e in zip(starts, ends))
    got = _grow(pkv, cuda_dev, tables, starts, ends, ref, bs, cap)
    t, r = [list(x) for x in tables], list(ref)
    cu, slots, bits = _model_grow(t, starts, ends, r, bs, cap)
    assert got == (t, r, cu, slots, bits)


def test_grow_bad_lengths(pkv, cuda_dev):
    starts, ends = [0, -3, 10, 4, 6, 0], [5, 4, 7, 4 * 6 + 1, 8, 24]
    tables = [[-1] * 6 for _ in starts]
    tables[4][1] = 99  # sequence 4 continues in a block that does not exist
    ref = [0] * 12
    cap = sum(max(0, e - s) for s, e in zip(starts, ends))
    got = _grow(pkv, cuda_dev, tables, starts, ends, ref, 4, cap)
    t, r = [list(x) for x in tables], list(ref)
    cu, slots, bits = _model_grow(t, starts, ends, r, 4, cap)
    assert bits == pkv.ERRBIT_CONTEXT | pkv.ERRBIT_BLOCK_RANGE
    assert got == (t, r, cu, slots, bits)


@pytest.mark.parametrize("B,bs,nb,max_new,width", [(3, 4, 60, 9, 8), (64, 16, 5000, 100, 40), (700, 16, 9001, 33, 5)])
def test_shrink_undoes_grow(pkv, cuda_dev, B, bs, nb, max_new, width):
    rng = random.Random(B)
    tables, starts, ends, ref = _state(rng, B, bs, nb, max_new, width)
    t = torch.tensor(tables, dtype=torch.int32, device=cuda_dev)
    r = torch.tensor(ref, dtype=torch.int32, device=cuda_dev)
    s = torch.tensor(starts, dtype=torch.int32, device=cuda_dev)
    e = torch.tensor(ends, dtype=torch.int32, device=cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    cap = sum(y - x for x, y in zip(starts, ends))
    first = pkv.pkv_grow_block_tables(t, s, e, r, bs, num_new_tokens=cap, err_flag=err)
    grown = t.tolist()
    pkv.pkv_shrink_block_tables(t, s, e, r, bs, err_flag=err)
    assert t.tolist() == tables and r.tolist() == ref
    again = pkv.pkv_grow_block_tables(t, s, e, r, bs, num_new_tokens=cap, err_flag=err)
    assert t.tolist() == grown and all(torch.equal(a, b) for a, b in zip(first, again))
    # releasing everything frees this batch's blocks and no others
    pkv.pkv_shrink_block_tables(t, torch.zeros_like(s), e, r, bs, err_flag=err)
    mine = {x for row in grown for x in row if x >= 0}
    want = [0 if i in mine else c for i, c in enumerate(ref)]
    assert r.tolist() == want and int(t.max()) == -1
    assert int(err.item()) & ~pkv.ERRBIT_NO_BLOCKS == 0


def test_shrink_errors(pkv, cuda_dev):
    """Shared blocks keep a count; unreferenced, bad and missing entries are reported or skipped."""
    bs = 4
    t = torch.tensor([[0, 1, 2], [0, 1, -1], [3, 77, -1], [4, 4, 4], [5, 6, 7]], dtype=torch.int32, device=cuda_dev)
    r = torch.tensor([2, 2, 1, 0, 2, 1, 1, 1], dtype=torch.int32, device=cuda_dev)
    keeps = torch.tensor([0, 4, 0, 0, 9], dtype=torch.int32, device=cuda_dev)
    lens = torch.tensor([12, 12, 8, 12, 5], dtype=torch.int32, device=cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    pkv.pkv_shrink_block_tables(t, keeps, lens, r, bs, err_flag=err)
    assert t.tolist() == [[-1] * 3, [0, -1, -1], [-1] * 3, [-1] * 3, [5, 6, 7]]
    assert r.tolist() == [1, 0, 0, 0, 0, 1, 1, 1]
    assert int(err.item()) == pkv.ERRBIT_BLOCK_RANGE | pkv.ERRBIT_REF_COUNT | pkv.ERRBIT_CONTEXT


def test_grow_follows_the_host_allocator(pkv, cuda_dev):
    """Random admits, growth and releases: the tables and slots of both allocators agree step by step."""
    rng = random.Random(5)
    bs, nb, width, B = 8, 200, 20, 12
    host = pkv.pkv_allocator_create(nb, bs)
    t = torch.full((B, width), -1, dtype=torch.int32, device=cuda_dev)
    r = torch.zeros(nb, dtype=torch.int32, device=cuda_dev)
    lens = [0] * B
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    for _ in range(40):
        if any(lens) and rng.random() < 0.3:  # a sequence ends
            b = rng.choice([i for i in range(B) if lens[i]])
            pkv.pkv_allocator_release(host, b)
            keep = [0 if i == b else n for i, n in enumerate(lens)]
            pkv.pkv_shrink_block_tables(t, torch.tensor(keep, dtype=torch.int32, device=cuda_dev),
                                        torch.tensor(lens, dtype=torch.int32, device=cuda_dev), r, bs, err_flag=err)
            lens = keep
        ends = [min(n + rng.randint(0, 12), width * bs) for n in lens]
        if sum(_cdiv(e, bs) for e in ends) > nb:
            continue
        want = []
        for b, (s, e) in enumerate(zip(lens, ends)):
            if s == 0 and e > 0:
                pkv.pkv_allocator_add_sequence(host, b, 0)
            want += pkv.pkv_allocator_append(host, b, e - s) if e > s else []
        _, slots = pkv.pkv_grow_block_tables(t, torch.tensor(lens, dtype=torch.int32, device=cuda_dev),
                                             torch.tensor(ends, dtype=torch.int32, device=cuda_dev), r, bs,
                                             num_new_tokens=len(want), err_flag=err)
        assert slots.tolist() == want
        lens = ends
        for b in range(B):
            if lens[b]:
                row, _, used = pkv.pkv_allocator_block_table(host, b, width)
                assert t[b, :used].tolist() == row[:used]
    assert int(err.item()) == 0


def test_grow_in_a_graph(pkv, cuda_dev):
    """One captured step replayed: every replay continues from the lengths the last one left."""
    bs, nb, B = 4, 64, 5
    t = torch.full((B, 10), -1, dtype=torch.int32, device=cuda_dev)
    r = torch.zeros(nb, dtype=torch.int32, device=cuda_dev)
    lens = torch.tensor([0, 1, 2, 3, 0], dtype=torch.int32, device=cuda_dev)
    start = torch.zeros_like(lens)
    pkv.pkv_grow_block_tables(t, start, lens, r, bs, num_new_tokens=6)
    model_t, model_r, now = t.tolist(), r.tolist(), lens.tolist()
    step = torch.tensor([3, 1, 0, 2, 5], dtype=torch.int32, device=cuda_dev)
    ends, cu = torch.empty_like(lens), torch.empty(B + 1, dtype=torch.int32, device=cuda_dev)
    slots = torch.empty(16, dtype=torch.int32, device=cuda_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=cuda_dev)
    with torch.cuda.stream(side):
        torch.add(lens, step, out=ends)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        torch.add(lens, step, out=ends)
        pkv.pkv_grow_block_tables(t, lens, ends, r, bs, num_new_tokens=16, cu_new=cu, out=slots, workspace=ws)
        lens.copy_(ends)
    for _ in range(4):
        g.replay()
        nxt = [a + b for a, b in zip(now, step.tolist())]
        want_cu, want, bits = _model_grow(model_t, now, nxt, model_r, bs, 16)
        now = nxt
        assert bits == 0 and slots.tolist() == want and cu.tolist() == want_cu
        assert t.tolist() == model_t and r.tolist() == model_r


def test_grown_tables_serve_store_and_attention(pkv, orc, cuda_dev):
    """grow -> store -> prefill -> grow -> fused decode step, against the oracle on the same tables."""
    from conftest import attn_error

    torch.manual_seed(3)
    B, Hq, Hkv, d, bs, nb = 3, 8, 2, 128, 16, 40
    dt = torch.bfloat16
    kc = torch.full((nb, bs, Hkv, d), float("nan"), dtype=dt, device=cuda_dev)
    vc = kc.clone()
    t = torch.full((B, 12), -1, dtype=torch.int32, device=cuda_dev)
    r = torch.zeros(nb, dtype=torch.int32, device=cuda_dev)
    r[::2] = 1  # someone else's
    zero = torch.zeros(B, dtype=torch.int32, device=cuda_dev)
    lens = torch.tensor([37, 1, 90], dtype=torch.int32, device=cuda_dev)
    n = int(lens.sum())
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    cu, slots = pkv.pkv_grow_block_tables(t, zero, lens, r, bs, num_new_tokens=n + 5, err_flag=err)
    k, v = (torch.randn(n + 5, Hkv, d, device=cuda_dev).to(dt) for _ in range(2))
    pkv.pkv_store_kvcache(k, v, kc, vc, slots, err_flag=err)
    q = torch.randn(n, Hq, d, device=cuda_dev).to(dt)
    out = pkv.pkv_paged_attention_prefill(q, kc, vc, t, zero, cu, d ** -0.5, 90, err_flag=err)
    ref, bad = orc.paged_attention_prefill(q, kc, vc, t, zero, cu, d ** -0.5)
    assert bad == 0 and attn_error(out, ref) <= 2e-2
    pkv.pkv_grow_block_tables(t, lens, lens + 1, r, bs, num_new_tokens=B, err_flag=err)
    qd, kd, vd = (torch.randn(B, h, d, device=cuda_dev).to(dt) for h in (Hq, Hkv, Hkv))
    kr, vr = kc.clone(), vc.clone()
    out = pkv.pkv_paged_attention_decode_append(qd, kd, vd, kc, vc, t, lens + 1, d ** -0.5, 192, err_flag=err)
    rows = [int(t[b, int(lens[b]) // bs]) * bs + int(lens[b]) % bs for b in range(B)]
    kr.view(-1, Hkv, d)[rows] = kd
    vr.view(-1, Hkv, d)[rows] = vd
    ref, bad = orc.paged_attention_decode(qd, kr, vr, t, lens + 1, d ** -0.5)
    assert bad == 0 and attn_error(out, ref) <= 2e-2
    assert int(err.item()) == 0
