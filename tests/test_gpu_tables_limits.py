"""Growth of block tables at its limits: no sequences, lengths and sizes near 2^31."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nb", [0, 10, 300000])
@pytest.mark.parametrize("cap", [0, 5, 20000])
def test_grow_of_no_sequences(pkv, cuda_dev, nb, cap):
    """An empty batch: the offset 0, and a slot map of -1 that a store skips."""
    i32 = lambda v, *shape: torch.full(shape, v, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    none, ref, cu, slots = i32(0, 0), i32(0, nb), i32(7, 1), i32(5, cap)
    err = i32(0, 1)
    got = pkv.pkv_grow_block_tables(i32(0, 0, 6), none, none, ref, 16, num_new_tokens=cap, cu_new=cu, out=slots, err_flag=err)
    assert got[0] is cu and got[1] is slots
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for cu, slots in (got, pkv.pkv_grow_block_tables(i32(0, 0, 6), none, none, ref, 16, num_new_tokens=cap),
                      pkv.pkv_grow_block_tables(i32(0, 0, 6), none, none, ref, 16, num_new_tokens=cap, stream=side)):
        torch.cuda.synchronize()
        assert cu.tolist() == [0] and slots.numel() == cap and bool((slots == -1).all())
    assert int(err.item()) == 0 and not bool(ref.any())


@pytest.mark.parametrize("B", [1, 2000])
def test_grow_with_blocks_near_2_31_positions(pkv, cuda_dev, B):
    """One block of 2^31 - 1 positions: the last block of the pool's numbering space."""
    bs = 2 ** 31 - 1
    t = torch.full((B, 1), -1, dtype=torch.int32, device=cuda_dev)
    starts = torch.zeros(B, dtype=torch.int32, device=cuda_dev)
    ends = torch.zeros(B, dtype=torch.int32, device=cuda_dev)
    ends[B // 2] = 5
    ref = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    cu, slots = pkv.pkv_grow_block_tables(t, starts, ends, ref, bs, num_new_tokens=8, err_flag=err)
    assert slots.tolist() == [0, 1, 2, 3, 4, -1, -1, -1] and int(cu[-1]) == 5 and int(cu[B // 2]) == 0
    assert ref.tolist() == [1] and int(t[B // 2]) == 0 and int((t == -1).sum()) == B - 1
    again = pkv.pkv_grow_block_tables(t, ends, (ends + 2 * (ends > 0)).int(), ref, bs, num_new_tokens=3, err_flag=err)
    assert again[1].tolist() == [5, 6, -1] and int(err.item()) == 0
    t2, two = torch.full((B, 3), -1, dtype=torch.int32, device=cuda_dev), torch.zeros(2, dtype=torch.int32, device=cuda_dev)
    cu, slots = pkv.pkv_grow_block_tables(t2, starts, ends, two, 2 ** 30 - 1, num_new_tokens=20000, err_flag=err)
    assert slots[:5].tolist() == [0, 1, 2, 3, 4] and bool((slots[5:] == -1).all()) and two.tolist() == [1, 0]


@pytest.mark.parametrize("B", [3, 2000])
def test_grow_lengths_that_span_2_32(pkv, cuda_dev, B):
    """Garbage lengths, each span as long as 32 bits allow: no slots, the tables as they were, at once."""
    t = torch.full((B, 4), 3, dtype=torch.int32, device=cuda_dev)
    starts = torch.full((B,), -2 ** 31, dtype=torch.int32, device=cuda_dev)
    ends = torch.full((B,), 2 ** 31 - 1, dtype=torch.int32, device=cuda_dev)
    ref = torch.zeros(9, dtype=torch.int32, device=cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    cu, slots = pkv.pkv_grow_block_tables(t, starts, ends, ref, 16, num_new_tokens=1000, err_flag=err)
    assert cu.tolist() == [0] + [2 ** 31 - 1] * B and bool((slots == -1).all())
    assert bool((t == 3).all()) and not bool(ref.any())
    assert int(err.item()) == pkv.ERRBIT_CONTEXT | pkv.ERRBIT_SPAN
