"""The smallest and largest counts of the calls on a paged cache: nothing at all,
refused past the documented limits (on the host), right up to them (on the GPU: pair
arrays of 2^31 words)."""

import pytest
import torch

import global_attention_swa_b200 as mimo
from tests.test_paged_cpu import FAKE, UNSUPPORTED, _append, _attend, _compact, _fork, _hold, p

I32 = torch.int32


@pytest.mark.parametrize("width", [0, 1])
@pytest.mark.parametrize("rows", [2 ** 30 + 1, 2 ** 31 - 1])
def test_more_rows_than_the_kernels_count_are_refused(rows, width):
    assert _hold(seqs=rows, width=width) == UNSUPPORTED
    assert _fork(seqs=rows, width=width, to=0x7000000000) == UNSUPPORTED
    assert _fork(n=rows, width=width, table=0x7000000000, to=0x100000) == UNSUPPORTED
    assert mimo.lib.mimo_attn_page_compact(p(FAKE), 16, p(FAKE), rows, width, 4, p(FAKE), p(FAKE), p(FAKE), p(FAKE),
                                           p(FAKE), 1 << 20, None) == UNSUPPORTED


def test_more_moves_than_the_kernel_counts_are_refused():
    assert _compact(most=2 ** 30) == mimo.MIMO_ERR_INVALID_ARG


def _ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


@pytest.fixture
def big():
    """A function that makes an int32 CUDA tensor of one value, all freed at the end."""
    yield lambda shape, value: torch.full(shape, value, dtype=I32, device="cuda")
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_compact_with_room_for_the_most_moves(big):
    moves = big((2 ** 30 - 1, 2), 7)
    refs, table, got, info = mimo.mimo_attn_page_compact(_ints([0, 1, 0, 0, 2, 1]), _ints([[4, 1], [5, 4]]), 2 ** 30 - 1,
                                                         moves=moves)
    mimo.mimo_attn_device_status()
    assert got is moves and info.tolist() == [2, 3] and moves[:2].tolist() == [[4, 0], [5, 2]]
    assert refs.tolist() == [2, 1, 1, 0, 0, 0] and table.tolist() == [[0, 1], [2, 0]]
    assert (moves[2:] == -1).all()


@pytest.mark.gpu
def test_hold_of_the_most_rows(big):
    """2^30 - 1 rows of one entry.  The first and the last share a page and write into it:
    each gets a copy; one between gets its first page."""
    rows, between = 2 ** 30 - 1, 2 ** 30 - 70
    refs, table, lens = _ints([2, 1, 0, 0, 0, 0, 0]), big((rows, 1), -1), big((rows,), 0)
    for b, page, n in ((0, 0, 5), (between, -1, 16), (rows - 1, 0, 5)):
        table[b, 0], lens[b] = page, n
    moves = big((rows, 2), 7)
    _, _, _, info = mimo.mimo_attn_page_hold(refs, table, lens, 16, write_from=big((rows,), 3), refs_out=refs,
                                             table_out=table, moves=moves)
    mimo.mimo_attn_device_status()
    assert refs.tolist() == [0, 1, 1, 1, 1, 0, 0] and info.tolist() == [0, 3]
    assert [int(table[b]) for b in (0, between, rows - 1)] == [2, 3, 4] and int((table >= 0).sum()) == 3
    assert moves[0].tolist() == [0, 2] and moves[-1].tolist() == [0, 4] and (moves[1:-1] == -1).all()


@pytest.mark.gpu
def test_copy_by_the_rows_past_2_to_the_30(big):
    n = 2 ** 30 + 5
    moves = big((n, 2), -1)
    moves[2 ** 30 + 1], moves[-1] = _ints([2, 3]), _ints([0, 1])
    k = torch.randn((4, 16, 1, 192), device="cuda").bfloat16()
    v = torch.randn((4, 16, 1, 128), device="cuda").bfloat16()
    want = [t[[0, 0, 2, 2]] for t in (k, v)]
    mimo.mimo_attn_page_copy(k, v, moves)
    mimo.mimo_attn_device_status()
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_an_empty_batch_needs_no_tables():
    """Its tensors have no entries and no address: nothing to do, on the host."""
    assert _attend(seqs=0, table=0, lens=0) == mimo.MIMO_OK
    assert _append(seqs=0, lens=0) == mimo.MIMO_OK
