"""Edges of the paged cache on the GPU: rows of one warp that part ways, slots that
nothing sees, sinks far below the scores, windows longer than a sequence, empty
batches, many heads, and turns in the life of a PagedCache.  Inputs and tolerances
as in tests/test_paged_gpu.py."""

import numpy as np
import pytest
import torch

from oracle import paged
from tests import parity_util as P
from tests.test_paged_gpu import attend, build, check, ints, oracle_of

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import global_attention_swa_b200 as mimo
    from global_attention_swa_b200.paged_cache import PagedCache


# windows whose items are one block and two; rows of a warp that hold no token, beside
# rows that are done again (a value that is not finite, hidden from some of them)
@pytest.mark.parametrize("lens,news,window,hq,hkv", [
    ([300, 90, 40], [13, 29, 5], 129, 16, 1), ([300, 90], [37, 45], 120, 48, 4), ([200, 60], [33, 11], 100, 7, 1),
    ([260, 31], [90, 31], 9, 3, 3)])
@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16])
def test_rows_of_a_warp_that_part_ways(lens, news, window, hq, hkv, odt):
    x = build(lens, news, window, 16, hq, hkv, seed=sum(news))
    for b, (L, n) in enumerate(zip(lens, news)):
        for p in (L - n, L - n // 2, L - 1):
            x["vp"][int(x["table"][b, p // 16]), p % 16, :, ::40] = float("nan")
    want, want_lse, mass = oracle_of(x)
    out, lse = attend(x, out_dtype=odt)
    o = P.to64(out)
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(o), fine)
    bound = 2.0 ** -8 * (mass + np.abs(want)) + 5.2e-4 * mass + 1e-6
    if odt == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    assert np.all(np.abs(o - want)[fine] <= bound[fine])
    assert np.max(np.abs(P.to64(lse) - want_lse)) <= 3e-4


@pytest.mark.parametrize("lens,news,window,hq,hkv", [
    ([701, 333], [77, 161], 129, 16, 1), ([95], [90], 129, 32, 2), ([333, 61], [100, 60], 40, 7, 1), ([500], [300], 9, 2, 2),
    ([333, 90], [30, 11], 100, 64, 1), ([333, 90], [30, 11], 33, 128, 1)])  # items of fewer tokens than a box
@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16])
def test_slots_that_nothing_sees_do_not_show(lens, news, window, hq, hkv, odt):
    """Chunks of several items: the slots before the first key and past the end change no
    bit of the result, written or not."""
    x = build(lens, news, window, 16, hq, hkv, seed=len(lens))
    assert torch.isnan(x["vp"][int(x["table"][0, (lens[0] - 1) // 16]), lens[0] % 16:]).all() and lens[0] % 16
    out, lse = attend(x, out_dtype=odt)
    x["kp"], x["vp"] = x["kp"].nan_to_num(0.0), x["vp"].nan_to_num(0.0)
    want, want_lse = attend(x, out_dtype=odt)
    check(want, want_lse, oracle_of(x))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("sink", [-1e10, -1e30, float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("window", [0, 129])
@pytest.mark.parametrize("lens,n,times", [([700, 30], 1, 64), ([700, 30], 6, 64), ([300, 30], 30, 64), ([9, 5], 5, 256)])
def test_a_sink_out_of_sight_beside_large_scores(lens, n, times, window, sink):
    """A sink so low that the gap to the scores does not keep their digits: scores of
    hundreds, of either sign, decide alone."""
    x = build(lens, [n] * len(lens), window, 16, 16, 1, seed=12)
    x["q"] *= times
    x["sinks"] = torch.full((16,), sink)
    out, lse = attend(x, out_dtype=torch.float32)
    want, want_lse, mass = oracle_of(x)
    assert want_lse.max() > 100 and (times == 64 or want_lse.min() < -100)
    # the scores are `times` those of the module's bound, so is their error
    assert np.all(np.abs(P.to64(out) - want) <= 2.0 ** -8 * (mass + np.abs(want)) + times * 5.2e-4 * mass + 1e-6)
    assert np.max(np.abs(P.to64(lse) - want_lse)) <= times * 3e-4


@pytest.mark.parametrize("lens,news", [([5000, 300], [1, 1]), ([5000, 900, 40], [6, 3, 6]), ([2600], [300]),
                                       ([2000, 2000, 70], [40, 2000, 70])])
def test_a_window_past_the_length_is_no_window(lens, news):
    """Nothing is hidden, so the work is dealt out as without one: the same bits."""
    x = build(lens, news, 0, 64, 16, 1, seed=sum(lens))
    want, want_lse = attend(x, out_dtype=torch.float32)
    for window in (max(lens), 6000, 2 ** 31 - 1):
        x["window"] = window
        out, lse = attend(x, out_dtype=torch.float32)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("lens,news,window,hq", [([1500], [900], 700, 16), ([1500, 40, 900], [1100, 3, 1], 600, 16),
                                                 ([2500, 300], [300, 300], 1000, 6), ([700, 900], [700, 17], 650, 64)])
def test_chunks_that_grow_into_their_window(lens, news, window, hq):
    """First blocks that see less than a window, and later ones that see a whole one."""
    x = build(lens, news, window, 16, hq, 1, seed=window)
    check(*attend(x), oracle_of(x))


def test_a_fork_that_stands_still_needs_no_page():
    """Only the slots that get tokens part from the shared page: four beams, one free page,
    one beam goes on."""
    cache = PagedCache(1, 3, 16, 4, 3, 1)
    cache.extend(ints([20, 0, 0, 0]).cuda())
    cache.fork(ints([0, 0, 0, 0]).cuda())
    shared = cache.block_table[0, :2].tolist()
    info = cache.extend(ints([0, 1, 0, 0]).cuda())
    mimo.mimo_attn_device_status()
    assert info.tolist() == [0, 0] and cache.seqlens.tolist() == [20, 21, 20, 20]
    table = cache.block_table[:, :2].tolist()
    assert [table[i] for i in (0, 2, 3)] == [shared] * 3 and table[1] == [shared[0], ({0, 1, 2} - set(shared)).pop()]
    assert cache.page_refs[shared].tolist() == [4, 3]


@pytest.mark.parametrize("change", ["truncate", "fork"])
def test_a_sequence_without_room_stays_skipped_until_it_is_extended(change):
    """The pool has no page for slot 1's next tokens; freeing slot 0 does not give them to
    it: attend leaves what is there as it is until extend has."""
    g = torch.Generator().manual_seed(5)

    def chunk(n):
        return [torch.randn((n, h, d), generator=g).to(torch.bfloat16).cuda() for h, d in ((8, 192), (2, 192), (2, 128))]

    cache = PagedCache(1, 5, 16, 2, 5, 2)
    cache.extend(ints([40, 30]).cuda())
    cache.attend(0, *chunk(70), ints([0, 40, 70]).cuda(), 40, None, 1e4)
    assert cache.extend(ints([0, 8]).cuda())[0] == 1
    if change == "truncate":
        cache.truncate(ints([0, 30]).cuda())
    else:
        cache.fork(ints([-1, 1]).cuda())
    mimo.mimo_attn_device_status()
    k, v = cache.k_pages.clone(), cache.v_pages.clone()
    rows = chunk(8)
    cache.attend(0, *rows, ints([0, 0, 8]).cuda(), 8, None, 1e4)
    with pytest.raises(mimo.MimoAttnError) as e:
        mimo.mimo_attn_device_status()
    assert e.value.status == mimo.MIMO_ERR_INVALID_ARG
    assert torch.equal(cache.k_pages, k) and torch.equal(cache.v_pages, v)
    assert cache.extend(ints([0, 8]).cuda())[0] == 0 and cache.seqlens.tolist() == [0, 38]
    out, _ = cache.attend(0, *rows, ints([0, 0, 8]).cuda(), 8, None, 1e4)
    mimo.mimo_attn_device_status()
    assert torch.isfinite(out).all() and torch.equal(cache.v_pages[0, cache.block_table[1, 2].long(), :6], rows[2][2:])
    assert torch.equal(cache.v_pages[0, cache.block_table[1, 1].long(), :14], v[0, cache.block_table[1, 1].long(), :14])


def test_room_that_is_given_back_before_it_is_used():
    """extend for the most drafted tokens, truncate to those there are, then attend."""
    g = torch.Generator().manual_seed(6)
    cache = PagedCache(1, 8, 16, 2, 4, 1)
    cache.extend(ints([9, 9]).cuda())
    cache.truncate(ints([5, 3]).cuda())
    q, k, v = (torch.randn((8, h, d), generator=g).to(torch.bfloat16).cuda() for h, d in ((4, 192), (1, 192), (1, 128)))
    cache.attend(0, q, k, v, ints([0, 5, 8]).cuda(), 5, None)
    mimo.mimo_attn_device_status()
    for b, rows in enumerate((slice(0, 5), slice(5, 8))):
        page = int(cache.block_table[b, 0])
        assert torch.equal(cache.v_pages[0, page, :rows.stop - rows.start], v[rows])


@pytest.mark.parametrize("window", [0, 129])
def test_rows_of_skipped_sequences_stay_as_the_caller_had_them(window):
    """Slot 1 would pass its table: its rows of out and lse keep what they held, the others
    are those of a call that makes its own."""
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn((12, h, d), generator=g).to(torch.bfloat16).cuda() for h, d in ((8, 192), (2, 192), (2, 128)))
    cache = PagedCache(1, 16, 16, 3, 2, 2, window=window)
    cache.extend(ints([5, 40, 4]).cuda())
    cu = ints([0, 5, 8, 12]).cuda()
    want, want_lse = cache.attend(0, q, k, v, cu, 5, None, out_dtype=torch.float32)
    out, lse = torch.full((12, 8, 128), 7.0, device="cuda"), torch.full((8, 12), 7.0, device="cuda")
    got = cache.attend(0, q, k, v, cu, 5, None, out=out, lse=lse)
    assert got[0] is out or got[0].data_ptr() == out.data_ptr()
    with pytest.raises(mimo.MimoAttnError) as e:
        mimo.mimo_attn_device_status()
    assert e.value.status == mimo.MIMO_ERR_INVALID_ARG
    assert torch.all(out[5:8] == 7) and torch.all(lse[:, 5:8] == 7)
    for rows in (slice(0, 5), slice(8, 12)):
        assert torch.isfinite(out[rows]).all() and torch.equal(out[rows], want[rows])
        assert torch.equal(lse[:, rows], want_lse[:, rows])


def test_tensors_made_for_another_stream_are_not_memory_still_in_use():
    """A call on a stream of the caller's beside pending work on the current one: what it
    makes does not lie over a tensor that the pending work writes, though that was freed."""
    x = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in build([900, 60], [6, 6], 0, 16, 16, 1, 3).items()}
    x["kp"], x["vp"] = x["kp"].nan_to_num(0.0), x["vp"].nan_to_num(0.0)
    args = [x[k] for k in ("q", "kp", "vp", "table", "cu", "lens", "most", "window", "sinks")]
    g = torch.Generator().manual_seed(1)
    kv = [torch.randn((12, 1, d), generator=g).bfloat16().cuda() for d in (192, 128)]
    kp, vp = x["kp"].clone(), x["vp"].clone()
    refs, table, lens, parent = (ints(v).cuda() for v in ([1, 0, 1, 0, 0], [[2, 0, -1]], [48], [0, 0]))
    need = mimo.mimo_attn_paged_attention_workspace_size(16, 1, 2, 12, 6)
    side = torch.cuda.Stream()

    def calls(stream):
        return [*mimo.mimo_attn_paged_attention(*args, stream=stream),
                mimo.mimo_attn_paged_append(x["q"], *kv, kp, vp, *args[3:6], 1e4, stream=stream),
                *mimo.mimo_attn_page_hold(refs, table, lens, 16, stream=stream),
                *mimo.mimo_attn_page_fork(refs, table, parent, stream=stream),
                *mimo.mimo_attn_page_compact(refs, table, 2, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    for make in (lambda: mimo.mimo_attn_paged_attention(*args, stream=side),
                 lambda: [mimo.mimo_attn_paged_append(x["q"], *kv, kp, vp, *args[3:6], 1e4, stream=side)],
                 lambda: mimo.mimo_attn_page_hold(refs, table, lens, 16, stream=side),
                 lambda: mimo.mimo_attn_page_fork(refs, table, parent, stream=side),
                 lambda: mimo.mimo_attn_page_compact(refs, table, 2, stream=side)):
        first = make()
        torch.cuda.synchronize()
        first = [t.clone() for t in first]
        torch.cuda.synchronize()
        gone = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (need, *[t.nbytes for t in first], *[512] * 8)]
        torch.cuda._sleep(200_000_000)
        for t in gone:
            t.fill_(7)
        del t, gone
        got = make()
        side.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(got, first):
            assert torch.equal(a, b)
    got = calls(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    mimo.mimo_attn_device_status()


def test_calls_of_no_sequence():
    """An empty batch: nothing to do, no row touched."""
    empty = lambda *s, dt=torch.int32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    kp, vp = (torch.ones((4, 16, 1, d), dtype=torch.bfloat16, device="cuda") for d in (192, 128))
    for rows in (0, 3):
        q = torch.ones((rows, 4, 192), dtype=torch.bfloat16, device="cuda")
        out = torch.full((rows, 4, 128), 7.0, device="cuda")
        args = (kp, vp, empty(0, 5), ints([0]).cuda(), empty(0))
        got, lse = mimo.mimo_attn_paged_attention(q, *args, 0, 0, None, out=out)
        assert got.shape == out.shape and lse.shape == (4, rows) and torch.all(out == 7)
        qo = torch.full_like(q, 5.0)
        mimo.mimo_attn_paged_append(q, q[:, :1].contiguous(), q[:, :1, :128].contiguous(), *args, 1e4, q_out=qo)
        assert torch.all(qo == 5) and torch.all(kp == 1) and torch.all(vp == 1)
    refs, table, moves, info = mimo.mimo_attn_page_hold(ints([0, 2, 0]).cuda(), empty(0, 5), empty(0), 16)
    assert refs.tolist() == [0, 2, 0] and table.shape == (0, 5) and moves.shape == (0, 2) and info.tolist() == [0, 2]
    refs, table = mimo.mimo_attn_page_fork(ints([0, 2]).cuda(), empty(0, 5), empty(0))
    assert refs.tolist() == [0, 2] and table.shape == (0, 5)
    refs, table, moves, info = mimo.mimo_attn_page_compact(ints([0, 2]).cuda(), empty(0, 5), 1)
    assert refs.tolist() == [2, 0] and moves.tolist() == [[1, 0]] and info.tolist() == [1, 1]
    mimo.mimo_attn_device_status()


@pytest.mark.parametrize("hq,hkv", [(128, 1), (128, 32), (72, 24), (256, 64)])
@pytest.mark.parametrize("rotary", [192, 128, 64, 60, 0])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_of_more_heads_than_a_block_holds_at_once(hq, hkv, rotary, in_place):
    g = torch.Generator().manual_seed(hq + rotary)
    lens, news, ps, table = [20, 3, 70], [2, 3, 1], 32, [[1, -1, -1], [0, -1, -1], [-1, -1, 2]]
    cu = [0, 2, 5, 6]
    q, k, v = (torch.randn((6, h, d), generator=g).to(torch.bfloat16) for h, d in ((hq, 192), (hkv, 192), (hkv, 128)))
    kp, vp = (torch.randn((3, ps, hkv, d), generator=g).to(torch.bfloat16) for d in (192, 128))
    rq, rk, rv = paged.paged_append(q, k, v, kp, vp, table, cu, lens, 1e4, rotary)
    qd, kd, vd = q.cuda(), kp.cuda(), vp.cuda()
    qo = mimo.mimo_attn_paged_append(qd, k.cuda(), v.cuda(), kd, vd, ints(table).cuda(), ints(cu).cuda(), ints(lens).cuda(),
                                     1e4, rotary, q_out=qd if in_place else None)
    mimo.mimo_attn_device_status()
    for got, want in ((qo, rq), (kd, rk)):
        assert np.all(np.abs(P.to64(got) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)
    assert np.array_equal(P.to64(vd), rv)
