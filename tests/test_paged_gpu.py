"""Paged cache on the GPU against the fp64 / integer oracle (oracle/paged.py).

Tolerances, per element, for inputs ~N(0, 1):
* weights enter P.V rounded to bf16 (half a step, 2^-8 relative) and are
  normalised by the sum of the rounded ones, so the output moves by at most
  2^-8 sum_j w_j |v_j - out| <= 2^-8 (mass + |out|), mass = v_scale sum_j w_j |v_j|;
* a score is a sum of 192 products in fp32: its error is at most
  192 * 2^-24 * s sum_d |q_d k_d| <= 192 * 2^-24 * s |q| |k|, s |q| |k| < 22 for
  the norms drawn here, so 2.6e-4; a weight's relative error is at most twice
  that, and the log-sum-exp's error at most 2.6e-4 (3e-4 with its own roundings);
* a bf16 output is rounded once more: 2^-8 of its magnitude.
Rotated rows: half a bf16 step, 2^-8 relative, with the floor 1e-5 for the fp32
products.  Copies and whole numbers are compared bit for bit.

Every slot that no query sees is NaN, as are the pages that no table names.
"""

import random

import numpy as np
import pytest
import torch

from oracle import paged
from tests import parity_util as P

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import global_attention_swa_b200 as mimo
    from global_attention_swa_b200.paged_cache import PagedCache

I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32)


def build(lens, news, window, ps, hq, hkv, seed, poison=True, spare=3):
    """Random packed queries and a scattered paged cache; every page is drawn from the
    pool at random, pages wholly behind the window are not in the table."""
    g = torch.Generator().manual_seed(seed)
    r = random.Random(seed)
    width = max(1, max(-(-L // ps) for L in lens)) + 1
    lo = [max(0, L - n - window + 1) if window else 0 for L, n in zip(lens, news)]
    need = sum(-(-L // ps) - a // ps for L, a in zip(lens, lo))
    pool = need + spare
    order = r.sample(range(pool), need)
    kp = torch.full((pool, ps, hkv, 192), float("nan") if poison else 0.0).to(torch.bfloat16)
    vp = torch.full((pool, ps, hkv, 128), float("nan") if poison else 0.0).to(torch.bfloat16)
    table = []
    for L, a in zip(lens, lo):
        row = [-1] * width
        for j in range(a // ps, -(-L // ps)):
            row[j] = order.pop()
            s0, s1 = max(a, j * ps) - j * ps, min(L, (j + 1) * ps) - j * ps
            kp[row[j], s0:s1] = torch.randn((s1 - s0, hkv, 192), generator=g).to(torch.bfloat16)
            vp[row[j], s0:s1] = torch.randn((s1 - s0, hkv, 128), generator=g).to(torch.bfloat16)
        table.append(row)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], hq, 192), generator=g).to(torch.bfloat16)
    sinks = torch.randn(hq, generator=g)
    return dict(q=q, kp=kp, vp=vp, table=ints(table), cu=ints(cu), lens=ints(lens), sinks=sinks, most=max(news),
                window=window)


def attend(x, **kw):
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    got = mimo.mimo_attn_paged_attention(dev["q"], dev["kp"], dev["vp"], dev["table"], dev["cu"], dev["lens"],
                                         dev["most"], dev["window"], dev["sinks"], **kw)
    mimo.mimo_attn_device_status()
    return got


def check(out, lse, ref, rows=None):
    o, l = P.to64(out), P.to64(lse)
    want, want_lse, mass = ref
    if rows is not None:
        o, l, want, want_lse, mass = o[rows], l[:, rows], want[rows], want_lse[:, rows], mass[rows]
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(l))
    bound = 2.0 ** -8 * (mass + np.abs(want)) + 5.2e-4 * mass + 1e-6
    if out.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    err = np.abs(o - want)
    assert np.all(err <= bound), f"out: worst {np.max(err - bound):.3e} over, at {np.unravel_index(np.argmax(err - bound), err.shape)}"
    assert np.max(np.abs(l - want_lse), initial=0.0) <= 3e-4


def oracle_of(x, **kw):
    return paged.paged_attention(x["q"], x["kp"], x["vp"], x["table"].tolist(), x["cu"].tolist(), x["lens"].tolist(),
                                 x["window"], x["sinks"], **kw)


CASES = [
    # lens, new tokens, window, page size, Hq, Hkv
    ([1], [1], 0, 16, 16, 1),
    ([1, 2, 15, 16, 17], [1, 1, 1, 1, 1], 0, 16, 64, 4),
    ([63, 64, 65, 127, 128, 129, 130], [1] * 7, 0, 64, 16, 1),
    ([300, 1000, 4, 2049], [1, 1, 1, 1], 0, 48, 32, 2),
    ([3000, 5], [1, 1], 0, 16, 16, 1),
    ([1, 128, 129, 130, 700], [1] * 5, 129, 16, 16, 1),
    ([400, 33], [1, 1], 1, 32, 16, 1),
    ([500, 40, 77], [3, 1, 5], 0, 16, 64, 4),           # drafted tokens
    ([0, 50, 0, 9, 1], [0, 0, 0, 9, 1], 0, 16, 16, 1),  # empty sequences and chunks
    ([200], [200], 0, 64, 16, 1),                       # the whole prompt
    ([130, 20], [130, 7], 129, 16, 16, 1),
    ([700, 300], [77, 161], 129, 48, 32, 2),
    ([600, 300], [150, 33], 200, 16, 16, 1),
    ([520], [133], 5, 16, 16, 1),
    ([700], [130], 0, 128, 16, 1),
    ([700, 130], [40, 129], 0, 256, 16, 2),             # pages longer than a tile; G = 8
    ([300, 20], [140, 3], 0, 32, 24, 2),                # G = 12 does not divide 128
    ([300, 20], [140, 3], 129, 32, 24, 2),
    ([400, 20], [300, 3], 0, 16, 3, 3),                 # G = 1
    ([400, 20], [300, 3], 129, 16, 2, 2),
    ([300, 20], [20, 3], 0, 16, 32, 1),                 # G = 32
    ([150, 20], [9, 3], 0, 16, 128, 1),                 # G = 128: a tile of one token
    ([150, 20], [1, 1], 0, 16, 96, 1),                  # G = 96, single tokens
    ([260, 31], [40, 31], 0, 16, 7, 1),                 # G = 7
]


@pytest.mark.parametrize("lens,news,window,ps,hq,hkv", CASES)
def test_attention(lens, news, window, ps, hq, hkv):
    x = build(lens, news, window, ps, hq, hkv, seed=len(lens) + ps + hq)
    ref = oracle_of(x)
    for dt in (torch.bfloat16, torch.float32):
        out, lse = attend(x, out_dtype=dt)
        check(out, lse, ref)


@pytest.mark.parametrize("seed", range(16))
def test_attention_of_random_shapes(seed):
    r = random.Random(1000 + seed)
    hq, hkv = r.choice([(16, 1), (16, 2), (12, 1), (4, 4), (20, 1), (64, 1), (33, 3)])
    ps, window = r.choice([16, 32, 48, 64, 80, 128, 160]), r.choice([0, 0, 0, 1, 17, 128, 129, 130, 333])
    lens = [r.choice([r.randint(0, 40), r.randint(1, 700)]) for _ in range(r.randint(1, 6))] + [r.randint(1, 300)]
    top = r.choice([1, 4, 20, 160])
    news = [min(L, r.randint(0, top)) for L in lens]
    news[-1] = max(1, news[-1])
    x = build(lens, news, window, ps, hq, hkv, seed=seed)
    check(*attend(x), oracle_of(x))


def test_no_sinks_scale_and_value_scale():
    x = build([90, 33], [30, 2], 0, 16, 16, 1, seed=5)
    x["sinks"] = None
    check(*attend(x), oracle_of(x))
    check(*attend(x, softmax_scale=0.05, v_scale=0.707), oracle_of(x, scale=0.05, v_scale=0.707))
    assert attend(x, return_lse=False)[1] is None


@pytest.mark.parametrize("sink", [-60.0, 60.0])
@pytest.mark.parametrize("n", [1, 20])
def test_extreme_sinks(sink, n):
    x = build([333], [n], 0, 16, 16, 1, seed=6)
    x["sinks"] = torch.full((16,), sink)
    check(*attend(x), oracle_of(x))


@pytest.mark.parametrize("sink", [None, -40.0])
@pytest.mark.parametrize("window", [0, 129])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_large_scores(n, window, sink):
    """Scores of several hundred, both signs, rising along the row: no weight overflows,
    none is lost, and a reference that was taken early is moved."""
    x = build([700], [n], window, 16, 16, 1, seed=8)
    x["q"] *= 16
    x["sinks"] = None if sink is None else torch.full((16,), sink)
    out, lse = attend(x, out_dtype=torch.float32)
    want, want_lse, mass = oracle_of(x)
    # the scores are 16 times those of the module's bound, so is their error: 4.2e-3
    err = np.abs(P.to64(out) - want)
    assert np.all(err <= 2.0 ** -8 * (mass + np.abs(want)) + 16 * 5.2e-4 * mass + 1e-6)
    assert np.max(np.abs(P.to64(lse) - want_lse)) <= 16 * 3e-4


def test_a_longer_ragged_batch():
    """Chunks that span many tiles, split along the keys and not."""
    x = build([5000, 1, 900, 2600], [300, 1, 130, 17], 0, 64, 16, 1, seed=11)
    check(*attend(x), oracle_of(x))


@pytest.mark.parametrize("window", [0, 129])
def test_rows_of_no_sequence_are_left_alone(window):
    x = build([70, 30], [20, 1], window, 16, 16, 1, seed=3)
    rows = x["q"].shape[0]
    x["q"] = torch.cat([x["q"], torch.full((5, 16, 192), float("nan"), dtype=torch.bfloat16)])
    out = torch.full((rows + 5, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((16, rows + 5), 7.0, device="cuda")
    attend(x, out=out, lse=lse)
    check(out, lse, oracle_of(x), rows=slice(0, rows))
    assert torch.all(out[rows:] == 7) and torch.all(lse[:, rows:] == 7)


@pytest.mark.parametrize("n", [1, 5, 50])
def test_bad_sequences_are_skipped_and_recorded(n):
    """More new tokens than the length, and a length past the table, among good ones."""
    x = build([80, 90, 100, 60], [n] * 4, 0, 16, 16, 1, seed=4)
    ref = oracle_of(x)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    dev["lens"] = ints([80, n - 1, 16 * dev["table"].shape[1] + 1, 60]).cuda()
    out = torch.full((4 * n, 16, 128), 7.0, device="cuda")
    lse = torch.full((16, 4 * n), 7.0, device="cuda")
    mimo.mimo_attn_paged_attention(dev["q"], dev["kp"], dev["vp"], dev["table"], dev["cu"], dev["lens"], n, 0,
                                   dev["sinks"], out=out, lse=lse)
    with pytest.raises(mimo.MimoAttnError) as e:
        mimo.mimo_attn_device_status()
    assert e.value.status == mimo.MIMO_ERR_INVALID_ARG
    check(out, lse, ref, rows=slice(0, n))
    check(out, lse, ref, rows=slice(3 * n, 4 * n))
    assert torch.all(out[n:3 * n] == 7) and torch.all(lse[:, n:3 * n] == 7)


@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("n", [1, 5, 50])
def test_a_visible_entry_without_a_page_reads_as_zeros(bad, n):
    x = build([150, 40], [n, 1], 0, 16, 16, 1, seed=9)
    x["table"][0, 3] = bad
    ref = oracle_of(x)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    out, lse = mimo.mimo_attn_paged_attention(dev["q"], dev["kp"], dev["vp"], dev["table"], dev["cu"], dev["lens"],
                                              n, 0, dev["sinks"])
    with pytest.raises(mimo.MimoAttnError) as e:
        mimo.mimo_attn_device_status()
    assert e.value.status == mimo.MIMO_ERR_INVALID_ARG
    check(out, lse, ref)


@pytest.mark.parametrize("lens,news,window,hq,hkv", [
    ([200], [5], 0, 16, 1), ([200, 90], [40, 33], 0, 16, 1), ([3000], [30], 0, 16, 1), ([200, 40], [40, 9], 129, 16, 1),
    ([300], [40], 200, 16, 1), ([200], [7], 3, 16, 1), ([700], [300], 0, 2, 2), ([500], [200], 10, 2, 2),
    ([150, 70], [12, 3], 0, 8, 2), ([700], [90], 600, 16, 1)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(lens, news, window, hq, hkv, what):
    """Not finite: some value columns of one key, all of another, one key's own row; each
    seen by some queries of the chunk and hidden from others."""
    x = build(lens, news, window, 16, hq, hkv, seed=17)
    for b, (L, n) in enumerate(zip(lens, news)):
        first = L - n
        low = max(0, first - window + 1) if window else 0
        spots = [(first + n // 2, "v", slice(3, 9)), (L - 1, "v", slice(None)), (first + 3 * n // 4, "k", slice(0, 1))]
        if window:
            spots.append((low + min(n, window) // 2, "v", slice(100, 101)))
        for p, kind, cols in spots:
            page, slot = int(x["table"][b, p // 16]), p % 16
            x["kp" if kind == "k" else "vp"][page, slot, 0, cols] = what
    want, want_lse, mass = oracle_of(x)
    out, lse = attend(x, out_dtype=torch.float32)
    o, l = P.to64(out), P.to64(lse)
    fine, lfine = np.isfinite(want), np.isfinite(want_lse)
    assert not fine.all() and fine[:, :, 50].any()
    assert np.array_equal(np.isfinite(o), fine)
    bound = 2.0 ** -8 * (mass + np.abs(want)) + 5.2e-4 * mass + 1e-6
    ok = fine & np.isfinite(mass)
    assert np.all(np.abs(o - want)[ok] <= bound[ok])
    assert np.array_equal(np.isnan(l), np.isnan(want_lse)) and np.array_equal(np.isfinite(l), lfine)
    assert np.max(np.abs(l - want_lse)[lfine], initial=0.0) <= 3e-4


def test_agrees_with_prefill_and_decode():
    """The whole prompt as one chunk is the dense prefill; its last token alone is the dense decode."""
    T, hq, hkv = 321, 64, 4
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((T, h, d), generator=g).to(torch.bfloat16).cuda() for h, d in ((hq, 192), (hkv, 192), (hkv, 128)))
    sinks = torch.randn(hq, generator=g).cuda()
    table = torch.randperm(6, generator=g).int().cuda()[None]
    kp, vp = torch.zeros((6, 64, hkv, 192), dtype=torch.bfloat16).cuda(), torch.zeros((6, 64, hkv, 128), dtype=torch.bfloat16).cuda()
    pos = torch.arange(T).cuda()
    kp[table[0, pos // 64].long(), pos % 64] = k
    vp[table[0, pos // 64].long(), pos % 64] = v
    lens = ints([T]).cuda()
    for window in (0, 129):
        want, want_lse = mimo.mimo_attn_prefill(q, k, v, sinks, window, ints([0, T]).cuda(), T)
        out, lse = mimo.mimo_attn_paged_attention(q, kp, vp, table, ints([0, T]).cuda(), lens, T, window, sinks)
        # both are within half a bf16 step twice (weights, output) of the same value, of magnitude < 4
        assert (out.float() - want.float()).abs().max() <= 4 * 4 * 2.0 ** -8
        assert (lse - want_lse).abs().max() <= 6e-4
        one, one_lse = mimo.mimo_attn_paged_attention(q[-1:].contiguous(), kp, vp, table, ints([0, 1]).cuda(), lens, 1,
                                                      window, sinks)
        assert (one.float() - want[-1:].float()).abs().max() <= 4 * 4 * 2.0 ** -8
        assert (one_lse - want_lse[:, -1:]).abs().max() <= 6e-4
    mimo.mimo_attn_device_status()


@pytest.mark.parametrize("n", [1, 4, 60])
def test_twice_the_same(n):
    x = build([900, 40, 333], [n, min(n, 40), 1], 0, 32, 16, 1, seed=13)
    a, al = attend(x)
    b, bl = attend(x)
    assert torch.equal(a, b) and torch.equal(al, bl)


def test_a_pool_past_32_bit_offsets():
    """Pages whose element offsets pass 2^31 and byte offsets 2^32."""
    hkv, ps = 4, 64
    pool = 2 ** 32 // (ps * hkv * 192) + 3   # past 2^32 elements of keys
    kp = torch.zeros((pool, ps, hkv, 192), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros((pool, ps, hkv, 128), dtype=torch.bfloat16, device="cuda")
    for n in (1, 5, 90):
        x = build([150], [n], 0, ps, 64, 4, seed=n)
        at = [pool - 1, 0, pool - 2]
        for i, page in enumerate(at):
            src = int(x["table"][0, i])
            kp[page], vp[page] = x["kp"][src].cuda(), x["vp"][src].cuda()
        out, lse = mimo.mimo_attn_paged_attention(x["q"].cuda(), kp, vp, ints([at]).cuda(), x["cu"].cuda(), x["lens"].cuda(),
                                                  n, 0, x["sinks"].cuda())
        mimo.mimo_attn_device_status()
        check(out, lse, oracle_of(x))
    moves = ints([[pool - 1, pool - 3]]).cuda()
    mimo.mimo_attn_page_copy(kp, vp, moves)
    assert torch.equal(kp[pool - 3].nan_to_num(), kp[pool - 1].nan_to_num())
    assert torch.equal(vp[pool - 3].nan_to_num(), vp[pool - 1].nan_to_num())
    x = build([64], [64], 0, ps, 64, 4, seed=1)
    k, v = torch.randn((64, 4, 192), device="cuda").bfloat16(), torch.randn((64, 4, 128), device="cuda").bfloat16()
    mimo.mimo_attn_paged_append(x["q"].cuda(), k, v, kp, vp, ints([[pool - 2]]).cuda(), x["cu"].cuda(), x["lens"].cuda(),
                                1e4, 0)
    assert torch.equal(kp[pool - 2], k) and torch.equal(vp[pool - 2], v)
    mimo.mimo_attn_device_status()


def test_on_another_stream_and_two_at_once():
    xs = [build([1500, 40], [1, 1], 0, 16, 16, 1, seed=21), build([600, 50], [40, 50], 0, 16, 16, 1, seed=22)]
    devs = [{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()} for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], []
    for rep in range(5):
        for d, s in zip(devs, streams):
            with torch.cuda.stream(s):
                got.append(mimo.mimo_attn_paged_attention(d["q"], d["kp"], d["vp"], d["table"], d["cu"], d["lens"],
                                                          d["most"], 0, d["sinks"]))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        check(out, lse, oracle_of(xs[i % 2]))
    d = devs[0]
    out, lse = mimo.mimo_attn_paged_attention(d["q"], d["kp"], d["vp"], d["table"], d["cu"], d["lens"], 1, 0,
                                              d["sinks"], stream=streams[0])
    streams[0].synchronize()
    check(out, lse, oracle_of(xs[0]))


# ------------------------------------------------------------------ append


def _close(got, ref, what):
    g = P.to64(got)
    err = np.abs(g - ref)
    bound = 2.0 ** -8 * np.abs(ref) + 1e-5
    assert np.all(err <= bound), f"{what}: worst {np.max(err - bound):.3e}"


@pytest.mark.parametrize("theta,rotary", [(10000.0, 192), (1.0e6, 64), (500.0, 60), (1e4, 0), (1e4, 48)])
@pytest.mark.parametrize("lens,news,ps,hq,hkv", [
    ([1, 2, 17, 100], [1, 1, 1, 1], 16, 64, 4),
    ([40, 0, 5, 70], [33, 0, 5, 1], 48, 6, 2),
    ([262144], [3], 128, 16, 1),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_append(lens, news, ps, hq, hkv, theta, rotary, in_place):
    g = torch.Generator().manual_seed(7)
    r = random.Random(7)
    width = -(-max(lens) // ps)
    pool = sum(-(-n // ps) + 1 for n in news) + 2
    order, table = r.sample(range(pool), pool), []
    for L, n in zip(lens, news):
        row = [-1] * width
        for j in range((L - n) // ps, -(-L // ps) if n else 0):
            row[j] = order.pop()
        table.append(row)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    nt = cu[-1] + 2  # two rows of no sequence
    q, k, v = (torch.randn((nt, h, d), generator=g).to(torch.bfloat16) for h, d in ((hq, 192), (hkv, 192), (hkv, 128)))
    kp = torch.randn((pool, ps, hkv, 192), generator=g).to(torch.bfloat16)
    vp = torch.randn((pool, ps, hkv, 128), generator=g).to(torch.bfloat16)
    rq, rk, rv = paged.paged_append(q, k, v, kp, vp, table, cu, lens, theta, rotary)
    qd, kd, vd = q.cuda(), kp.cuda(), vp.cuda()
    qo = qd if in_place else torch.full_like(qd, 3.0)
    got = mimo.mimo_attn_paged_append(qd, k.cuda(), v.cuda(), kd, vd, ints(table).cuda(), ints(cu).cuda(),
                                      ints(lens).cuda(), theta, rotary, q_out=qo)
    mimo.mimo_attn_device_status()
    assert got is qo
    _close(qo[:-2], rq[:-2], "q")
    _close(kd, rk, "keys")
    assert np.array_equal(P.to64(vd), rv)
    same = np.isin(np.arange(pool * ps), [table[b][p // ps] * ps + p % ps for b in range(len(lens))
                                         for p in range(lens[b] - news[b], lens[b])], invert=True)
    assert torch.equal(kd.cpu().flatten(0, 1)[same], kp.flatten(0, 1)[same])
    if in_place:
        assert torch.equal(qo[-2:].cpu(), q[-2:])
    else:
        assert torch.all(qo[-2:] == 3) and torch.equal(qd.cpu(), q)


def test_append_without_a_page_or_of_a_bad_length():
    z = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for table, lens in (([[-1, 1]], [16]), ([[9, 1]], [16]), ([[0, 1]], [33]), ([[0, 1]], [3])):
        kp, vp = torch.zeros((2, 16, 1, 192), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 16, 1, 128), dtype=torch.bfloat16, device="cuda")
        q = z(4, 2, 192)
        qo = torch.full_like(q, 5.0)
        mimo.mimo_attn_paged_append(q, z(4, 1, 192), z(4, 1, 128), kp, vp, ints(table).cuda(), ints([0, 4]).cuda(),
                                    ints(lens).cuda(), 1e4, q_out=qo)
        with pytest.raises(mimo.MimoAttnError) as e:
            mimo.mimo_attn_device_status()
        assert e.value.status == mimo.MIMO_ERR_INVALID_ARG
        assert not kp.any() and not vp.any()
        assert torch.all(qo == 5) == (lens[0] in (33, 3))


# ------------------------------------------------------------------ bookkeeping


def _state(seed, pool, B, M, ps):
    """A sound random state: pages shared by some rows, holes, sequences of many lengths."""
    r = random.Random(seed)
    refs, table, lens = [0] * pool, [[-1] * M for _ in range(B)], [0] * B
    free = r.sample(range(pool), pool)
    for b in range(B):
        lens[b] = r.choice([0, r.randint(0, M * ps), r.randint(0, M * ps)])
        if b and r.random() < 0.4:  # shares the first pages of the row before
            lens[b] = r.randint(0, lens[b - 1])
            for j in range(-(-lens[b] // ps)):
                table[b][j] = table[b - 1][j]
                if table[b][j] >= 0:
                    refs[table[b][j]] += 1
        else:
            n = min(-(-lens[b] // ps), len(free) // 2)
            lens[b] = min(lens[b], n * ps)
            for j in range(r.randint(0, n) if r.random() < 0.2 else 0, n):
                table[b][j] = free.pop()
                refs[table[b][j]] = 1
    return refs, table, lens


def _lists(*ts):
    return [t.tolist() for t in ts]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pool,B,M,ps", [(5, 1, 3, 16), (40, 7, 5, 16), (300, 33, 12, 64), (3001, 150, 61, 16),
                                         (70000, 40, 1500, 16)])
@pytest.mark.parametrize("seed", range(4))
def test_hold(pool, B, M, ps, seed, in_place):
    refs, table, lens = _state(seed, pool, B, M, ps)
    r = random.Random(seed)
    after = [r.choice([0, L, min(M * ps, L + r.randint(0, 3 * ps)), r.randint(0, L)]) for L in lens]
    first = [r.randint(0, L) for L in after] if seed % 2 else None
    wf = [r.choice([min(a, L), r.randint(0, a)]) for a, L in zip(after, lens)] if seed >= 1 else None
    want = paged.page_hold(refs, table, after, ps, first, wf)
    dr, dt = ints(refs).cuda(), ints(table).cuda()
    cuda = lambda x: None if x is None else ints(x).cuda()  # noqa: E731
    got = mimo.mimo_attn_page_hold(dr, dt, cuda(after), ps, cuda(first), cuda(wf),
                                   refs_out=dr if in_place else None, table_out=dt if in_place else None)
    mimo.mimo_attn_device_status()
    assert _lists(*got) == list(want)
    if not in_place:
        assert _lists(dr, dt) == [refs, table]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pool,B,M", [(30, 6, 9), (5000, 64, 200)])
def test_hold_without_enough_pages(pool, B, M, in_place):
    """Releases, copies on write and fresh pages asked for at once, and too few pages: all as before."""
    refs, table, lens = _state(3, pool, B, M, 16)
    after = [M * 16] * B
    after[1] = 0
    wf = [0] * B
    want = paged.page_hold(refs, table, after, 16, None, wf)
    assert want[3][0] > 0
    dr, dt = ints(refs).cuda(), ints(table).cuda()
    got = mimo.mimo_attn_page_hold(dr, dt, ints(after).cuda(), 16, write_from=ints(wf).cuda(),
                                   refs_out=dr if in_place else None, table_out=dt if in_place else None)
    mimo.mimo_attn_device_status()
    assert _lists(*got) == list(want) and want[0] == refs and want[1] == table


def test_hold_records_bad_rows_and_entries():
    refs, table = [1, 1, 0, 0], [[0, -1], [1, -1], [-1, -1]]
    for lens, first, wf, tab in (([16, 99, 0], None, None, table), ([16, -1, 0], None, None, table),
                                 ([16, 16, 0], [0, -1, 0], None, table), ([16, 16, 0], None, [0, -5, 0], table),
                                 ([16, 16, 0], None, None, [[0, -1], [1, 7], [-1, -1]])):
        cuda = lambda x: None if x is None else ints(x).cuda()  # noqa: E731
        r2, t2, moves, info = mimo.mimo_attn_page_hold(ints(refs).cuda(), ints(tab).cuda(), cuda(lens), 16, cuda(first), cuda(wf))
        with pytest.raises(mimo.MimoAttnError) as e:
            mimo.mimo_attn_device_status()
        assert e.value.status == mimo.MIMO_ERR_INVALID_ARG
        assert r2.tolist() == refs and t2.tolist()[0] == [0, -1] and t2.tolist()[1][0] == 1
        assert info.tolist() == [0, 2]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pool,B,M,n", [(5, 1, 3, 4), (40, 7, 5, 7), (3001, 150, 61, 200), (70000, 40, 1500, 9),
                                        (100, 3000, 2, 5000)])
@pytest.mark.parametrize("seed", range(3))
def test_fork(pool, B, M, n, seed, in_place):
    refs, table, _ = _state(seed, pool, B, M, 16)
    r = random.Random(seed)
    parent = [r.randrange(-1, B) for _ in range(n)]
    if seed == 2:
        parent = [min(i, B - 1) for i in range(n)]
    want = paged.page_fork(refs, table, parent)
    dr, dt = ints(refs).cuda(), ints(table).cuda()
    got = mimo.mimo_attn_page_fork(dr, dt, ints(parent).cuda(), refs_out=dr if in_place else None)
    mimo.mimo_attn_device_status()
    assert _lists(*got) == list(want)
    assert dt.tolist() == table


def test_fork_to_nothing_and_of_a_row_that_is_not_there():
    refs, table = [2, 1, 0], [[0, 1], [0, -1]]
    got = mimo.mimo_attn_page_fork(ints(refs).cuda(), ints(table).cuda(), torch.zeros(0, dtype=I32).cuda())
    mimo.mimo_attn_device_status()
    assert got[0].tolist() == [0, 0, 0] and got[1].shape == (0, 2)
    got = mimo.mimo_attn_page_fork(ints(refs).cuda(), ints(table).cuda(), ints([0, 2]).cuda())
    with pytest.raises(mimo.MimoAttnError):
        mimo.mimo_attn_device_status()
    assert got[0].tolist() == [1, 1, 0] and got[1].tolist() == [[0, 1], [-1, -1]]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pool,B,M", [(5, 1, 3), (40, 7, 5), (3001, 150, 61), (70000, 40, 1500)])
@pytest.mark.parametrize("most", [0, 3, 100000])
def test_compact(pool, B, M, most, in_place):
    refs, table, _ = _state(5, pool, B, M, 16)
    want = paged.page_compact(refs, table, most)
    dr, dt = ints(refs).cuda(), ints(table).cuda()
    got = mimo.mimo_attn_page_compact(dr, dt, most, refs_out=dr if in_place else None, table_out=dt if in_place else None)
    mimo.mimo_attn_device_status()
    assert _lists(*got) == list(want)


@pytest.mark.parametrize("layers,pool,ps,hkv", [(None, 9, 16, 1), (3, 20, 48, 2), (2, 40, 64, 4)])
def test_copy(layers, pool, ps, hkv):
    g = torch.Generator().manual_seed(2)
    lead = () if layers is None else (layers,)
    kp = torch.randn((*lead, pool, ps, hkv, 192), generator=g).to(torch.bfloat16)
    vp = torch.randn((*lead, pool, ps, hkv, 128), generator=g).to(torch.bfloat16)
    moves = [[3, 0], [-1, -1], [pool - 1, 2], [3, 5], [-1, -1]]
    wk, wv = kp.clone(), vp.clone()
    for s, d in moves:
        if s >= 0:
            wk[..., d, :, :, :], wv[..., d, :, :, :] = kp[..., s, :, :, :], vp[..., s, :, :, :]
    k, v = mimo.mimo_attn_page_copy(kp.cuda(), vp.cuda(), ints(moves).cuda())
    mimo.mimo_attn_device_status()
    assert torch.equal(k.cpu(), wk) and torch.equal(v.cpu(), wv)
    k, v = mimo.mimo_attn_page_copy(kp.cuda(), vp.cuda(), ints([[pool, 0], [0, pool], [-1, 2], [3, -1]]).cuda())
    with pytest.raises(mimo.MimoAttnError):
        mimo.mimo_attn_device_status()
    assert torch.equal(k.cpu(), kp) and torch.equal(v.cpu(), vp)


# ------------------------------------------------------------------ the binding's two ways


def test_native_calls_and_marshalling_give_the_same(monkeypatch):
    """Every call through the native part of the binding and through Python's own
    marshalling: the same outputs, the same refusals."""
    assert mimo._fast is not None, "the native part of the binding is not built: run __graft_entry__.build()"
    x = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in build([90, 40], [20, 3], 0, 16, 16, 1, 2).items()}
    refs, table, lens = (ints(v).cuda() for v in _state(1, 40, 7, 5, 16))
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn((23, 1, d), generator=g, device="cuda").bfloat16() for d in (192, 128))

    def calls(native):
        taken = []
        if native:
            spy = type("Spy", (), {n: staticmethod(lambda *a, f=getattr(real, n): taken.append(f(*a)) or taken[-1])
                                   for n in dir(real) if not n.startswith("_")})
            monkeypatch.setattr(mimo, "_fast", spy)
        else:
            monkeypatch.setattr(mimo, "_fast", None)
        kp, vp = x["kp"].clone(), x["vp"].clone()
        out = torch.empty((23, 16, 128), device="cuda")
        args = (x["q"], kp, vp, x["table"], x["cu"], x["lens"], x["most"])
        got = [*mimo.mimo_attn_paged_attention(*args, 0, x["sinks"]),
               *mimo.mimo_attn_paged_attention(*args, 129, None, out=out, softmax_scale=0.1, v_scale=0.7, return_lse=False),
               *mimo.mimo_attn_paged_attention(*args, 0, x["sinks"], out_dtype=torch.float32,
                                               workspace=torch.empty(1 << 26, dtype=torch.uint8, device="cuda")),
               mimo.mimo_attn_paged_append(x["q"], k, v, kp, vp, x["table"], x["cu"], x["lens"], 1e4),
               mimo.mimo_attn_paged_append(x["q"], k, v, kp, vp, x["table"], x["cu"], x["lens"], 1e4, 64,
                                           q_out=torch.empty_like(x["q"])),
               *mimo.mimo_attn_page_hold(refs, table, lens, 16, first=lens // 2, write_from=lens),
               *mimo.mimo_attn_page_fork(refs, table, lens % 7), *mimo.mimo_attn_page_compact(refs, table, 3),
               *mimo.mimo_attn_page_copy(kp, vp, ints([[0, 1], [-1, -1]]).cuda())]
        mimo.mimo_attn_device_status()
        said = []
        for bad in (lambda: mimo.mimo_attn_paged_attention(x["q"].half(), *args[1:], 0, x["sinks"]),
                    lambda: mimo.mimo_attn_paged_attention(x["q"], kp[:, :8], *args[2:], 0, x["sinks"]),
                    lambda: mimo.mimo_attn_paged_attention(*args, -1, x["sinks"]),
                    lambda: mimo.mimo_attn_paged_attention(*args[:4], x["cu"].cpu(), *args[5:], 0, x["sinks"]),
                    lambda: mimo.mimo_attn_paged_attention(*args, 0, x["sinks"], workspace=torch.empty(8, device="cuda")),
                    lambda: mimo.mimo_attn_paged_append(x["q"], k, v, kp, vp, x["table"], x["cu"], x["lens"], 1e4, 7),
                    lambda: mimo.mimo_attn_page_hold(refs, table, lens[:3], 16),
                    lambda: mimo.mimo_attn_page_fork(refs, table, ints([0]).cuda(), table_out=table[:1]),
                    lambda: mimo.mimo_attn_page_compact(refs, table, -1),
                    lambda: mimo.mimo_attn_page_copy(kp, vp, torch.zeros((2, 2), device="cuda"))):
            with pytest.raises((ValueError, TypeError, RuntimeError)) as e:
                bad()
            said.append((type(e.value), str(e.value)))
        return got, said, taken

    real = mimo._fast
    a, said_a, taken = calls(True)
    assert sum(r is not None for r in taken) >= 9  # the native calls did run
    b, said_b, _ = calls(False)
    assert said_a == said_b
    for p, q in zip(a, b):
        assert (p is None and q is None) or (p.dtype == q.dtype and torch.equal(p.nan_to_num(), q.nan_to_num()))


# ------------------------------------------------------------------ a run of them together


@pytest.mark.parametrize("window,ps", [(0, 16), (129, 16), (129, 64)])
def test_a_serving_run(window, ps):
    """Prompts in chunks, single tokens, drafts taken back, beams forked, sequences ended and
    the pool compacted, each step's outputs against the oracle on a dense record of what
    every sequence holds."""
    hq, hkv, B, layers, theta = 8, 2, 5, 2, 10000.0
    r = random.Random(window + ps)
    g = torch.Generator().manual_seed(window + ps)
    cache = PagedCache(layers, 160 if ps == 16 else 48, ps, B, 64, hkv, window=window, rollback=4)
    sinks = torch.randn(hq, generator=g).cuda()
    seen = [[[] for _ in range(layers)] for _ in range(B)]  # (rotated k, v) rows per slot and layer
    lens = [0] * B
    for step in range(14):
        news = [[40, 0, 17, 130, 1], [60, 33, 1, 1, 1], [1] * 5, [3, 5, 1, 2, 4]][step % 4]
        news = [0 if lens[b] + n > 300 else n for b, n in enumerate(news)]
        nt = sum(news)
        cache.extend(ints(news).cuda())
        old, lens = lens, [a + n for a, n in zip(lens, news)]
        if nt:
            cu = [0]
            for n in news:
                cu.append(cu[-1] + n)
            for layer in range(layers):
                q, k, v = (torch.randn((nt, h, d), generator=g).to(torch.bfloat16) for h, d in ((hq, 192), (hkv, 192), (hkv, 128)))
                out, lse = cache.attend(layer, q.cuda(), k.cuda(), v.cuda(), ints(cu).cuda(), max(news), sinks, theta)
                # the oracle reads what the cache stores: bf16 rotated keys
                rq, rk, _ = paged.paged_append(q, k, v, torch.zeros(0, ps, hkv, 192), torch.zeros(0, ps, hkv, 128),
                                               [[-1] * 64] * B, cu, lens, theta)
                rq = torch.from_numpy(rq).to(torch.bfloat16)
                for b in range(B):
                    pos = np.arange(old[b], lens[b])
                    rows = slice(cu[b], cu[b + 1])
                    turned = torch.from_numpy(paged.rope(k[rows], pos, theta)).to(torch.bfloat16)
                    seen[b][layer] += list(zip(turned, v[rows]))
                width = max(1, -(-max(lens) // ps))
                kp = torch.zeros((B * width, ps, hkv, 192), dtype=torch.bfloat16)
                vp = torch.zeros((B * width, ps, hkv, 128), dtype=torch.bfloat16)
                for b in range(B):
                    for p, (kk, vv) in enumerate(seen[b][layer]):
                        kp[b * width + p // ps, p % ps], vp[b * width + p // ps, p % ps] = kk, vv
                dense = [[b * width + j for j in range(width)] for b in range(B)]
                want, want_lse, mass = paged.paged_attention(rq, kp, vp, dense, cu, lens, window, sinks.cpu())
                # on top of the module's bound: a rotated value may sit one bf16 step off where the
                # rounding of fp32 and fp64 differ, which moves a score by at most 2^-7 s |q| |k| < 0.03
                # for a whole row at once; the rows' mean effect is far below, 0.03 bounds it
                assert np.all(np.abs(P.to64(out) - want) <= 2.0 ** -7 * (mass + 2 * np.abs(want)) + 0.06 * mass + 1e-6)
                assert np.max(np.abs(P.to64(lse) - want_lse)) <= 0.031
        if step % 4 == 3:  # drafts: some are taken back
            lens = [max(o, n - r.randint(0, 2)) for o, n in zip(old, lens)]
            cache.truncate(ints(lens).cuda())
            seen = [[x[:L] for x in s] for s, L in zip(seen, lens)]
        if step % 5 == 4:
            parent = [0, 0, -1, 3, 1] if step % 2 else [0, 1, 1, 2, 4]
            cache.fork(ints(parent).cuda())
            lens = [lens[p] if p >= 0 else 0 for p in parent]
            seen = [[list(x) for x in seen[p]] if p >= 0 else [[] for _ in range(layers)] for p in parent]
        if step % 3 == 2:
            assert cache.compact(50).tolist()[1] == int((cache.page_refs > 0).sum())
        assert cache.seqlens.tolist() == lens
        held = torch.bincount(cache.block_table[cache.block_table >= 0].flatten().long(), minlength=cache.page_refs.numel())
        assert torch.equal(held.int(), cache.page_refs)
    mimo.mimo_attn_device_status()
    # more pages than the pool has: nothing changes
    before = cache.block_table.clone(), cache.page_refs.clone()
    info = cache.extend(ints([600] * B).cuda())
    assert info[0] > 0 and cache.seqlens.tolist() == lens
    assert torch.equal(cache.block_table, before[0]) and torch.equal(cache.page_refs, before[1])


def test_the_cache_keeps_its_sequences_through_bad_requests():
    """Past the table's width, a negative length, a parent that is no slot: recorded, the
    rest goes on, nothing is lost."""
    cache = PagedCache(1, 32, 16, 3, 4, 1)
    cache.extend(ints([20, 30, 5]).cuda())
    mimo.mimo_attn_device_status()
    for call, lens in ((lambda: cache.extend(ints([1, 100, 1]).cuda()), [21, 30, 6]),
                       (lambda: cache.truncate(ints([21, -4, 2]).cuda()), [21, 30, 2]),
                       (lambda: cache.fork(ints([1, 7, 0]).cuda()), [30, 0, 21])):
        call()
        with pytest.raises(mimo.MimoAttnError) as e:
            mimo.mimo_attn_device_status()
        assert e.value.status == mimo.MIMO_ERR_INVALID_ARG
        assert cache.seqlens.tolist() == lens
        held = [sum(x >= 0 for x in row) for row in cache.block_table.tolist()]
        assert held == [-(-n // 16) for n in lens] and int(cache.page_refs.sum()) == sum(held)


def test_attend_after_an_extend_without_room_writes_nothing():
    """Neither where the pool lacks pages nor in the sequence that would pass its table: the
    keys and values that are there stay, the rows of the output too, and it is recorded."""
    g = torch.Generator().manual_seed(3)

    def chunk(n):
        return [torch.randn((n, h, d), generator=g).to(torch.bfloat16).cuda() for h, d in ((8, 192), (2, 192), (2, 128))]

    for pool, news, skipped in ((6, [30, 30], [0, 1]), (40, [30, 50], [1])):
        cache = PagedCache(1, pool, 16, 2, 5, 2)
        cu = ints([0, 40, 80]).cuda()
        cache.extend(ints([40, 40]).cuda())
        cache.attend(0, *chunk(80), cu, 40, None, 1e4)
        mimo.mimo_attn_device_status()
        k, v = cache.k_pages.clone(), cache.v_pages.clone()
        cache.extend(ints(news).cuda())
        cu = ints([0, news[0], sum(news)]).cuda()
        try:
            mimo.mimo_attn_device_status()
            assert skipped == [0, 1]
        except mimo.MimoAttnError:
            assert skipped == [1]
        cache.attend(0, *chunk(sum(news)), cu, max(news), None, 1e4)
        with pytest.raises(mimo.MimoAttnError) as e:
            mimo.mimo_attn_device_status()
        assert e.value.status == mimo.MIMO_ERR_INVALID_ARG
        for b in skipped:
            assert cache.seqlens[b] == 40
            held = cache.block_table[b, :3].long()
            assert torch.equal(cache.k_pages[0, held], k[0, held]) and torch.equal(cache.v_pages[0, held], v[0, held])
        # the next step goes on
        cache.extend(ints([0, 1] if skipped == [1] else [8, 8]).cuda())
        n = 1 if skipped == [1] else 16
        cu = ints([0, 0, 1] if skipped == [1] else [0, 8, 16]).cuda()
        out, _ = cache.attend(0, *chunk(n), cu, min(n, 8), None, 1e4)
        mimo.mimo_attn_device_status()
        assert torch.isfinite(out).all()


def test_a_windowed_cache_goes_back_more_than_once():
    """Down to the length before the last extend (less the rollback), in steps: what the
    queries from there on see is still held, in the same pages."""
    W, ps, rollback = 129, 16, 5
    cache = PagedCache(1, 64, ps, 2, 40, 1, window=W, rollback=rollback)
    cache.extend(ints([400, 300]).cuda())
    cache.extend(ints([100, 60]).cuda())
    table = cache.block_table.clone()
    for back in ([500, 360], [430, 330], [400, 300], [395, 295]):
        cache.truncate(ints(back).cuda())
        assert cache.seqlens.tolist() == back
        for b, L in enumerate(back):
            for j in range((L - W + 1) // ps, -(-L // ps)):
                assert table[b, j] >= 0 and cache.block_table[b, j] == table[b, j]
            assert (cache.block_table[b, -(-L // ps):] < 0).all()
    cache.truncate(ints([0, 0]).cuda())
    assert int(cache.page_refs.sum()) == 0 and (cache.block_table < 0).all()
    cache.extend(ints([40, 1]).cuda())
    assert (cache.block_table >= 0).sum().item() == 4
    mimo.mimo_attn_device_status()


def test_arguments_that_the_native_call_leaves_to_the_binding():
    x = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in build([40], [3], 0, 16, 8, 2, 5).items()}
    args = [x[k] for k in ("q", "kp", "vp", "table", "cu", "lens", "most", "window", "sinks")]
    with pytest.raises(TypeError, match="out must be"):
        mimo.mimo_attn_paged_attention(*args, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="out must be"):
        mimo.mimo_attn_paged_attention(*args, out=torch.empty((3, 8, 128), dtype=torch.float16, device="cuda"))
    for big in (2 ** 31, 2 ** 32 + 3, 2 ** 70):
        with pytest.raises(ValueError, match="max_seqlen_q"):
            mimo.mimo_attn_paged_attention(*args[:6], big, *args[7:])
    want = mimo.mimo_attn_paged_attention(*args)
    got = mimo.mimo_attn_paged_attention(*args[:6], np.int64(3), *args[7:], return_lse=1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a scale in a tensor, changed between two calls
    scale, side = torch.tensor(0.5), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    seen = []
    for v in (0.5, 0.05):
        scale.fill_(v)
        seen.append(mimo.mimo_attn_paged_attention(*args, softmax_scale=scale, stream=side)[0])
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(seen[-1], mimo.mimo_attn_paged_attention(*args, softmax_scale=v)[0])
    assert not torch.equal(*seen)


@pytest.mark.parametrize("n,window", [(1, 0), (1, 129), (5, 0), (40, 0), (40, 129)])
def test_after_a_recorded_timeout_nothing_is_written(n, window):
    x = build([300, 60], [n, n], window, 16, 16, 1, seed=2)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    out = torch.full((2 * n, 16, 128), 7.0, device="cuda")
    lse = torch.full((16, 2 * n), 7.0, device="cuda")
    call = lambda: mimo.mimo_attn_paged_attention(dev["q"], dev["kp"], dev["vp"], dev["table"], dev["cu"], dev["lens"],  # noqa: E731
                                                  n, window, dev["sinks"], out=out, lse=lse)
    mimo.mimo_attn_set_device_status(mimo.MIMO_ERR_TIMEOUT)
    call()
    with pytest.raises(mimo.MimoAttnError) as e:
        mimo.mimo_attn_device_status()
    assert e.value.status == mimo.MIMO_ERR_TIMEOUT
    assert torch.all(out == 7) and torch.all(lse == 7)
    call()
    mimo.mimo_attn_device_status()
    check(out, lse, oracle_of(x))


def test_many_sequences():
    """More sequences than a CTA has threads, most of them without new tokens."""
    r = random.Random(1)
    lens = [r.randint(1, 40) for _ in range(900)]
    for n in (1, 3, 20):
        for window in (0, 9):
            news = [min(L, n) if r.random() < 0.1 else 0 for L in lens]
            news[-1] = min(lens[-1], n)
            x = build(lens, news, window, 16, 4, 1, seed=n)
            x["most"] = n
            check(*attend(x), oracle_of(x))


def test_a_step_captured_in_a_graph_and_replayed():
    """extend, append, attention and truncate of a decode step, captured once; each replay
    against an eager twin of the cache."""
    hq, hkv, B, ps = 16, 1, 3, 16
    g = torch.Generator().manual_seed(0)
    twins = [PagedCache(1, 64, ps, B, 16, hkv) for _ in range(2)]
    sinks = torch.randn(hq, generator=g).cuda()
    cu = ints([0, 1, 2, 3]).cuda()
    one = ints([1, 1, 1]).cuda()
    rows = lambda: [torch.randn((B, h, d), generator=g).to(torch.bfloat16).cuda() for h, d in ((hq, 192), (hkv, 192), (hkv, 128))]  # noqa: E731
    prompt = [torch.randn((40 + 17 + 3, h, d), generator=g).to(torch.bfloat16).cuda() for h, d in ((hq, 192), (hkv, 192), (hkv, 128))]

    def step(cache, q, k, v):
        cache.extend(one)
        return cache.attend(0, q, k, v, cu, 1, sinks, 1e4)

    for c in twins:
        c.extend(ints([40, 17, 3]).cuda())
        c.attend(0, *prompt, ints([0, 40, 57, 60]).cuda(), 40, sinks, 1e4)
    buf = rows()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm-up, undone again
        step(twins[0], *buf)
        twins[0].truncate(ints([40, 17, 3]).cuda())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(twins[0], *buf)
    for _ in range(20):
        new = rows()
        for b, n in zip(buf, new):
            b.copy_(n)
        graph.replay()
        want, want_lse = step(twins[1], *new)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert torch.equal(twins[0].block_table, twins[1].block_table)
        assert torch.equal(twins[0].seqlens, twins[1].seqlens)
    mimo.mimo_attn_device_status()
    graph.reset()
