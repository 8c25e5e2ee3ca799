"""The calls on a paged cache through the bounds-checked build of the library.

Run as its own process with MIMO_ATTN_CHECKED=1 (tests/test_checked_paged_gpu.py
does so).  Every kernel of them runs, at small sizes and at large ones; each call
must leave the device status word clear and record no bounds site, and at the
small sizes match the fp64 oracle.
"""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import global_attention_swa_b200 as mimo  # noqa: E402
from global_attention_swa_b200.paged_cache import PagedCache  # noqa: E402
from oracle import paged  # noqa: E402
from tests import test_paged_gpu as T  # noqa: E402

# lengths, new tokens, window, page size, query heads, key/value heads: one token
# (decode kernel), a short window (one block and two), one tile, two tiles, and
# sequences whose items are divided among CTAs
SMALL = [
    ([70, 1, 16, 0], [1, 1, 1, 0], 0, 16, 16, 4), ([300, 129, 5], [1, 1, 1], 129, 32, 64, 4),
    ([200, 33], [5, 3], 0, 16, 32, 2), ([400, 64], [60, 64], 129, 16, 64, 4), ([90, 20], [8, 7], 40, 16, 64, 4),
    ([900, 77, 1], [130, 77, 1], 0, 48, 8, 2), ([900], [300], 0, 16, 64, 4), ([700, 300], [100, 9], 300, 64, 12, 4),
]
LARGE = [
    ([32768] * 8, [1] * 8, 0, 64, 64, 4), ([20000 + 77 * i for i in range(16)], [4] * 16, 0, 64, 64, 4),
    ([16384], [1024], 0, 64, 64, 4), ([5000, 1, 700, 4096], [2500, 1, 9, 600], 129, 64, 64, 4),
]


def clean(what):
    st = mimo.lib.mimo_attn_device_status(None)
    site = mimo.mimo_attn_checked_site()
    assert st == mimo.MIMO_OK and site == 0, f"{what}: status {st}, bounds site {site}"


def main():
    assert mimo.CHECKED and mimo.mimo_attn_is_checked_build(), "not the checked build"
    torch.cuda.set_device(0)
    for case in SMALL:
        x = T.build(*case, seed=len(case[0]) + case[2])
        ref = paged.paged_attention(x["q"], x["kp"], x["vp"], x["table"].tolist(), x["cu"].tolist(), x["lens"].tolist(),
                                    x["window"], x["sinks"])
        for odt in (torch.float32, torch.bfloat16):
            out, lse = T.attend(x, out_dtype=odt)
            clean(f"attention {case}")
            T.check(out, lse, ref)
    for lens, news, window, ps, hq, hkv in LARGE:  # results: the parity tests
        pages = [-(-L // ps) for L in lens]
        order = torch.randperm(sum(pages), device="cuda", dtype=torch.int32)
        table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        cu = T.ints([sum(news[:i]) for i in range(len(news) + 1)]).cuda()
        randn = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)  # noqa: E731
        kp, vp, nt = randn(at, ps, hkv, 192), randn(at, ps, hkv, 128), sum(news)
        q = mimo.mimo_attn_paged_append(randn(nt, hq, 192), randn(nt, hkv, 192), randn(nt, hkv, 128), kp, vp, table, cu,
                                        T.ints(lens).cuda(), 1e6, 64)
        clean(f"append {lens[:3]}")
        out, lse = mimo.mimo_attn_paged_attention(q, kp, vp, table, cu, T.ints(lens).cuda(), max(news), window,
                                                  torch.zeros(hq, device="cuda"))
        clean(f"attention {lens[:3]}")
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # the bookkeeping: a cache's life, with sizes of one CTA and of a whole cluster
    for slots, width, pool in ((3, 5, 20), (200, 300, 50000)):
        cache = PagedCache(2, pool, 16, slots, width, 1, window=129, rollback=3)
        for n in (40, 1, 17):
            cache.extend(torch.full((slots,), n, dtype=torch.int32, device="cuda"))
            clean("extend")
        cache.truncate(cache.seqlens - 2)
        cache.fork(torch.arange(slots, dtype=torch.int32, device="cuda").clamp_(max=slots // 2))
        clean("truncate, fork")
        cache.extend(torch.ones(slots, dtype=torch.int32, device="cuda"))
        cache.compact(pool)
        clean("extend, compact")
        held = torch.bincount(cache.block_table[cache.block_table >= 0].flatten().long(), minlength=pool)
        assert torch.equal(held.int(), cache.page_refs)
    print("checked ok")


if __name__ == "__main__":
    main()
