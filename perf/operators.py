"""Cases of the paged-cache operators: attention of a chunk of new tokens over a
paged cache, the rotation and write of those tokens into the pages, and the
page bookkeeping (hold and release, fork, compact) with the page copies it asks
for.  Each case is run in a plain form of elementary torch operations or, with
``own`` set, through the framework's entry points.
"""

import math
import random

import torch

own = False

QK, V = 192, 128  # the framework's query/key and value head dimensions


# ------------------------------------------------------------------- cases
def listed():
    heads = dict(hq=64, hkv=4)
    return [
        # attention: seqs sequences whose lengths (the chunk included) lie in
        # len_lo..len_hi and whose chunks in new_lo..new_hi tokens.
        # A few short chats, one token each: latency counts.
        dict(name="attend_chat_token", op="attend", **heads, seqs=3, len_lo=60, len_hi=700, new_lo=1, new_hi=1,
             page=16, window=0, ragged=1),
        # One serving step of a global layer: a batch of single tokens over long ragged caches.
        dict(name="attend_batch_token", op="attend", **heads, seqs=64, len_lo=1024, len_hi=32768, new_lo=1,
             new_hi=1, page=64, window=0, ragged=2),
        # The same step in a sliding-window layer: pages behind the window were released.
        dict(name="attend_batch_token_window", op="attend", **heads, seqs=64, len_lo=1024, len_hi=32768, new_lo=1,
             new_hi=1, page=16, window=129, ragged=3),
        # Drafted tokens to be checked: a handful for each sequence.
        dict(name="attend_draft_check", op="attend", **heads, seqs=32, len_lo=512, len_hi=16384, new_lo=1,
             new_hi=6, page=32, window=0, ragged=4),
        # The next chunk of a long prompt in a global layer: bound by the matrix products.
        dict(name="attend_prompt_chunk", op="attend", **heads, seqs=1, len_lo=32768, len_hi=32768, new_lo=2048,
             new_hi=2048, page=64, window=0, ragged=5),
        # A mixed step of a sliding-window layer: chunks of prompts beside empty and single-token ones.
        dict(name="attend_mixed_window", op="attend", **heads, seqs=9, len_lo=1, len_hi=5000, new_lo=0,
             new_hi=1500, page=16, window=129, ragged=6),
        # append: one new token of each running sequence, and the chunks of several prompts.
        dict(name="append_tokens", op="append", **heads, seqs=48, len_lo=1, len_hi=16384, new_lo=1, new_hi=1,
             page=64, rotary=192, ragged=7),
        dict(name="append_chunks", op="append", **heads, seqs=5, len_lo=300, len_hi=4100, new_lo=200, new_hi=3500,
             page=64, rotary=64, ragged=8),
        # pages: the hold-and-release of one serving step over a large pool (some
        # sequences end, some grow, a window leaves pages behind) ...
        dict(name="pages_step", op="pages_step", seqs=64, pool=40000, table=1024, page=64, ragged=9),
        # ... beams that fork: tables gathered, the shared last page of each beam copied in every layer ...
        dict(name="pages_fork", op="pages_fork", hkv=4, layers=6, prompts=8, beams=4, len_lo=100, len_hi=2000,
             page=64, pool=1600, ragged=10),
        # ... and compaction of a pool with holes: a small one, and one of several layers.
        dict(name="pages_compact_small", op="pages_compact", hkv=4, layers=1, seqs=6, held=90, pool=256, page=16,
             moves=24, ragged=11),
        dict(name="pages_compact_large", op="pages_compact", hkv=4, layers=6, seqs=48, held=2000, pool=4096, page=64,
             moves=900, ragged=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend"] * 6 + ["append"] * 2 + ["pages_step", "pages_fork", "pages_compact"])
    hq, hkv = rng.choice([(64, 4), (64, 4), (64, 4), (16, 1), (32, 4), (64, 8), (24, 2), (6, 6)])
    page = rng.choice([16, 32, 48, 64, 128])
    c = dict(op=op, ragged=rng.randrange(1 << 20))
    if op == "attend":
        kind = rng.choice(["token", "token", "draft", "chunk", "mixed"])
        window = rng.choice([0, 0, 129, 129, _log(rng, 1, 2000)])
        if kind == "token":
            seqs, hi, new = _log(rng, 1, 64), _log(rng, 16, 32768), (1, 1)
        elif kind == "draft":
            seqs, hi, new = _log(rng, 1, 32), _log(rng, 64, 16384), (1, rng.randint(2, 12))
        elif kind == "chunk":
            seqs, hi = 1, _log(rng, 600, 32768)
            n = min(hi, _log(rng, 17, 2000))
            new = (n, n)
        else:
            seqs, hi, new = rng.randint(2, 10), _log(rng, 100, 5000), (0, _log(rng, 20, 1500))
        return dict(c, hq=hq, hkv=hkv, seqs=seqs, len_lo=max(1, hi // 16) if kind != "chunk" else hi, len_hi=hi,
                    new_lo=new[0], new_hi=new[1], page=page, window=window)
    if op == "append":
        seqs = _log(rng, 1, 64)
        new = rng.choice([1, _log(rng, 1, 8000 // seqs)])
        return dict(c, hq=hq, hkv=hkv, seqs=seqs, len_lo=1, len_hi=max(new, _log(rng, 30, 16000 // seqs)), new_lo=1,
                    new_hi=new, page=page, rotary=rng.choice([192, 64, 128, 60]))
    if op == "pages_step":
        seqs, table = _log(rng, 1, 200), _log(rng, 8, 1024)
        return dict(c, seqs=seqs, table=table, pool=max(2 * seqs, min(seqs * table, _log(rng, 100, 40000))), page=page)
    if op == "pages_fork":
        prompts, beams, hi = rng.randint(1, 8), rng.randint(2, 4), _log(rng, 40, 1500)
        need = prompts * (beams + 1) * (hi // page + 2)
        return dict(c, hkv=hkv, layers=rng.randint(1, 6), prompts=prompts, beams=beams, len_lo=1 + hi // 8, len_hi=hi,
                    page=page, pool=need + rng.randint(0, 200))
    pool = _log(rng, 40, 4096)
    held = max(4, int(pool * rng.uniform(0.2, 0.7)))
    return dict(c, hkv=hkv, layers=rng.randint(1, 4), seqs=_log(rng, 1, 48), held=held, pool=pool, page=rng.choice([16, 48, 64]),
                moves=_log(rng, 2, 800))


# ------------------------------------------------------------------- sizes that follow from a case alone
def _lengths(case):
    """(length, new tokens) of each sequence: ragged, the same for every seed."""
    r = random.Random(case["ragged"])
    got = []
    for _ in range(case["seqs"]):
        total = r.randint(case["len_lo"], case["len_hi"])
        got.append((total, min(total, r.randint(case["new_lo"], case["new_hi"]))))
    if not any(n for _, n in got):
        got[0] = (got[0][0], 1)
    return got


def _visible(total, new, window):
    """Query-key pairs of one sequence, and the keys that at least one query sees."""
    first = total - new
    if new == 0:
        return 0, 0
    if not window:
        return sum(range(first + 1, total + 1)), total
    lo = max(0, first - window + 1)
    return sum(min(window, p + 1) for p in range(first, total)), total - lo


def work(case):
    op, page = case["op"], case.get("page")
    if op == "attend":
        hq, hkv = case["hq"], case["hkv"]
        pairs = keys = tokens = pages = 0
        for total, new in _lengths(case):
            p, k = _visible(total, new, case["window"])
            pairs, keys, tokens, pages = pairs + p, keys + k, tokens + new, pages + -(-k // page)
        by = tokens * hq * (QK * 2 + V * 2 + 4) + keys * hkv * (QK + V) * 2 + 4 * (pages + 2 * case["seqs"] + 1 + hq)
        return {"bytes": by, "flops": 2 * (QK + V) * hq * pairs}
    if op == "append":
        tokens = sum(n for _, n in _lengths(case))
        row = case["hq"] * QK * 2 + case["hkv"] * (QK + V) * 2
        return {"bytes": 2 * tokens * row + 4 * (3 * case["seqs"] + 1), "flops": 3 * tokens * (case["hq"] + case["hkv"]) * case["rotary"]}
    if op == "pages_step":  # counts and table, in and out
        return {"bytes": 8 * (case["pool"] + case["seqs"] * case["table"]) + 12 * case["seqs"], "flops": 0}
    page_bytes = 2 * page * case["hkv"] * (QK + V) * case["layers"]
    if op == "pages_fork":
        lens, width = _fork_lengths(case)
        copies = sum(1 for n in lens if n % page) * case["beams"]
        return {"bytes": 2 * copies * page_bytes + 8 * (case["pool"] + case["prompts"] * (case["beams"] + 1) * width), "flops": 0}
    moved = min(case["moves"], _holes(case))
    return {"bytes": 2 * moved * page_bytes + 16 * case["pool"], "flops": 0}


def _fork_lengths(case):
    r = random.Random(case["ragged"])
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["prompts"])]
    return lens, case["len_hi"] // case["page"] + 2


def _held(case):
    """The pages in use of a pool with holes."""
    return random.Random(case["ragged"]).sample(range(case["pool"]), case["held"])


def _holes(case):
    return sum(1 for p in _held(case) if p >= case["held"])


# ------------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("attend", "append"):
        hq, hkv, page, window = case["hq"], case["hkv"], case["page"], case.get("window", 0)
        lens = _lengths(case)
        width = max(-(-t // page) for t, _ in lens) + 1
        cu = [0]
        rows, need = [], 0
        for total, new in lens:
            cu.append(cu[-1] + new)
            lo = max(0, total - new - window + 1) // page if window else 0
            rows.append((lo, -(-total // page)))
            need += rows[-1][1] - lo
        pool = need + need // 16 + 2
        order = r.sample(range(pool), need)
        table = []
        for lo, hi in rows:
            table.append([-1] * lo + [order.pop() for _ in range(hi - lo)] + [-1] * (width - hi))
        tokens = cu[-1]
        s.update(q=_normal(g, tokens, hq, QK), kp=_normal(g, pool, page, hkv, QK), vp=_normal(g, pool, page, hkv, V),
                 table=_ints(table), cu=_ints(cu), lens=_ints([t for t, _ in lens]), most=max(n for _, n in lens),
                 longest=max(t for t, _ in lens))
        if op == "attend":
            s["sinks"] = torch.randn(hq, generator=g, device="cuda")
        else:
            s.update(k=_normal(g, tokens, hkv, QK), v=_normal(g, tokens, hkv, V), theta=10000.0)
        return s
    pool, page = case["pool"], case["page"]
    if op == "pages_step":
        # Held ranges before and after the step: most sequences grow by a page or
        # less, some end, some start; every third one lives in a window.
        seqs, width = case["seqs"], case["table"]
        most = max(1, min(width, 3 * pool // (4 * seqs)))
        free = r.sample(range(pool), pool)
        refs = [0] * pool
        table, first, after = [], [], []
        for b in range(seqs):
            held = 0 if b % 8 == 7 else r.randint(0, most)
            lo = r.randint(0, held) if b % 3 == 0 else 0
            row = [-1] * width
            for j in range(lo, held):
                row[j] = free.pop()
                refs[row[j]] = 1
            table.append(row)
            end = 0 if b % 11 == 5 else min(width, held + r.randint(0, 1 + most // 8)) * page - r.randint(0, page - 1)
            after.append(max(0, end))
            first.append(min(max(0, end), lo * page + r.randint(0, page)) if lo else 0)
        s.update(refs=_ints(refs), table=_ints(table), first=_ints(first), lens=_ints(after))
        return s
    layers, hkv = case["layers"], case["hkv"]
    s.update(kp=_normal(g, layers, pool, page, hkv, QK), vp=_normal(g, layers, pool, page, hkv, V))
    if op == "pages_fork":
        lens, width = _fork_lengths(case)
        order = r.sample(range(pool), pool)
        refs, table, parent = [0] * pool, [], []
        for b, n in enumerate(lens):
            row = [order.pop() for _ in range(-(-n // page))]
            for p in row:
                refs[p] = 1
            table.append(row + [-1] * (width - len(row)))
        slots = case["prompts"] * case["beams"]
        table += [[-1] * width for _ in range(slots - len(table))]
        parent = [i // case["beams"] for i in range(slots)]
        r.shuffle(parent)
        before = [lens[p] for p in parent]
        s.update(refs=_ints(refs), table=_ints(table), parent=_ints(parent), before=_ints(before),
                 after=_ints([n + 1 for n in before]))
        return s
    held = list(_held(case))
    r.shuffle(held)
    seqs = case["seqs"]
    each = -(-len(held) // seqs)
    refs, table = [0] * pool, []
    for b in range(seqs):
        row = held[b * each:(b + 1) * each]
        table.append(row + [-1] * (each + 1 - len(row)))
        for p in row:
            refs[p] += 1
    for b in range(1, seqs, 4):  # some share the first pages of the row before
        for j in range(min(3, each)):
            old, new = table[b][j], table[b - 1][j]
            if old >= 0 and new >= 0 and refs[old] == 1:
                table[b].append(old)  # kept, further back
                table[b][j] = new
                refs[new] += 1
    width = max(len(x) for x in table)
    table = [x + [-1] * (width - len(x)) for x in table]
    s.update(refs=_ints(refs), table=_ints(table))
    return s


# ------------------------------------------------------------------- the plain forms
def _token_places(cu, lens, tokens):
    """Of each packed token: its sequence, its place in the chunk and its position."""
    t = torch.arange(tokens, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True).clamp(max=lens.numel() - 1)
    i = t - cu[b].long()
    return b, i, lens[b].long() - (cu[b + 1] - cu[b]).long() + i


def _plain_attend(s):
    case = s["case"]
    hq, hkv, page, window = case["hq"], case["hkv"], case["page"], case["window"]
    q, table, cu, lens = s["q"], s["table"], s["cu"], s["lens"].long()
    tokens, seqs, group, most = q.shape[0], lens.numel(), hq // hkv, s["most"]
    new = (cu[1:] - cu[:-1]).long()
    # the pages that at least one query sees: of a window, those from its first key on
    wide = -(-s["longest"] // page)
    low = torch.zeros_like(lens)
    if window:
        low = (lens - new - window + 1).clamp(min=0) // page
        wide = min(wide, (most + window - 2) // page + 2)
    place = low[:, None] + torch.arange(wide, device=q.device)
    pages = table.gather(1, place.clamp(max=table.shape[1] - 1)).clamp(min=0).long()
    k = s["kp"][pages].reshape(seqs, -1, hkv, QK).permute(0, 2, 3, 1).float()
    v = s["vp"][pages].reshape(seqs, -1, hkv, V).permute(0, 2, 1, 3).float()
    keys = k.shape[-1]
    at = (cu[:-1].long()[:, None] + torch.arange(most, device=q.device)).clamp(max=tokens - 1)
    qp = q[at].reshape(seqs, most, hkv, group, QK).permute(0, 2, 1, 3, 4).reshape(seqs, hkv, most * group, QK).float()
    scores = (qp @ k).mul_(1.0 / math.sqrt(QK)).view(seqs, hkv, most, group, keys)
    pos = (lens - new - low * page)[:, None] + torch.arange(most, device=q.device)
    j = torch.arange(keys, device=q.device)
    hidden = j > pos[..., None]
    if window:
        hidden |= j <= pos[..., None] - window
    scores.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    sink = s["sinks"].view(1, hkv, 1, group, 1)
    top = torch.maximum(scores.amax(-1, keepdim=True), sink)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True) + torch.exp(sink - top)
    out = (weights.view(seqs, hkv, most * group, keys) @ v).view(seqs, hkv, most, group, V) / total
    lse = (top + torch.log(total))[..., 0]
    b, i, _ = _token_places(cu, lens, tokens)
    return out[b, :, i].reshape(tokens, hq, V).bfloat16(), lse[b, :, i].reshape(tokens, hq).t().contiguous()


def _plain_rotate(x, pos, theta, rotary):
    half = rotary // 2
    angle = pos.double()[:, None] * torch.pow(theta, -torch.arange(half, device=x.device, dtype=torch.float64) * 2 / rotary)
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, c, rest = x[..., :half].float(), x[..., half:rotary].float(), x[..., rotary:]
    return torch.cat([(a * cos - c * sin).to(x.dtype), (c * cos + a * sin).to(x.dtype), rest], -1)


def _plain_append(s):
    case = s["case"]
    b, _, pos = _token_places(s["cu"], s["lens"], s["q"].shape[0])
    page, slot = s["table"][b, pos // case["page"]].long(), pos % case["page"]
    s["kp"][page, slot] = _plain_rotate(s["k"], pos, s["theta"], case["rotary"])
    s["vp"][page, slot] = s["v"]
    return _plain_rotate(s["q"], pos, s["theta"], case["rotary"]), s["kp"], s["vp"]


def _kth(flags, size):
    """The indexes at which flags is set, in rising order, then -1; size + 1 entries, the last one always -1."""
    at = torch.where(flags, torch.cumsum(flags, 0) - 1, size).clamp(max=size)
    found = torch.full((size + 1,), -1, dtype=torch.int64, device=flags.device)
    found.scatter_(0, at, torch.arange(flags.numel(), device=flags.device))
    found[size] = -1
    return found


def _plain_hold(refs, table, lens, page, first=None, write_from=None):
    """Exactly the pages of positions [first, lens) are held afterwards, those that
    reach past write_from by this sequence alone."""
    pool, width = refs.numel(), table.shape[1]
    j = torch.arange(width, device=table.device)
    lo = (torch.zeros_like(lens) if first is None else first).long() // page
    hi = (lens.long() + page - 1) // page
    wanted = (j >= lo[:, None]) & (j < hi[:, None])
    has = table >= 0
    drop = has & ~wanted
    count = refs.clone().index_add_(0, table.clamp(min=0).flatten().long(), -drop.flatten().int())
    free = count == 0
    fresh = wanted & ~has
    split = torch.zeros_like(fresh)
    if write_from is not None:
        split = wanted & has & (j >= (write_from.long() // page)[:, None]) & (count[table.clamp(min=0).long()] > 1)
    take = (fresh | split).flatten()
    rank = torch.cumsum(take, 0) - 1
    missing = (take.sum() - free.sum()).clamp(min=0)
    ok = missing == 0
    given = _kth(free, pool)[rank.clamp(min=0, max=pool)].view_as(table).int()
    moved = torch.where(take.view_as(table), given, torch.where(drop, torch.full_like(table, -1), table))
    table_out = torch.where(ok, moved, table)
    after = count.index_add(0, table.clamp(min=0).flatten().long(), -split.flatten().int())
    after = after.index_add_(0, given.clamp(min=0).flatten().long(), take.int())
    refs_out = torch.where(ok, after, refs)
    copied = split & ((j * page) < (lens if write_from is None else write_from)[:, None]) & ok
    pair = torch.stack([table, given], -1)
    pair = torch.where(copied[..., None], pair, torch.full_like(pair, -1)).amax(1)
    info = torch.stack([missing, (refs_out == 0).sum()]).int()
    return refs_out, table_out, pair, info


def _plain_fork(refs, table, parent):
    rows = table[parent.clamp(min=0).long()]
    out = torch.where((parent >= 0)[:, None], rows, torch.full_like(rows, -1))
    count = refs.clone()
    count.index_add_(0, table.clamp(min=0).flatten().long(), -(table >= 0).flatten().int())
    count.index_add_(0, out.clamp(min=0).flatten().long(), (out >= 0).flatten().int())
    return count, out


def _plain_compact(refs, table, most):
    pool = refs.numel()
    used = refs > 0
    total = used.sum()
    at = torch.arange(pool, device=refs.device)
    src, dst = _kth(used & (at >= total), most)[:most], _kth(~used & (at < total), most)[:most]
    moves = torch.stack([src, dst], -1).int()
    real = src >= 0
    to = torch.arange(pool + 1, device=refs.device)
    to.scatter_(0, torch.where(real, src, pool), torch.where(real, dst, pool))
    table_out = torch.where(table >= 0, to[table.clamp(min=0).long()], table.long()).int()
    # a page that moved leaves its old place empty, one that stayed keeps its own
    refs_out = torch.where(to[:pool] != at, torch.zeros_like(refs), refs)
    refs_out = refs_out.index_add(0, dst.clamp(min=0), torch.where(real, refs[src.clamp(min=0)], torch.zeros_like(refs[:1])))
    return refs_out, table_out, moves, torch.stack([real.sum(), total]).int()


def _plain_copy(kp, vp, moves):
    """Pages moves[:, 0] over pages moves[:, 1]; a row of -1 is none (it repeats the first real one, or page 0 onto itself)."""
    real = moves[:, :1] >= 0
    stand = moves[real.int().argmax(0)].clamp(min=0)
    src, dst = torch.where(real, moves, stand).long().unbind(1)
    kp[:, dst] = kp[:, src]
    vp[:, dst] = vp[:, src]


# ------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    op, page = case["op"], case["page"]
    if own:
        import global_attention_swa_b200 as mimo

        if op == "attend":
            return mimo.mimo_attn_paged_attention(s["q"], s["kp"], s["vp"], s["table"], s["cu"], s["lens"], s["most"],
                                                  case["window"], s["sinks"])
        if op == "append":
            q = mimo.mimo_attn_paged_append(s["q"], s["k"], s["v"], s["kp"], s["vp"], s["table"], s["cu"], s["lens"],
                                            s["theta"], case["rotary"])
            return q, s["kp"], s["vp"]
        if op == "pages_step":
            refs, table, _, info = mimo.mimo_attn_page_hold(s["refs"], s["table"], s["lens"], page, first=s["first"])
            return refs, table, info
        if op == "pages_fork":
            refs, table = mimo.mimo_attn_page_fork(s["refs"], s["table"], s["parent"])
            refs, table, moves, info = mimo.mimo_attn_page_hold(refs, table, s["after"], page, write_from=s["before"])
            mimo.mimo_attn_page_copy(s["kp"], s["vp"], moves)
            return refs, table, moves, info, s["kp"], s["vp"]
        refs, table, moves, info = mimo.mimo_attn_page_compact(s["refs"], s["table"], case["moves"])
        mimo.mimo_attn_page_copy(s["kp"], s["vp"], moves)
        return refs, table, moves, info, s["kp"], s["vp"]
    if op == "attend":
        return _plain_attend(s)
    if op == "append":
        return _plain_append(s)
    if op == "pages_step":
        refs, table, _, info = _plain_hold(s["refs"], s["table"], s["lens"], page, first=s["first"])
        return refs, table, info
    if op == "pages_fork":
        refs, table = _plain_fork(s["refs"], s["table"], s["parent"])
        refs, table, moves, info = _plain_hold(refs, table, s["after"], page, write_from=s["before"])
    else:
        refs, table, moves, info = _plain_compact(s["refs"], s["table"], case["moves"])
    _plain_copy(s["kp"], s["vp"], moves)
    return refs, table, moves, info, s["kp"], s["vp"]


# ------------------------------------------------------------------- in 64 bits, from the definition
def exact(case, seed):
    if case["op"] not in ("attend", "append"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    q, kp, vp, page = s["q"], s["kp"], s["vp"], case["page"]
    hq, hkv = case["hq"], case["hkv"]
    group = hq // hkv
    cu, table = s["cu"].tolist(), s["table"].tolist()
    if case["op"] == "attend":
        out = torch.empty((q.shape[0], hq, V), dtype=torch.float64, device=q.device)
        lse = torch.empty((hq, q.shape[0]), dtype=torch.float64, device=q.device)
        for b, (total, new) in enumerate(_lengths(case)):
            if not new:
                continue
            lo = max(0, total - new - case["window"] + 1) if case["window"] else 0
            ids = torch.tensor(table[b][lo // page:-(-total // page)], device=q.device)
            cut = slice(lo % page, lo % page + total - lo)
            for h in range(hkv):
                k = kp[ids, :, h].flatten(0, 1)[cut].double()
                v = vp[ids, :, h].flatten(0, 1)[cut].double()
                for n0 in range(0, new, 512):  # queries n0.. of the chunk
                    n1 = min(new, n0 + 512)
                    x = q[cu[b] + n0:cu[b] + n1, h * group:(h + 1) * group].double()
                    z = torch.einsum("ngd,jd->ngj", x, k) / 192 ** 0.5
                    back = (total - new + torch.arange(n0, n1, device=q.device))[:, None] - torch.arange(lo, total, device=q.device)
                    seen = (back >= 0) & ((back < case["window"]) if case["window"] else True)
                    z = torch.where(seen[:, None], z, -torch.inf)
                    z = torch.cat([z, s["sinks"][h * group:(h + 1) * group].double()[None, :, None].expand(n1 - n0, -1, 1)], -1)
                    norm = torch.logsumexp(z, -1)
                    out[cu[b] + n0:cu[b] + n1, h * group:(h + 1) * group] = torch.einsum("ngj,jd->ngd", torch.exp(z[..., :-1] - norm[..., None]), v)
                    lse[h * group:(h + 1) * group, cu[b] + n0:cu[b] + n1] = norm.t()
        return out, lse
    rd = case["rotary"]
    freq = [s["theta"] ** (-2.0 * i / rd) for i in range(rd // 2)]
    freq = torch.tensor(freq, dtype=torch.float64, device=q.device)

    def turned(x, p):
        z = torch.complex(x[..., :rd // 2].double(), x[..., rd // 2:rd].double())
        z = z * torch.polar(torch.ones_like(freq), p * freq)
        return torch.cat([z.real, z.imag, x[..., rd:].double()], -1)

    qx, kx, vx = torch.empty(q.shape, dtype=torch.float64, device=q.device), kp.double(), vp.double()
    for b, (total, new) in enumerate(_lengths(case)):
        p = torch.arange(total - new, total, device=q.device)
        mine = slice(cu[b], cu[b + 1])
        qx[mine] = turned(q[mine], p[:, None, None].double())
        ids = torch.tensor(table[b], device=q.device)[p // page]
        kx[ids, p % page] = turned(s["k"][mine], p[:, None, None].double())
        vx[ids, p % page] = s["v"][mine].double()
    return qx, kx, vx
