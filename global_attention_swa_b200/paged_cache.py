"""A paged key/value cache of several layers, kept with the library's calls.

``PagedCache`` holds what a serving loop needs between steps: the pools of pages,
the block table, the pages' holder counts and the sequence lengths, all on the
device.  Nothing is read back to the host, so a step can be captured in a CUDA
graph; ``info`` holds what the last bookkeeping call reported.

A hybrid stack (MiMo-V2-Flash model doc, "Key features": sliding-window and
global layers, 5:1) keeps two: one for its global layers, and one with
``window`` set for its sliding-window layers, whose pages are released as the
window leaves them.

    cache = PagedCache(num_layers=8, num_pages=4096, page_size=64, num_seqs=32, max_pages=512)
    cache.extend(new_tokens)                      # int32 [num_seqs]: pages for the next step
    for layer in ...:
        out, lse = cache.attend(layer, q, k, v, cu_seqlens_q, max_new, sinks, rope_theta)
    cache.truncate(accepted)                      # rejected drafted tokens go
    cache.fork(parent)                            # beams: slot i goes on as parent[i] did
"""

from __future__ import annotations

import torch

import global_attention_swa_b200 as mimo


class PagedCache:
    """Pools k_pages [layers, num_pages, page_size, Hkv, 192] and v_pages [..., 128], and
    num_seqs sequence slots of at most max_pages pages, empty at first.

    ``window`` > 0 (the layers' sliding window) lets ``extend`` release the pages that no
    later query sees.  ``truncate`` can then take back the tokens of the last
    ``extend``, and ``rollback`` more: the pages that the windows of those would see are
    kept.  What an earlier ``extend`` released does not come back: going back in several
    steps, extending between, reaches no further."""

    def __init__(self, num_layers, num_pages, page_size, num_seqs, max_pages, num_heads_kv=4, head_dim_qk=192,
                 head_dim_v=128, window=0, rollback=0, device="cuda"):
        if min(num_layers, num_pages, page_size, num_seqs, max_pages, num_heads_kv) < 1:
            raise ValueError("sizes must be positive")
        if page_size % 16:
            raise ValueError("page_size must be a multiple of 16")
        if window < 0 or rollback < 0:
            raise ValueError("window and rollback must be >= 0")
        shape = (num_layers, num_pages, page_size, num_heads_kv)
        ints = dict(dtype=torch.int32, device=device)
        self.k_pages = torch.zeros((*shape, head_dim_qk), dtype=torch.bfloat16, device=device)
        self.v_pages = torch.zeros((*shape, head_dim_v), dtype=torch.bfloat16, device=device)
        self.page_refs = torch.zeros(num_pages, **ints)
        self.block_table = torch.full((num_seqs, max_pages), -1, **ints)
        self._spare_table = torch.empty_like(self.block_table)
        self.seqlens = torch.zeros(num_seqs, **ints)
        self.info = torch.zeros(2, **ints)
        self._attend = torch.zeros(num_seqs, **ints)  # what attend goes by: -1 since extend found no room
        self._kept = torch.zeros(num_seqs, **ints)  # first position whose page was never released
        self.page_size, self.window, self.rollback = page_size, window, rollback
        self.capacity = max_pages * page_size

    def _first(self):
        """First position that queries from ``rollback`` before the present lengths on see;
        never one already released."""
        if not self.window:
            return None
        return torch.maximum(self._kept, self.seqlens - (self.window - 1 + self.rollback))

    def _hold(self, lens, first, write_from):
        _, _, moves, _ = mimo.mimo_attn_page_hold(
            self.page_refs, self.block_table, lens, self.page_size, first=first, write_from=write_from,
            refs_out=self.page_refs, table_out=self.block_table, info=self.info)
        return moves

    def extend(self, new_tokens):
        """Pages for new_tokens [num_seqs] int32 more positions of each sequence, and its
        length advanced over them.  A page that a fork shares and that will be written
        is replaced by a copy, in every layer.  If the pool does not have the pages,
        nothing changes and ``info[0]`` says how many were missing; a sequence that
        would pass max_pages pages stays as it is and is recorded as an invalid
        argument in the device status.  ``attend`` skips sequences that were not
        extended, until they are, and records that too.  Returns ``info``."""
        lens = self.seqlens + new_tokens
        first = self._first()
        # a sequence without new tokens writes nothing and parts from no page
        moves = self._hold(lens, first, torch.where(new_tokens > 0, self.seqlens, self.capacity))
        mimo.mimo_attn_page_copy(self.k_pages, self.v_pages, moves)
        done = (self.info[0] == 0) & (lens >= 0) & (lens <= self.capacity)
        self._attend.copy_(torch.where(done, lens, -1))
        self.seqlens.copy_(torch.where(done, lens, self.seqlens))
        if first is not None:
            self._kept.copy_(torch.where(done, first, self._kept))
        return self.info

    def attend(self, layer, q, k, v, cu_seqlens_q, max_seqlen_q, sinks, rope_theta=None, rotary_dim=None,
               out_dtype=torch.bfloat16, softmax_scale=None, v_scale=1.0, out=None, lse=None):
        """One layer's attention of the tokens that ``extend`` made room for: q and k are
        rotated (rope_theta None: they already are), k and v written, and q attends over
        the cache.  Rows are packed by cu_seqlens_q.  Returns (out [Nt,Hq,128], lse [Hq,Nt]):
        the tensors given, or new ones.  Rows of skipped sequences, and of none, are left
        as they were: in new tensors they hold no particular values, so a step that goes on
        past a failed ``extend`` brings tensors of its own."""
        kp, vp = self.k_pages[layer], self.v_pages[layer]
        q = mimo.mimo_attn_paged_append(q, k, v, kp, vp, self.block_table, cu_seqlens_q, self._attend,
                                        1.0 if rope_theta is None else rope_theta,
                                        0 if rope_theta is None else rotary_dim,
                                        q_out=q if rope_theta is None else None)
        return mimo.mimo_attn_paged_attention(q, kp, vp, self.block_table, cu_seqlens_q, self._attend,
                                              max_seqlen_q, self.window, sinks, out=out, lse=lse,
                                              out_dtype=out_dtype, softmax_scale=softmax_scale, v_scale=v_scale)

    def truncate(self, lens):
        """Take the sequences back to lens [num_seqs] int32 (at most their present length):
        pages behind that are released.  With a window: not below the greatest length
        that the sequence had before an ``extend`` (since it was empty) less ``rollback``,
        or to 0."""
        lens = torch.minimum(lens, self.seqlens)
        # what extend kept stays, so that a later call may go back further
        self._hold(lens, self._kept if self.window else None, None)
        self.seqlens.copy_(torch.where(lens >= 0, lens, self.seqlens))  # a negative one was recorded
        self._attend.copy_(torch.where(self._attend < 0, self._attend, self.seqlens))
        self._kept.mul_(lens != 0)
        return self.info

    def fork(self, parent):
        """Slot i goes on as slot parent[i] [num_seqs] int32 was, sharing its pages; a
        negative parent leaves the slot empty (so does one that is no slot, and is
        recorded as an invalid argument in the device status)."""
        mimo.mimo_attn_page_fork(self.page_refs, self.block_table, parent, refs_out=self.page_refs,
                                 table_out=self._spare_table)
        self.block_table.copy_(self._spare_table)
        slots = self.seqlens.numel()
        source, real = parent.clamp(0, slots - 1).long(), (parent >= 0) & (parent < slots)
        for t in (self.seqlens, self._kept, self._attend):
            t.copy_(t[source] * real)

    def compact(self, max_moves):
        """Move used pages from the end of the pools to free places at their front, at most
        max_moves of them.  Returns ``info`` (moves made, pages in use)."""
        _, _, moves, _ = mimo.mimo_attn_page_compact(
            self.page_refs, self.block_table, max_moves, refs_out=self.page_refs, table_out=self.block_table,
            info=self.info)
        mimo.mimo_attn_page_copy(self.k_pages, self.v_pages, moves)
        return self.info
