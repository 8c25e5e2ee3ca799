// What the paged-cache kernels share: the description of a call's sequences
// and pages, and the checks that keep a bad table or length inside the
// caller's buffers.
//
// A paged cache holds key/value rows in pages of page_size token slots:
// k_pages [num_pages, page_size, Hkv, 192], v_pages [num_pages, page_size,
// Hkv, 128].  block_table [num_seqs, max_pages] names the page of each run of
// page_size positions of a sequence; a negative entry is "no page".  A call
// brings n_b = cu_q[b+1] - cu_q[b] new tokens of sequence b, packed, which sit
// at positions L_b - n_b .. L_b - 1 (L_b = seqlens[b], the new tokens included).
#pragma once

#include "common.cuh"

namespace mimo {

struct PagedBatch {
  const int32_t* table;    // [num_seqs, max_pages]
  const int32_t* cu_q;     // [num_seqs + 1]
  const int32_t* seqlens;  // [num_seqs]
  int num_seqs, total_q;
  int max_q;               // >= every n_b
  int num_pages, page_size, max_pages;
};

// One sequence of a call: its first packed row, new tokens and length.
struct PagedSeq {
  int b0, n, len;
  bool ok;  // false: an argument of this sequence is out of range, nothing of it is read or written
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& p, int b) {
  PagedSeq s;
  s.b0 = p.cu_q[b];
  s.n = p.cu_q[b + 1] - s.b0;
  s.len = p.seqlens[b];
  s.ok = seq_in_bounds(s.b0, s.n, p.max_q, p.total_q) && s.n <= s.len &&
         s.len <= (long long)p.max_pages * p.page_size;
  return s;
}

// wait_bounded for a whole warp, polled by its first lane alone: each lane's poll
// is a shared-memory operation of its own, and 32 of them from a warp with
// nothing else to do take bandwidth from the operands of the tensor cores.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_bounded(bar, parity, abort);
  return __shfl_sync(0xffffffffu, ok, 0);
}

// wait_bounded for a whole warp, polled by every lane, with one answer for all of
// them.  Lanes leave the poll one by one, and where time runs out some may have seen
// the phase and others not; what follows such a wait is done by the whole warp at
// once (TMEM accesses, ldmatrix, votes), and needs every lane there.  (A long chunk
// takes 0.4 % more with the vote, and nothing shows elsewhere; polled by one lane and
// passed on, a step under a short window takes 93 us for 83.)
__device__ __forceinline__ bool wait_lanes(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort));
}

// The sequence of packed row t, found by the whole warp: how many sequences
// end at or before t (32 of cu_q at a time, 32 runs of it first); -1 for a row
// that none owns.  For a sound cu_q that is the sequence with cu_q[b] <= t <
// cu_q[b+1]; for any other the caller's range check decides.
__device__ __forceinline__ int paged_seq_of_row(const PagedBatch& p, int t) {
  const int lane = threadIdx.x & 31;
  int b = 0, step = p.num_seqs;
  while (step > 32) {  // sequences [b, b + step) are left
    const int run = (step + 31) / 32;
    const int at = b + min(step, (lane + 1) * run);
    const int full = __popc(__ballot_sync(0xffffffffu, p.cu_q[at] <= t));
    const int skip = min(step, full * run);
    b += skip;
    step = min(step - skip, run);
  }
  const bool before = lane < step && p.cu_q[b + lane + 1] <= t;
  b += __popc(__ballot_sync(0xffffffffu, before));
  return (b < p.num_seqs && p.cu_q[b] <= t) ? b : -1;
}

// The page that holds positions [j * page_size, (j + 1) * page_size) of
// sequence b; -1 (recorded as MIMO_ERR_INVALID_ARG) where the table names none.
__device__ __forceinline__ int paged_page(const PagedBatch& p, int b, int j) {
  const int e = p.table[(size_t)b * p.max_pages + j];
  if (e >= 0 && e < p.num_pages) return e;
  record_status(1 /* MIMO_ERR_INVALID_ARG */);
  return -1;
}

}  // namespace mimo
