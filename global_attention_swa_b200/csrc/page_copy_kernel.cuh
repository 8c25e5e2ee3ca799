// Copies whole pages of a paged cache, in every layer: the moves that
// page_hold (a shared page that is about to be written) and page_compact ask
// for.  Moving bytes is all it does; a CTA takes one piece of one page of one
// layer, reads it in 16-byte vectors, several of them before the first store.
//
// Bound by memory bandwidth: 900 pages of 64 tokens in 6 layers, 1.77 GB read and
// written, in 278 us: 6.36 TB/s, 97 % of a plain copy's rate (286 us with the
// compaction that names them; with 2 and 8 vectors in flight per thread 285 and
// 282, and 8 is the slower for few pages: 24 of 16 tokens 8.2 against 8.0 us).
#pragma once

#include "paged_common.cuh"

#undef MIMO_FILE_ID
#define MIMO_FILE_ID 14  // site numbers of the checked build

namespace mimo {

constexpr int kPcThreads = 256;
constexpr int kPcVecs = 4;                                  // 16-byte vectors in flight per thread
constexpr int kPcPiece = kPcThreads * kPcVecs;              // vectors of a piece (16 KB)

struct PageCopyParams {
  uint4* k;              // [layers, P] pages of k_vecs vectors
  uint4* v;              // [layers, P] pages of v_vecs vectors
  const int32_t* moves;  // [n, 2]: source, destination
  int n, layers, P;
  int k_vecs, v_vecs;    // 16-byte vectors of a page
  int k_pieces, pieces;  // pieces of a page's keys, and of its keys and values
};

__global__ void __launch_bounds__(kPcThreads) page_copy_kernel(const PageCopyParams p) {
  const long long units = (long long)p.n * p.layers * p.pieces;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = (int)(u % p.pieces);
    const long long r = u / p.pieces;
    const int layer = (int)(r % p.layers), m = (int)(r / p.layers);
    const int src = p.moves[2LL * m], dst = p.moves[2LL * m + 1];
    if (src < 0 || dst < 0 || src >= p.P || dst >= p.P) {
      if ((src >= p.P || dst >= p.P || (src < 0) != (dst < 0)) && threadIdx.x == 0)
        record_status(1 /* MIMO_ERR_INVALID_ARG */);
      continue;
    }
    const bool key = piece < p.k_pieces;
    const int vecs = key ? p.k_vecs : p.v_vecs;
    uint4* base = key ? p.k : p.v;
    const uint4* from = base + ((long long)layer * p.P + src) * vecs;
    uint4* to = base + ((long long)layer * p.P + dst) * vecs;
    const int at = (key ? piece : piece - p.k_pieces) * kPcPiece + threadIdx.x;
    uint4 x[kPcVecs];
#pragma unroll
    for (int i = 0; i < kPcVecs; ++i)
      if (at + i * kPcThreads < vecs) x[i] = from[at + i * kPcThreads];
#pragma unroll
    for (int i = 0; i < kPcVecs; ++i)
      if (at + i * kPcThreads < vecs) to[at + i * kPcThreads] = x[i];
  }
}

}  // namespace mimo
