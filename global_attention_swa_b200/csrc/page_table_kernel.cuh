// Page bookkeeping of the paged cache, on the device: which pages each
// sequence holds, forks that share pages, and compaction.
//
// State: page_refs[P], how many table entries name each page (0 = free), and
// block_table[B][M].  Free pages are always handed out lowest index first, to
// the entries that need one in table order, so results do not depend on
// timing: the only atomics are integer adds, whose order does not matter.
//
// Each kernel is one thread-block cluster: what it needs across CTAs is a few
// counts, exchanged through distributed shared memory at a hardware cluster
// barrier (no flags in memory, no waiting loops).  Every warp owns one run of
// consecutive elements and ranks its flagged ones by ballot, so a pass is one
// read of the array.
#pragma once

#include "paged_common.cuh"

#undef MIMO_FILE_ID
#define MIMO_FILE_ID 13  // site numbers of the checked build

namespace mimo {

constexpr int kPtThreads = 1024;
constexpr int kPtWarps = kPtThreads / 32;
constexpr int kPtMaxCtas = 16;      // a cluster of 16 is past the portable size: opted into at the first launch
constexpr int kPtForkRows = 2048;   // table rows of one histogram round

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Cluster-wide barrier; global and shared writes before it are visible to the
// whole cluster after it.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The word at this CTA's shared address `addr`, in the CTA of the given rank.
__device__ __forceinline__ int ld_cluster(const int* addr, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(addr)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

struct PtShared {
  int warp_count[2][kPtWarps];
  int cta_count[2];
};

// From two counts per warp (the same in all its lanes): the sum over all warps
// before this one in the cluster, and over all of them.  Ends in a state where
// the shared arrays may be used again only after another cluster barrier.
struct PtOffsets {
  int before[2], total[2];
};
__device__ __forceinline__ PtOffsets pt_offsets(PtShared& sh, int c0, int c1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    sh.warp_count[0][warp] = c0;
    sh.warp_count[1][warp] = c1;
  }
  __syncthreads();
  PtOffsets r;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int v = sh.warp_count[k][lane];
    r.before[k] = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
    const int sum = __reduce_add_sync(0xffffffffu, v);
    if (threadIdx.x == 0) sh.cta_count[k] = sum;
  }
  cluster_sync_all();
  const uint32_t me = cluster_rank();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int v = lane < (int)gridDim.x ? ld_cluster(&sh.cta_count[k], lane) : 0;
    r.before[k] += __reduce_add_sync(0xffffffffu, lane < (int)me ? v : 0);
    r.total[k] = __reduce_add_sync(0xffffffffu, v);
  }
  return r;
}

// The run of consecutive elements that this warp owns of n.
struct PtRun {
  int begin, end;
};
__device__ __forceinline__ PtRun pt_run(int n) {
  const long long warps = (long long)gridDim.x * kPtWarps;
  const long long each = ((n + warps - 1) / warps + 31) / 32 * 32;
  const long long w = (long long)blockIdx.x * kPtWarps + (threadIdx.x >> 5);
  PtRun r;
  r.begin = (int)min((long long)n, w * each);
  r.end = (int)min((long long)n, (w + 1) * each);
  return r;
}

// ------------------------------------------------------------------ hold

struct PageHoldParams {
  const int32_t* refs;        // [P]
  const int32_t* table;       // [B, M]
  const int32_t* seqlens;     // [B]
  const int32_t* first;       // [B] or null (0)
  const int32_t* write_from;  // [B] or null (nothing will be written)
  int32_t* refs_out;          // [P]; may be refs
  int32_t* table_out;         // [B, M]; may be table
  int32_t* moves;             // [B, 2]
  int32_t* info;              // [2]: pages missing, pages free afterwards
  int32_t* ws;                // [P + 1]: a counter, then the free pages to hand out
  int P, B, M, page_size;
};

// What the call wants of the entries of one row.
struct HoldRow {
  int lo, hi;      // entries [lo, hi) are wanted
  int own;         // wanted entries from here on will be written
  int write_from;
  bool ok;
};
__device__ __forceinline__ HoldRow hold_row(const PageHoldParams& p, int b) {
  HoldRow r = {};
  if (b >= p.B) return r;
  const int len = p.seqlens[b];
  const int first = p.first ? p.first[b] : 0;
  r.write_from = p.write_from ? p.write_from[b] : len;
  r.ok = len >= 0 && first >= 0 && r.write_from >= 0 && len <= (long long)p.M * p.page_size;
  r.lo = first / p.page_size;
  r.hi = (int)(((long long)len + p.page_size - 1) / p.page_size);
  r.own = p.write_from ? r.write_from / p.page_size : r.hi;
  return r;
}

// A lane's way through a run, 32 entries at a time: the entry's row and place,
// and the row's wants, worked out again only where the row changes.
struct HoldCursor {
  int b, j;
  HoldRow row;
  __device__ __forceinline__ HoldCursor(const PageHoldParams& p, int i) {
    b = i / p.M;
    j = i - b * p.M;
    row = hold_row(p, b);
  }
  __device__ __forceinline__ void step(const PageHoldParams& p) {
    j += 32;
    if (j >= p.M) {
      do {
        j -= p.M;
        ++b;
      } while (j >= p.M);
      row = hold_row(p, b);
    }
  }
  __device__ __forceinline__ bool wanted() const { return row.ok && j >= row.lo && j < row.hi; }
  __device__ __forceinline__ bool written() const { return wanted() && j >= row.own; }
};

constexpr int kPtBatch = 4;  // loads in flight per lane (2 and 8: 16.0 and 16.1 us for 15.4, page_hold)

// Passes, each ended by a cluster barrier: copy the counts; take the dropped
// entries off them; count the free pages and the entries in need (fresh ones,
// and written ones whose page others hold too); list the free pages; hand them
// out.  Nothing of a caller's state has changed but the counts of dropped
// pages when it is known whether the pages suffice, and those are put back if
// they do not.  A written entry that is to be replaced is marked -2 - page in
// table_out between the passes, since the counts that decided it then move.
//
// Bound by latency: five barriers and the passes between them, each a load or two
// deep.  64 rows of 1024 entries and 40000 pages take 15.4 us on 16 CTAs (17.6 on
// 8, 26.3 on 4); their 0.8 MB would take 0.13 us.
__global__ void __launch_bounds__(kPtThreads, 1) page_hold_kernel(const PageHoldParams p) {
  __shared__ PtShared sh;
  const int lane = threadIdx.x & 31;
  const int tid = blockIdx.x * kPtThreads + threadIdx.x, threads = gridDim.x * kPtThreads;
  const PtRun pages = pt_run(p.P), entries = pt_run(p.B * p.M);

  if (p.refs_out != p.refs)
    for (int i = tid; i < p.P; i += threads) p.refs_out[i] = p.refs[i];
  for (long long i = tid; i < 2LL * p.B; i += threads) p.moves[i] = -1;
  if (tid == 0) p.ws[0] = 0;
  cluster_sync_all();

  // entries that change at all in this warp's run: most warps have none
  int need = 0;
  bool touched = false;
  if (entries.begin < entries.end) {
    HoldCursor c(p, entries.begin + lane);
    for (int i0 = entries.begin; i0 < entries.end; i0 += 32 * kPtBatch) {
      int pg[kPtBatch];
#pragma unroll
      for (int u = 0; u < kPtBatch; ++u) {
        const int i = i0 + 32 * u + lane;
        pg[u] = i < entries.end ? p.table[i] : -1;
      }
#pragma unroll
      for (int u = 0; u < kPtBatch; ++u) {
        const int i = i0 + 32 * u + lane;
        bool fresh = false;
        if (i < entries.end) {
          const bool has = pg[u] >= 0 && pg[u] < p.P, wanted = c.wanted();
          if ((c.j == 0 && !c.row.ok) || pg[u] >= p.P) record_status(1 /* MIMO_ERR_INVALID_ARG */);
          fresh = wanted && !has;
          const bool drop = c.row.ok && !wanted && has;
          if (drop && atomicSub(&p.refs_out[pg[u]], 1) <= 0)
            record_status(1 /* MIMO_ERR_INVALID_ARG: a held page whose count says free */);
          const int v = (has || !c.row.ok) ? pg[u] : -1;
          if (p.table_out != p.table || v != pg[u]) p.table_out[i] = v;
          touched |= fresh || drop;
        }
        need += __popc(__ballot_sync(0xffffffffu, fresh));
        if (i0 + 32 * u + 32 < entries.end) c.step(p);
      }
    }
  }
  cluster_sync_all();

  if (p.write_from && entries.begin < entries.end) {
    need = 0;
    HoldCursor c(p, entries.begin + lane);
    for (int i0 = entries.begin; i0 < entries.end; i0 += 32) {
      const int i = i0 + lane;
      bool take = false;
      if (i < entries.end && c.wanted()) {
        const int v = p.table_out[i];
        const bool split = c.written() && v >= 0 && __ldcg(&p.refs_out[v]) > 1;
        take = split || v < 0;
        if (split) p.table_out[i] = -2 - v;
      }
      touched |= take;
      need += __popc(__ballot_sync(0xffffffffu, take));
      if (i0 + 32 < entries.end) c.step(p);
    }
  }
  touched = __any_sync(0xffffffffu, touched);
  int free_pages = 0;
  for (int i0 = pages.begin; i0 < pages.end; i0 += 32 * kPtBatch) {
    int v[kPtBatch];
#pragma unroll
    for (int u = 0; u < kPtBatch; ++u) {
      const int i = i0 + 32 * u + lane;
      v[u] = i < pages.end ? __ldcg(&p.refs_out[i]) : 1;
    }
#pragma unroll
    for (int u = 0; u < kPtBatch; ++u) free_pages += __popc(__ballot_sync(0xffffffffu, v[u] == 0));
  }
  const PtOffsets off = pt_offsets(sh, need, free_pages);
  const int missing = max(0, off.total[0] - off.total[1]);

  if (missing > 0) {  // the same decision in every thread of the cluster
    if (touched) {
      HoldCursor c(p, entries.begin + lane);
      for (int i = entries.begin + lane; i < entries.end; i += 32, c.step(p)) {
        const int v = p.table_out[i];
        if (c.row.ok && v <= -2) p.table_out[i] = -2 - v;
        if (c.row.ok && !c.wanted() && v >= 0 && atomicAdd(&p.refs_out[v], 1) == 0) atomicAdd(&p.ws[0], 1);
      }
    }
    cluster_sync_all();
    if (tid == 0) {
      p.info[0] = missing;
      p.info[1] = off.total[1] - __ldcg(&p.ws[0]);
    }
    return;
  }

  int rank = off.before[1];
  for (int i0 = pages.begin; i0 < pages.end && rank < off.total[0]; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t f = __ballot_sync(0xffffffffu, i < pages.end && __ldcg(&p.refs_out[i]) == 0);
    const int k = rank + __popc(f & ((1u << lane) - 1));
    if ((f >> lane & 1) && k < off.total[0]) p.ws[1 + k] = i;
    rank += __popc(f);
  }
  cluster_sync_all();

  if (touched) {
    rank = off.before[0];
    HoldCursor c(p, entries.begin + lane);
    for (int i0 = entries.begin; i0 < entries.end; i0 += 32 * kPtBatch) {
      int w[kPtBatch];
#pragma unroll
      for (int u = 0; u < kPtBatch; ++u) {
        const int i = i0 + 32 * u + lane;
        w[u] = i < entries.end ? p.table_out[i] : 0;
      }
#pragma unroll
      for (int u = 0; u < kPtBatch; ++u) {
        const int i = i0 + 32 * u + lane, v = w[u];
        const bool in = i < entries.end && c.row.ok;
        const bool take = in && (v <= -2 || (v == -1 && c.wanted()));
        const uint32_t f = __ballot_sync(0xffffffffu, take);
        if (take) {
          const int pg = __ldcg(&p.ws[1 + rank + __popc(f & ((1u << lane) - 1))]);
          p.table_out[i] = pg;
          p.refs_out[pg] = 1;
          if (v <= -2) {
            if (atomicSub(&p.refs_out[-2 - v], 1) == 1) atomicAdd(&p.ws[0], 1);
            if ((long long)c.j * p.page_size < c.row.write_from) {  // at most one page of a sequence
              p.moves[2LL * c.b] = -2 - v;
              p.moves[2LL * c.b + 1] = pg;
            }
          }
        } else if (in && v >= 0 && !c.wanted()) {
          p.table_out[i] = -1;
        }
        rank += __popc(f);
        if (i0 + 32 * u + 32 < entries.end) c.step(p);
      }
    }
  }
  cluster_sync_all();
  if (tid == 0) {
    p.info[0] = 0;
    p.info[1] = off.total[1] - off.total[0] + __ldcg(&p.ws[0]);
  }
}

// ------------------------------------------------------------------ fork

struct PageForkParams {
  const int32_t* refs;    // [P]
  const int32_t* table;   // [B, M]
  const int32_t* parent;  // [B_out]
  int32_t* refs_out;      // [P]; may be refs
  int32_t* table_out;     // [B_out, M]; not table
  int P, B, B_out, M;
};

// Row i of the new table is row parent[i] of the old one.  A row with c
// children changes the count of each of its pages by c - 1: rows that go on
// unforked touch no count at all.  Bound by latency, as page_hold; 32 beams of 6
// layers forked in 4.6 us, their last pages taken apart in 11.2 (page_hold) and
// copied in 6.6, 55 MB that need 8.4 where they are not in L2: 22.4 us in all.
__global__ void __launch_bounds__(kPtThreads, 1) page_fork_kernel(const PageForkParams p) {
  __shared__ int children[kPtForkRows];
  const int tid = blockIdx.x * kPtThreads + threadIdx.x, threads = gridDim.x * kPtThreads;
  if (p.refs_out != p.refs) {
    for (int i = tid; i < p.P; i += threads) p.refs_out[i] = p.refs[i];
    cluster_sync_all();  // the kernel argument decides: the whole cluster takes this branch
  }
  const int each = (p.B + gridDim.x - 1) / gridDim.x;
  const int r_end = min(p.B, (int)(blockIdx.x + 1) * each);
  for (int r0 = blockIdx.x * each; r0 < r_end; r0 += kPtForkRows) {
    const int rows = min(kPtForkRows, r_end - r0);
    for (int i = threadIdx.x; i < rows; i += kPtThreads) children[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.B_out; i += kPtThreads) {
      const int r = p.parent[i];
      if (r >= r0 && r < r0 + rows) atomicAdd(&children[r - r0], 1);
    }
    __syncthreads();
    const int step_b = kPtThreads / max(1, p.M), step_j = kPtThreads - step_b * p.M;
    int b = p.M > 0 ? threadIdx.x / p.M : rows, j = threadIdx.x - b * p.M;
    for (; b < rows; b += step_b, j += step_j) {
      if (j >= p.M) {  // step_j < M: once at most
        j -= p.M;
        if (++b >= rows) break;
      }
      const int d = children[b] - 1;
      const int pg = p.table[(long long)(r0 + b) * p.M + j];
      if (pg >= p.P) record_status(1 /* MIMO_ERR_INVALID_ARG */);
      if (d != 0 && pg >= 0 && pg < p.P && atomicAdd(&p.refs_out[pg], d) <= 0)
        record_status(1 /* MIMO_ERR_INVALID_ARG: a held page whose count says free */);
    }
    __syncthreads();
  }
  const int step_b = threads / max(1, p.M), step_j = threads - step_b * p.M;
  int b = p.M > 0 ? tid / p.M : p.B_out, j = tid - b * p.M;
  for (; b < p.B_out; b += step_b, j += step_j) {
    if (j >= p.M) {
      j -= p.M;
      if (++b >= p.B_out) break;
    }
    const int r = p.parent[b];
    if (r >= p.B && j == 0) record_status(1 /* MIMO_ERR_INVALID_ARG */);
    p.table_out[(long long)b * p.M + j] = (r >= 0 && r < p.B) ? p.table[(long long)r * p.M + j] : -1;
  }
}

// ------------------------------------------------------------------ compact

struct PageCompactParams {
  const int32_t* refs;   // [P]
  const int32_t* table;  // [B, M]
  int32_t* refs_out;     // [P]; may be refs
  int32_t* table_out;    // [B, M]; may be table
  int32_t* moves;        // [max_moves, 2]
  int32_t* info;         // [2]: moves made, pages in use
  int32_t* ws;           // [P]: rank of a page that may move, -1 otherwise
  int P, B, M, max_moves;
};

// With u pages in use, the k-th used page at or above u goes to the k-th free
// page below u, for the first max_moves of them.  Three passes over the counts and
// one over the table, bound by latency: 5.3 us for 256 pages (7.5 with
// the copy of the 24 that move), 7.2 for 4096 and a table of 48 rows.
__global__ void __launch_bounds__(kPtThreads, 1) page_compact_kernel(const PageCompactParams p) {
  __shared__ PtShared sh[2];
  const int lane = threadIdx.x & 31;
  const int tid = blockIdx.x * kPtThreads + threadIdx.x, threads = gridDim.x * kPtThreads;
  const PtRun pages = pt_run(p.P);
  int used = 0;
  for (int i0 = pages.begin; i0 < pages.end; i0 += 32) {
    const int i = i0 + lane;
    used += __popc(__ballot_sync(0xffffffffu, i < pages.end && p.refs[i] > 0));
  }
  const int u = pt_offsets(sh[0], used, 0).total[0];

  int nsrc = 0, ndst = 0;
  for (int i0 = pages.begin; i0 < pages.end; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < pages.end, use = in && p.refs[i] > 0;
    nsrc += __popc(__ballot_sync(0xffffffffu, use && i >= u));
    ndst += __popc(__ballot_sync(0xffffffffu, in && !use && i < u));
  }
  const PtOffsets off = pt_offsets(sh[1], nsrc, ndst);
  const int count = min(p.max_moves, off.total[0]);

  int ks = off.before[0], kd = off.before[1];
  for (int i0 = pages.begin; i0 < pages.end; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < pages.end;
    const int c = in ? p.refs[i] : 0;
    const uint32_t s = __ballot_sync(0xffffffffu, c > 0 && i >= u);
    const uint32_t d = __ballot_sync(0xffffffffu, in && c <= 0 && i < u);
    const uint32_t before = (1u << lane) - 1;
    const int rs = ks + __popc(s & before), rd = kd + __popc(d & before);
    if (in) {
      const bool src = (s >> lane & 1) && rs < count;
      p.ws[i] = src ? rs : -1;
      if (src) p.moves[2 * rs] = i;
      if ((d >> lane & 1) && rd < count) p.moves[2 * rd + 1] = i;
      if (p.refs_out != p.refs) p.refs_out[i] = c;
    }
    ks += __popc(s);
    kd += __popc(d);
  }
  for (long long i = 2LL * count + tid; i < 2LL * p.max_moves; i += threads) p.moves[i] = -1;
  cluster_sync_all();

  for (int k = tid; k < count; k += threads) {
    const int src = __ldcg(&p.moves[2 * k]), dst = __ldcg(&p.moves[2 * k + 1]);
    p.refs_out[dst] = p.refs[src];  // one thread for both: refs_out may be refs
    p.refs_out[src] = 0;
  }
  for (int i = tid; i < p.B * p.M; i += threads) {
    const int pg = p.table[i];
    if (pg >= p.P) record_status(1 /* MIMO_ERR_INVALID_ARG */);
    const int r = pg >= 0 && pg < p.P ? __ldcg(&p.ws[pg]) : -1;
    p.table_out[i] = r >= 0 ? __ldcg(&p.moves[2 * r + 1]) : pg;
  }
  if (tid == 0) {
    p.info[0] = count;
    p.info[1] = u;
  }
}

}  // namespace mimo
