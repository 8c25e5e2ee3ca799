// Attention of a chunk of new tokens over a paged cache, on 5th-generation
// tensor cores (tcgen05).
//
// Row (token i of the chunk, query head h) at position p = L - n + i sees the
// keys j with 0 <= p - j and, in a window, p - j <= window - 1:
//   m = max(sigma_h, max_j S_j),  Z = exp(sigma_h - m) + sum_j exp(S_j - m),
//   out = v_scale * sum_j exp(S_j - m) v_j / Z,  lse = m + ln Z.
//
// A tile is the G query heads of one key/value head x TQ = 128 / G tokens: its
// 128 rows share every key and value they read.  An item is one key/value
// head x kTiles tiles of consecutive tokens of a sequence; its keys pass in
// tiles of 128 through shared memory, each feeding kTiles score products.
//
// Work is dealt out in keys, not in items.  All items laid end to end (by
// sequence, key/value head, token block) are cut into equal shares, one per
// CTA, wherever the cut falls; an item that a cut divides leaves its parts
// (unnormalised O, reference m, sums l) in the workspace, and
// paged_combine_kernel joins them.  Lengths are read on the device: every CTA
// finds its own share from them.  With short windows an item is a tile or two
// and only whole items are dealt out.
//
//   warp 8      loads Q and K (TMA), allocates TMEM
//   warp 9      issues the MMAs (one thread): S = Q K^T (SS), O += P V (TS, P from TMEM)
//   warp 10     loads V (TMA) and keeps values out of the sum that must not reach
//               it (pg_zero_unseen, pg_look)
//   warp 11     works out the items of this CTA's share, ahead of the others
//   warps 0-3   softmax and epilogue of tile 0 (one row per thread)
//   warps 4-7   softmax and epilogue of tile 1
//
// The page table is looked up by the loading warps, one lane per box of
// box_rows keys (a divisor of the page size): a key tile may span many pages
// or part of one.  An entry that names no page is loaded from past the end of
// the pool, which the TMA unit fills with zeros.
//
// Softmax as in prefill_kernel: base 2, against a reference m that moves only
// when a tile's sum would leave the safe range; P is rounded to bf16 for the
// P.V product (the tensor cores take 16-bit operands beside bf16 V) and the
// output is normalised by the sum of the rounded values; l, m and O are fp32.
//
// Bounds, measured on one B200 (64 query heads, 4 key/value heads):
//   one tile   the cache's bytes: 32 sequences of up to 16384 keys and 1 to 6 new
//              tokens, 697 MB in 133 us, 5.2 TB/s (80 % of a plain copy's rate).
//              CTAs of equal shares end between 109 and 127 us.
//   two tiles  the products and, beside them, the exponentials: 2048 tokens at
//              length 32768, 2.66 TFLOP in 2.28 to 2.33 ms, 1140 to 1170 TFLOP/s (70 %
//              of a large bf16 GEMM's burst rate; 2.5 ms, 75 % of its sustained rate,
//              where power holds the clocks down).  Tensor pipe 55 %, XU pipe 44 %
//              active: per pair of 128 x 128 score tiles the exponentials take
//              about as long as the products, and each softmax waits for its scores.
//              A second chain runs beside that: V has one stage, so the next tile's
//              values are asked for when both products of this one are done.
//   short      (a window past what paged_window_kernel takes) 5197 new tokens under a
//              window of 300: 186 us against 36 for the bytes.  Two of an item's three
//              tiles are looked over between V's load and its product (pg_look), with
//              one stage of V, and with one Q and one O an item's steps run mostly one
//              after the other.
#pragma once

#include "paged_common.cuh"

#undef MIMO_FILE_ID
#define MIMO_FILE_ID 11  // site numbers of the checked build

namespace mimo {

constexpr int kPgThreads = 384;
constexpr int kPgKeys = 128;                 // keys of a tile
constexpr int kPgQBytes = 128 * 192 * 2;     // 3 boxes of [128 rows][64 dims]
constexpr int kPgKBytes = kPgKeys * 192 * 2;
constexpr int kPgVBytes = kPgKeys * 128 * 2;
constexpr int kPgKStages = 2;

// Two tiles share a key tile: Q 2 x 48 KB, K 2 x 48 KB, V 32 KB.  One tile (a
// handful of new tokens: bound by the cache's bytes): V has two stages too.
// Each is the faster one on its side: 2048 new tokens 2.28 ms with two tiles,
// 2.43 with one; 1 to 6 new tokens 133 us with one, 171 with two.
template <int kTiles>
struct PgLayout {
  static constexpr int kVStages = kTiles == 1 ? 2 : 1;
  static constexpr int kOffK = kTiles * kPgQBytes;
  static constexpr int kOffV = kOffK + kPgKStages * kPgKBytes;
  static constexpr int kOffBar = kOffV + kVStages * kPgVBytes;
  static constexpr int kOffItems = kOffBar + 512;            // barriers and plan before it
  static constexpr int kSmemBytes = kOffItems + 512 + 1024;  // the queue of items; alignment slack
};

// Partial results in the workspace: one descriptor per CTA, then for each CTA
// two slots (0: the item its share begins inside of, 1: the item its share
// ends inside of) of kTiles * 128 rows.
struct PgDesc {
  int open0;    // slot 0 holds a part: 1, and 2 if the item ends there
  int open1;    // slot 1 holds the first part of an item
  int row0;     // slot 1's item: first packed row (token)
  int h0;       //   first query head
  int rows;     //   valid rows (tokens * G)
  int pad[3];
};

struct PagedAttnParams {
  PagedBatch pb;
  const __nv_bfloat16* q;  // [total_q, Hq, 192]
  const __nv_bfloat16* k;  // [num_pages, page_size, Hkv, 192]
  const __nv_bfloat16* v;  // [num_pages, page_size, Hkv, 128]
  const float* sinks;      // [Hq] or null
  void* out;               // [total_q, Hq, 128]
  float* lse;              // [Hq, total_q] or null
  PgDesc* ws_desc;         // [ctas]
  float4* ws_ml;           // [ctas, 2, kTiles * 128]: m, l, sum of the rounded P
  float* ws_o;             // [ctas, 2, kTiles * 128, 128]
  int Hq, Hkv, G;
  int TQ;                  // tokens of a tile: 128 / G
  int window;
  int box_rows;            // keys of one TMA box; divides page_size and 128
  int split;               // 1: cut items anywhere, 0: deal out whole items
  float scale_log2, v_scale;
  int out_f32;
  int out_v8;              // out is 32-byte aligned
};

// A place in the list of all items: an item, and a key tile of it.
struct PgPlace {
  int b, g, i, t;
};

// Cost of an item of a sequence, in keys: what it reads, and kPgItemCost for
// its queries, its latencies and its epilogue (a fit over the CTAs of a batch of
// drafts: 1.6 us a key tile, 4.7 an item).
// Block i reads the D (i + 1) keys of the chunk up to its own (D: tokens of a block)
// and those before the chunk, but no more of the keys before it than its window: the
// cost rises by D a block as long as the window reaches back to the sequence's first
// key, and is the same for all blocks from there on.  With whole items only, 1.
// (Those drafts take 133 us with a cost of three key tiles, 134 with two, 135 with
// four, 142 without.)
constexpr int kPgItemCost = 3 * kPgKeys;
// Quotient of non-negative values; nearly always both fit 32 bits, and a 64-bit
// division is a long chain of dependent instructions.
__device__ __forceinline__ long long pg_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}

struct PgCost {
  long long base;  // block 0
  int slope;       // each further one of the first `rising`
  int rising;
  int blocks;
  long long flat;  // each block from there on
  __device__ __forceinline__ long long upto(int i) const {  // blocks 0 .. i-1
    const int r = min(i, rising);
    return base * r + (long long)slope * ((long long)r * (r - 1) / 2) + flat * (i - r);
  }
  // the block that holds cost y of [0, upto(blocks))
  __device__ __forceinline__ int block_of(long long y) const {
    if (blocks <= 1) return 0;
    const long long rise = upto(rising);
    if (y >= rise) return min(blocks - 1, rising + (int)pg_div(y - rise, flat));
    // the root of upto(i) = y, near enough for the steps below to find it
    const float h = (float)base - 0.5f * slope, z = 2.f * (float)y;
    int i = (int)(z / (sqrtf(h * h + slope * z) + h));
    i = max(0, min(i, rising - 1));
    while (i > 0 && upto(i) > y) --i;
    while (i + 1 < rising && upto(i + 1) <= y) ++i;
    return i;
  }
};
template <int kTiles>
__device__ __forceinline__ PgCost pg_cost(const PagedAttnParams& p, const PagedSeq& s) {
  PgCost c;
  const int D = kTiles * p.TQ;
  c.blocks = s.ok ? (s.n + D - 1) / D : 0;
  c.slope = D;
  c.base = (long long)(s.len - s.n) + D + kPgItemCost;
  c.rising = c.blocks;
  c.flat = 1;
  if (!p.split) {
    c.rising = 0;
  } else if (p.window > 0) {  // block i begins at position first + D i
    const int first = s.len - s.n;
    c.rising = first >= p.window ? 0 : min(c.blocks, (p.window - first - 1) / D + 1);
    c.flat = (long long)p.window + D + kPgItemCost;
  }
  return c;
}

// One item as a role sees it: its keys and the tiles of them in this share.
struct PgItem {
  int b, g, i;      // sequence, key/value head, block
  int tok0;         // packed row of its first token
  int p0;           // that token's position
  int tokens;       // valid tokens, 1 .. kTiles * TQ
  int outer;        // of its boxes of 16 keys, some reach past the sequence's end or before its chunk's first key
  int lo, hi;       // keys that some row sees: [lo, hi]
  int early;        // of those, [lo, early) and (p0, hi] are hidden from some rows
  int start;        // first key of tile 0: lo rounded down to a box
  int n_kt;         // key tiles
  int t0, t1;       // the tiles of this share
  int turn;         // the order of their passage: from t0 + turn on, then from t0
  int n_last;       // keys that the products take of the last tile, a multiple of 16
  int e0, e1;       // tiles below e0 and from e1 on hold values that some row must not meet
  __device__ __forceinline__ int count() const { return t1 - t0; }
  __device__ __forceinline__ int width(int t) const { return t == n_kt - 1 ? n_last : kPgKeys; }
  __device__ __forceinline__ bool edge(int t) const { return t < e0 || t >= e1; }
  // The tile that passes j-th.
  __device__ __forceinline__ int tile(int j) const {
    const int t = t0 + turn + j;
    return t < t1 ? t : t - (t1 - t0);
  }
};

// Walks the items of a share.
template <int kTiles>
struct PgWalk {
  PgPlace at, end;
  PagedSeq s;
  int blocks;
  bool first;
  int passed;  // tiles of this share in the items before
  __device__ __forceinline__ void seq(const PagedAttnParams& p) {
    const int D = kTiles * p.TQ;
    blocks = 0;
    while (at.b < p.pb.num_seqs) {
      s = paged_seq(p.pb, at.b);
      blocks = s.ok ? (s.n + D - 1) / D : 0;
      if (blocks > 0) break;
      ++at.b;
    }
  }
  __device__ __forceinline__ PgWalk(const PagedAttnParams& p, const PgPlace* plan) : at(plan[0]), end(plan[1]), first(true), passed(0) {
    seq(p);
  }
  // The next item with work in this share; false at its end.
  __device__ __forceinline__ bool next(const PagedAttnParams& p, PgItem& it) {
    while (true) {
      if (!first) {  // past the item of the last call
        if (at.b == end.b && at.g == end.g && at.i == end.i) return false;
        at.t = 0;
        if (++at.i >= blocks) {
          at.i = 0;
          if (++at.g >= p.Hkv) {
            at.g = 0;
            ++at.b;
            seq(p);
          }
        }
      }
      first = false;
      const bool last = at.b == end.b && at.g == end.g && at.i == end.i;
      if (at.b >= p.pb.num_seqs || (last && end.t == 0)) return false;
      const int D = kTiles * p.TQ;
      it.b = at.b;
      it.g = at.g;
      it.i = at.i;
      it.tok0 = s.b0 + at.i * D;
      it.p0 = s.len - s.n + at.i * D;
      it.tokens = min(D, s.n - at.i * D);
      it.hi = it.p0 + it.tokens - 1;
      it.lo = p.window > 0 ? max(0, it.p0 - p.window + 1) : 0;
      it.early = p.window > 0 ? max(it.lo, it.hi - p.window + 1) : it.lo;
      it.start = it.lo / p.box_rows * p.box_rows;
      it.outer = it.start < max(0, s.len - s.n - p.window + 1) || it.start + ((it.hi - it.start + 16) & ~15) > s.len;
      it.n_kt = (it.hi - it.start) / kPgKeys + 1;
      const int left = it.hi + 1 - (it.start + (it.n_kt - 1) * kPgKeys);
      it.n_last = min(kPgKeys, (left + 15) & ~15);
      it.e0 = (max(it.early, it.lo) - it.start + kPgKeys - 1) / kPgKeys;
      it.e1 = it.hi > it.p0 ? (it.p0 + 1 - it.start) / kPgKeys : left < it.n_last ? it.n_kt - 1 : it.n_kt;
      it.t0 = at.t;
      it.t1 = last ? min(end.t, it.n_kt) : it.n_kt;
      if (it.t0 < it.t1) {
        // All CTAs pass about as many tiles in a time, so the count so far is a
        // clock they share: each begins an item at the tile the clock is at.  Those
        // that work on blocks of one sequence then read the same keys at the same
        // time, from L2, wherever their shares began.
        const int at_clock = passed % it.n_kt;
        it.turn = at_clock > it.t0 && at_clock < it.t1 ? at_clock - it.t0 : 0;
        passed += it.t1 - it.t0;
        return true;
      }
    }
  }
};

// A key tile of an item: its first key, how many the products take (a multiple
// of 16), and rows of it: [0, zlo) and [zhi, n) are seen by nothing, [lo, lo_end)
// and [hi, hi_end) by some rows only.
struct PgTile {
  int k0, n, zlo, zhi, lo, lo_end, hi, hi_end;
};
__device__ __forceinline__ PgTile pg_keys(const PgItem& it, int k0, int most) {
  PgTile r;
  r.k0 = k0;
  const int left = it.hi + 1 - k0;
  r.n = min(most, (left + 15) & ~15);
  r.zlo = max(0, it.lo - k0);
  r.zhi = min(r.n, left);
  r.lo = r.zlo;
  r.lo_end = min(r.zhi, it.early - k0);
  r.hi = max(0, it.p0 + 1 - k0);
  r.hi_end = r.zhi;
  return r;
}
__device__ __forceinline__ PgTile pg_tile(const PgItem& it, int t) { return pg_keys(it, it.start + t * kPgKeys, kPgKeys); }

// 0 * v is NaN where v is not finite, so a value row must not enter the product
// of rows that do not see its key.  Rows that nothing sees are zeroed in shared
// memory.  Rows that some rows of the item see are looked over, and where one
// holds a value that is not finite it is zeroed too, and the epilogue adds it to
// the rows that see it (pg_add_hidden).  All by one warp; vb: shared address of
// [rows][64 columns] boxes `box` bytes apart.  At most a tile or two of an item
// have such rows; looking costs 0.7 % of a long chunk (2.295 against 2.277 ms).
__device__ __forceinline__ bool bf16x2_not_finite(uint32_t u) {
  return (u & 0x7F80u) == 0x7F80u || (u & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ bool not_finite(const uint4& u) {
  return bf16x2_not_finite(u.x) || bf16x2_not_finite(u.y) || bf16x2_not_finite(u.z) || bf16x2_not_finite(u.w);
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr) : "memory");
  return u;
}
__device__ __forceinline__ void sts_zero(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}
// Shared address of vector w of a list of value rows, 16 vectors a row (8 in each
// box): [0, na) of the list from row a on, the rest from row b on.
__device__ __forceinline__ uint32_t pg_vec(uint32_t vb, int box, int w, int a, int na, int b) {
  const int i = w >> 4;
  return vb + ((w >> 3) & 1) * box + (i < na ? a + i : b + i - na) * 128 + (w & 7) * 16;
}
// Zeroes the rows that nothing sees.
__device__ __forceinline__ void pg_zero_unseen(const PgTile& tl, uint32_t vb, int box) {
  for (int w = threadIdx.x & 31; w < (tl.zlo + tl.n - tl.zhi) * 16; w += 32)
    sts_zero(pg_vec(vb, box, w, 0, tl.zlo, tl.zhi));
}
// Whether the rows that only some rows of the item see hold a value that is not finite.
__device__ __forceinline__ bool pg_look(const PgTile& tl, uint32_t vb, int box) {
  const int lane = threadIdx.x & 31;
  const int na = max(0, tl.lo_end - tl.lo), rows = na + max(0, tl.hi_end - tl.hi);
  bool any = false;
#pragma unroll 1
  for (int w0 = 0; w0 < rows * 16; w0 += 256) {
    uint4 u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // past the end: the first vector again
      const int w = w0 + 32 * i + lane;
      u[i] = lds_v4(pg_vec(vb, box, w < rows * 16 ? w : 0, tl.lo, na, tl.hi));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= not_finite(u[i]);
  }
  return __any_sync(0xffffffffu, any);
}
// Zeroes those of them that do.
__device__ __forceinline__ void pg_take_out(const PgTile& tl, uint32_t vb, int box) {
  const int lane = threadIdx.x & 31;
  const int na = max(0, tl.lo_end - tl.lo), rows = na + max(0, tl.hi_end - tl.hi);
#pragma unroll 1
  for (int w0 = 0; w0 < rows * 16; w0 += 32) {  // two rows at a time
    const int w = w0 + lane;
    const uint32_t at = pg_vec(vb, box, w, tl.lo, na, tl.hi);
    const bool bad = w < rows * 16 && not_finite(lds_v4(at));
    if (__ballot_sync(0xffffffffu, bad) >> (lane & 16) & 0xFFFFu) sts_zero(at);
  }
}

// The items of a CTA's share, worked out by one thread and read by every role: a
// ring of kPgItems in shared memory.  (Walking the list in each role instead cost
// a copy of that code per role, more instructions than their cache holds beside
// the loops, and its latency in each.)
constexpr int kPgItems = 4;
struct PgQueue {
  PgItem it[kPgItems];
  int more[kPgItems];   // 0: past the last item
  int dirty[kPgItems];  // pg_look found something
};
template <int kTiles>
__device__ __forceinline__ void pg_schedule(const PagedAttnParams& p, const PgPlace* plan, PgQueue& q, uint64_t* full,
                                            uint64_t* empty, volatile int* abort) {
  PgWalk<kTiles> walk(p, plan);
  bool more = true;
  for (int n = 0; more; ++n) {
    const int s = n % kPgItems;
    if (n >= kPgItems && !wait_bounded(&empty[s], (n / kPgItems - 1) & 1, abort)) return;
    PgItem it;
    more = walk.next(p, it);
    q.it[s] = it;
    q.more[s] = more;
    q.dirty[s] = 0;
    mbar_arrive(&full[s]);
  }
}
// Item n is there to read; false past the last one, or after a timed-out wait.
// Each reader arrives once on empty[n % kPgItems] when it is done with it.  kWarp:
// the reader is a whole warp, not one thread.
template <bool kWarp>
__device__ __forceinline__ bool pg_item(const PgQueue& q, uint64_t* full, int n, volatile int* abort) {
  const int s = n % kPgItems;
  const uint32_t parity = (n / kPgItems) & 1;
  return (kWarp ? wait_lanes(&full[s], parity, abort) : wait_bounded(&full[s], parity, abort)) &&
         *const_cast<const volatile int*>(&q.more[s]);
}

// This CTA's share.  All threads call it; plan (shared) holds the first place
// and the one past the last afterwards.  Returns false where there is no share.
template <int kTiles, int kThreads = kPgThreads>
__device__ __forceinline__ bool pg_plan(const PagedAttnParams& p, PgPlace* plan, long long* warp_sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int each = (p.pb.num_seqs + kThreads - 1) / kThreads;
  const int b0 = threadIdx.x * each, b1 = min(p.pb.num_seqs, b0 + each);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const PagedSeq s = paged_seq(p.pb, b);
    if (!s.ok && blockIdx.x == 0) record_status(1 /* MIMO_ERR_INVALID_ARG */);
    const PgCost c = pg_cost<kTiles>(p, s);
    mine += c.upto(c.blocks) * p.Hkv;
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (threadIdx.x == 0) plan[0] = plan[1] = PgPlace{p.pb.num_seqs, 0, 0, 0};
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long x = warp_sum[w];
    if (w < warp) before += x;
    total += x;
  }
  before += incl - mine;
  // no share below a key tile: with at least two tiles to a share three chats of up
  // to 700 keys take 1.4 us more (of 15), with four 5.4
  const long long unit = p.split ? kPgKeys : 1;
  const long long shares = max(1LL, min((long long)gridDim.x, pg_div(total, unit)));
  const int c = blockIdx.x;
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const long long x = pg_div(total * min((long long)c + k, shares), shares);
    if (x < before || x >= before + mine) continue;
    long long y = x - before;
    for (int b = b0; b < b1; ++b) {
      const PgCost cost = pg_cost<kTiles>(p, paged_seq(p.pb, b));
      const long long group = cost.upto(cost.blocks), all = group * p.Hkv;
      if (y >= all) {
        y -= all;
        continue;
      }
      PgPlace pl;
      pl.b = b;
      pl.g = (int)pg_div(y, group);
      y -= pl.g * group;
      pl.i = cost.block_of(y);
      pl.t = p.split ? (int)(max(0LL, y - cost.upto(pl.i) - kPgItemCost) / kPgKeys) : 0;
      plan[k] = pl;
      break;
    }
  }
  __syncthreads();
  return c < shares && total > 0;
}

// The pool row (page * page_size + slot) at which box j of a tile begins; past
// the pool's end, where the loads read zeros, for an entry that names no page.
__device__ __forceinline__ int pg_box_row(const PagedAttnParams& p, const PgItem& it, const PgTile& tl, int j) {
  const int pos = tl.k0 + j * p.box_rows;
  const int page = pos / p.pb.page_size;
  int e = -1;
  if (MIMO_ROW_OK((long long)it.b * p.pb.max_pages + page, (long long)p.pb.num_seqs * p.pb.max_pages))
    e = paged_page(p.pb, it.b, page);
  return e < 0 ? p.pb.num_pages * p.pb.page_size : e * p.pb.page_size + (pos - page * p.pb.page_size);
}

// What was taken out of the product: adds P v to `kN` columns (from column c0 on)
// of the row (packed row tok, head h, position pos, reference m) for the keys in
// [k_begin, k_end) that it sees, some rows of its item do not, and whose values
// are not all finite.
template <int kN>
__device__ __noinline__ void pg_add_hidden(const PagedAttnParams& p, const PgItem& it, int k_begin, int k_end, int tok,
                                           int h, int pos, float m, int c0, float (&o)[kN]) {
  const int see = p.window > 0 ? max(0, pos - p.window + 1) : 0;
#pragma unroll 1
  for (int j = max(it.lo, k_begin); j < min(it.hi + 1, k_end); ++j) {
    if (j >= it.early && j <= it.p0) {  // every row sees these
      j = it.p0;
      continue;
    }
    if (j < see || j > pos) continue;
    const int e = p.pb.table[(size_t)it.b * p.pb.max_pages + j / p.pb.page_size];
    if (e < 0 || e >= p.pb.num_pages) continue;
    const size_t row = ((size_t)e * p.pb.page_size + j % p.pb.page_size) * p.Hkv + it.g;
    const uint4* v = reinterpret_cast<const uint4*>(p.v + row * 128);
    bool bad = false;
#pragma unroll 1
    for (int i = 0; i < 16 && !bad; ++i) bad = not_finite(v[i]);
    if (!bad) continue;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p.q + ((size_t)tok * p.Hq + h) * 192);
    const uint32_t* k = reinterpret_cast<const uint32_t*>(p.k + row * 192);
    float s = 0.f;
#pragma unroll 1
    for (int i = 0; i < 96; ++i) s += bf16_lo(q[i]) * bf16_lo(k[i]) + bf16_hi(q[i]) * bf16_hi(k[i]);
    const float pe = bf16_lo(pack_bf16(ex2(s * p.scale_log2 - m), 0.f));  // as the product would have it
#pragma unroll
    for (int i = 0; i < kN / 8; ++i) {
      const uint4 u = v[c0 / 8 + i];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        o[8 * i + 2 * x] += pe * bf16_lo(w[x]);
        o[8 * i + 2 * x + 1] += pe * bf16_hi(w[x]);
      }
    }
  }
}

template <int kTiles>
__global__ void __launch_bounds__(kPgThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttnParams p) {
  using Lay = PgLayout<kTiles>;
  constexpr int kVStages = Lay::kVStages;
  extern __shared__ __align__(1024) uint8_t pgsmem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pgsmem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kOffBar);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;    // [2]
  uint64_t* k_empty = bars + 4;   // [2]
  uint64_t* v_full = bars + 6;    // [kVStages]
  uint64_t* v_empty = bars + 8;   // [kVStages]
  uint64_t* v_ready = bars + 10;  // [kVStages] the unseen rows of an edge tile are zeroed
  uint64_t* s_full = bars + 12;   // [2] two tiles: of tile i; one: of key tile parity i
  uint64_t* p_full = bars + 14;   // [2]
  uint64_t* o_full = bars + 16;   // [2]
  uint64_t* o_empty = bars + 18;  // [2]
  uint64_t* mma_drain = bars + 20;  // teardown after a timed-out wait only
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 21);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 22);
  volatile int* never_flag = reinterpret_cast<volatile int*>(bars + 23);  // never raised
  int* armed = reinterpret_cast<int*>(bars + 24);  // [4]: phases armed on Q, K, V; the MMA thread had work
  PgPlace* plan = reinterpret_cast<PgPlace*>(bars + 26);          // [2]
  uint64_t* i_full = bars + 30;                                      // [kPgItems]
  uint64_t* i_empty = bars + 34;                                     // [kPgItems]
  long long* warp_sum = reinterpret_cast<long long*>(bars + 40);     // [12]
  static_assert(sizeof(PgQueue) <= 512, "the queue's place");
  PgQueue& queue = *reinterpret_cast<PgQueue*>(smem + Lay::kOffItems);
  constexpr int kReaders = 3 + 4 * kTiles;  // warps 8, 9, 10 and the softmax warps

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 8) {
    if (lane == 0) {
      mbar_init(q_full, 1);
      mbar_init(q_empty, 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&k_full[i], 1);
        mbar_init(&k_empty[i], 1);
        mbar_init(&v_full[i], 1);
        mbar_init(&v_empty[i], 1);
        mbar_init(&v_ready[i], 1);
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], 128);
        mbar_init(&o_full[i], 1);
        mbar_init(&o_empty[i], 128);
      }
      for (int i = 0; i < kPgItems; ++i) {
        mbar_init(&i_full[i], 1);
        mbar_init(&i_empty[i], kReaders);
      }
      mbar_init(mma_drain, 1);
      *never_flag = 0;
      armed[0] = armed[1] = armed[2] = armed[3] = 0;
      // sampled once, so every thread of the CTA sees the same decision
      *abort_flag = timed_out_before() ? 1 : 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const bool share = pg_plan<kTiles>(p, plan, warp_sum);  // has the barriers the set-up needs
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  // after a recorded timeout elsewhere, do no work (but still free TMEM)
  const bool work = share && !*abort_flag;
  if (threadIdx.x == 0 && p.split) p.ws_desc[blockIdx.x] = PgDesc{};
  // the combine kernel may be set up while this one runs; it waits for its end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp >= 8) {
    setmaxnreg_dec<104>();
  }
  if (warp == 8) {
    // ------------------------------------------------------------ Q and K
    if (work) {
      int n = 0, kt = 0;  // items and key tiles loaded
      bool ok = true;
      while (ok && pg_item<true>(queue, i_full, n, abort_flag)) {
        const PgItem it = queue.it[n % kPgItems];
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[n % kPgItems]);
        if (n > 0 && !(ok = wait_warp(q_empty, (n - 1) & 1, abort_flag))) break;
        const bool has1 = kTiles == 2 && it.tokens > p.TQ;
        if (lane == 0) {
          const int bytes = p.TQ * p.G * 384;
          mbar_arrive_expect_tx(q_full, has1 ? 2 * bytes : bytes);
#pragma unroll
          for (int c = 0; c < 3; ++c) tma_load_3d(smem + c * 16384, &tm_q, q_full, c * 64, it.g * p.G, it.tok0);
          if (has1) {
#pragma unroll
            for (int c = 0; c < 3; ++c)
              tma_load_3d(smem + kPgQBytes + c * 16384, &tm_q, q_full, c * 64, it.g * p.G, it.tok0 + p.TQ);
          }
        }
        ++n;
        for (int j = 0; j < it.count(); ++j, ++kt) {
          const PgTile tl = pg_tile(it, it.tile(j));
          const int boxes = (tl.n + p.box_rows - 1) / p.box_rows;
          const int row = lane < boxes ? pg_box_row(p, it, tl, lane) : 0;
          const int ks = kt & 1;
          if (kt >= 2 && !(ok = wait_warp(&k_empty[ks], ((kt >> 1) - 1) & 1, abort_flag))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&k_full[ks], boxes * p.box_rows * 384);
            armed[1] = kt + 1;
          }
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = smem + Lay::kOffK + ks * kPgKBytes + lane * p.box_rows * 128;
#pragma unroll
            for (int c = 0; c < 3; ++c) tma_load_3d(dst + c * 16384, &tm_k, &k_full[ks], c * 64, it.g, row);
          }
        }
      }
      if (lane == 0) armed[0] = n;  // every item counted had its Q armed
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ V
    if (work) {
      int kt = 0;
      bool ok = true;
      for (int n = 0; ok && pg_item<true>(queue, i_full, n, abort_flag); ++n) {
        const PgItem it = queue.it[n % kPgItems];
        for (int j = 0; j < it.count(); ++j, ++kt) {
          const PgTile tl = pg_tile(it, it.tile(j));
          const int boxes = (tl.n + p.box_rows - 1) / p.box_rows;
          const int row = lane < boxes ? pg_box_row(p, it, tl, lane) : 0;
          const int vs = kt % kVStages;
          if (kt >= kVStages && !(ok = wait_warp(&v_empty[vs], (kt / kVStages - 1) & 1, abort_flag))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&v_full[vs], boxes * p.box_rows * 256);
            armed[2] = kt + 1;
          }
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = smem + Lay::kOffV + vs * kPgVBytes + lane * p.box_rows * 128;
#pragma unroll
            for (int c = 0; c < 2; ++c) tma_load_3d(dst + c * 16384, &tm_v, &v_full[vs], c * 64, it.g, row);
          }
          if (it.edge(it.tile(j))) {
            if (!(ok = wait_warp(&v_full[vs], (kt / kVStages) & 1, abort_flag))) break;
            const uint32_t vb = sbase + Lay::kOffV + vs * kPgVBytes;
            pg_zero_unseen(tl, vb, 16384);
            if (pg_look(tl, vb, 16384)) {
              pg_take_out(tl, vb, 16384);
              if (lane == 0) queue.dirty[n % kPgItems] = 1;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_ready[vs]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[n % kPgItems]);
      }
    }
  } else if (warp == 11) {
    if (lane == 0 && work) pg_schedule<kTiles>(p, plan, queue, i_full, i_empty, abort_flag);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && work) {
      armed[3] = 1;
      const uint32_t tS0 = tbase + 0, tS1 = tbase + 128, tO0 = tbase + 256, tO1 = tbase + 384;
      constexpr uint32_t dhi = desc_hi_sw128(1024);
      const uint32_t dQ0 = desc_lo_sw128(sbase, 16);
      const uint32_t dQ1 = desc_lo_sw128(sbase + (kTiles - 1) * kPgQBytes, 16);
      const uint32_t dK0 = desc_lo_sw128(sbase + Lay::kOffK, 16);
      const uint32_t dV0 = desc_lo_sw128(sbase + Lay::kOffV, 16384);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128, false, true);
      // S = Q K^T over 192 dims = 12 MMAs of K=16 (3 swizzle boxes x 4 steps of 32 B), n keys wide
      auto issue_s = [&](uint32_t tS, uint32_t dQ, int stage, int n) {
        const uint32_t idesc = idesc_bf16_f32(128, 0, false, false) | (static_cast<uint32_t>(n >> 3) << 17);
        const uint32_t dK = dK0 + static_cast<uint32_t>(stage) * (kPgKBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 12; ++kk) {
          const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          umma_ss_lo(tS, dQ + off, dK + off, dhi, idesc, kk > 0 ? 1u : 0u);
        }
      };
      // O += P V over n keys (P: 8 TMEM columns for 16 keys; V: 16 rows = 2 KB)
      auto issue_pv = [&](uint32_t tO, uint32_t tP, int stage, int n, bool acc) {
        const uint32_t dV = dV0 + static_cast<uint32_t>(stage) * (kPgVBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (kk * 16 < n) umma_ts_lo(tO, tP + kk * 8, dV + ((kk * 2048) >> 4), dhi, idesc_o, (acc || kk > 0) ? 1u : 0u);
      };
      int n = 0, n1 = 0;   // items, those with a second tile
      int kt = 0;          // key tiles (all items): K and V phases
      int c0 = 0, c1 = 0;  // score tiles of tile 0 / 1: s_full, p_full phases (two tiles)
      bool ok = true;
      uint32_t edges = 0;  // parity of each stage's edge tiles: v_ready phases
      // (a stage's next tile is loaded after this one's P.V, so neither wait can fall behind)
      auto wait_v = [&](bool edge) {
        const int vs = kt % kVStages;
        if (!edge) return wait_bounded(&v_full[vs], (kt / kVStages) & 1, abort_flag);
        edges ^= 1u << vs;
        return wait_bounded(&v_ready[vs], ~(edges >> vs) & 1, abort_flag);
      };
      while (ok && pg_item<false>(queue, i_full, n, abort_flag)) {
        const PgItem it = queue.it[n % kPgItems];
        mbar_arrive(&i_empty[n % kPgItems]);
        const bool has1 = kTiles == 2 && it.tokens > p.TQ;
        if (!(ok = wait_bounded(q_full, n & 1, abort_flag))) break;
        if constexpr (kTiles == 1) {
          // scores run one key tile ahead of the softmax, in two TMEM buffers
          auto scores = [&](int j, int kn) {
            if (!wait_bounded(&k_full[kn & 1], (kn >> 1) & 1, abort_flag)) return false;
            tc_fence_after();
            issue_s((kn & 1) ? tS1 : tS0, dQ0, kn & 1, it.width(it.tile(j)));
            umma_commit(&s_full[kn & 1]);
            umma_commit(&k_empty[kn & 1]);
            if (j == it.count() - 1) umma_commit(q_empty);
            return true;
          };
          if (!(ok = scores(0, kt))) break;
          if (it.count() > 1 && !(ok = scores(1, kt + 1))) break;
          for (int j = 0; j < it.count(); ++j, ++kt) {
            const int t = it.tile(j), w = it.width(t);
            if (!(ok = wait_v(it.edge(t)))) break;
            if (!(ok = wait_bounded(&p_full[kt & 1], (kt >> 1) & 1, abort_flag))) break;
            if (j == 0 && n > 0 && !(ok = wait_bounded(&o_empty[0], (n - 1) & 1, abort_flag))) break;
            tc_fence_after();
            issue_pv(tO0, (kt & 1) ? tS1 : tS0, kt % kVStages, w, j > 0);
            umma_commit(&v_empty[kt % kVStages]);
            if (j == it.count() - 1) umma_commit(&o_full[0]);
            if (j + 2 < it.count() && !(ok = scores(j + 2, kt + 2))) break;
          }
        } else {
          if (!(ok = wait_bounded(&k_full[kt & 1], (kt >> 1) & 1, abort_flag))) break;
          tc_fence_after();
          {
            const int w = it.width(it.tile(0));
            issue_s(tS0, dQ0, kt & 1, w);
            umma_commit(&s_full[0]);
            if (has1) {
              issue_s(tS1, dQ1, kt & 1, w);
              umma_commit(&s_full[1]);
            }
            umma_commit(&k_empty[kt & 1]);
            if (it.count() == 1) umma_commit(q_empty);
          }
          for (int j = 0; j < it.count(); ++j, ++kt) {
            const bool last = j == it.count() - 1;
            const int t = it.tile(j), w = it.width(t), wn = it.width(it.tile(j + 1));
            if (!(ok = wait_v(it.edge(t)))) break;
            if (!(ok = wait_bounded(&p_full[0], c0 & 1, abort_flag))) break;
            // O_0 is free once the previous item's epilogue has read it
            if (j == 0 && n > 0 && !(ok = wait_bounded(&o_empty[0], (n - 1) & 1, abort_flag))) break;
            tc_fence_after();
            issue_pv(tO0, tS0, 0, w, j > 0);
            ++c0;
            if (last) umma_commit(&o_full[0]);
            const int kn = kt + 1;
            if (!last) {
              if (!(ok = wait_bounded(&k_full[kn & 1], (kn >> 1) & 1, abort_flag))) break;
              tc_fence_after();
              issue_s(tS0, dQ0, kn & 1, wn);
              umma_commit(&s_full[0]);
              if (!has1 && j + 1 == it.count() - 1) umma_commit(q_empty);
            }
            if (has1) {
              if (!(ok = wait_bounded(&p_full[1], c1 & 1, abort_flag))) break;
              if (j == 0 && n1 > 0 && !(ok = wait_bounded(&o_empty[1], (n1 - 1) & 1, abort_flag))) break;
              tc_fence_after();
              issue_pv(tO1, tS1, 0, w, j > 0);
              ++c1;
              if (last) umma_commit(&o_full[1]);
            }
            umma_commit(&v_empty[0]);
            if (!last) {
              if (has1) {
                issue_s(tS1, dQ1, kn & 1, wn);
                umma_commit(&s_full[1]);
                if (j + 1 == it.count() - 1) umma_commit(q_empty);
              }
              umma_commit(&k_empty[kn & 1]);
            }
          }
        }
        ++n;
        if (has1) ++n1;
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax / epilogue
    setmaxnreg_inc<200>();
    const int i = warp >> 2;          // which tile
    const int r = threadIdx.x & 127;  // TMEM lane == row of the tile
    const int tr = r / p.G, hr = r - tr * p.G;  // its token and head
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tbase + lane_off + 256 + i * 128;
    int n = 0;   // items this tile slot took part in
    int tg = 0;  // score tiles it consumed
    bool ok = true;
    // The item stays in shared memory: the loop over key tiles needs every register.
    for (int item = 0; ok && work && (kTiles == 2 || i == 0) && pg_item<true>(queue, i_full, item, abort_flag); ++item) {
      const PgItem& it = queue.it[item % kPgItems];
      const auto done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[item % kPgItems]);
      };
      const int tokens = min(p.TQ, it.tokens - i * p.TQ);  // valid tokens of this tile
      const bool whole = it.t0 == 0 && it.t1 == it.n_kt;
      if (threadIdx.x == 0 && !whole) {
        PgDesc* desc = p.ws_desc + blockIdx.x;
        if (it.t0 > 0) {
          desc->open0 = it.t1 == it.n_kt ? 2 : 1;
        } else {
          desc->open1 = 1;
          desc->row0 = it.tok0;
          desc->h0 = it.g * p.G;
          desc->rows = it.tokens * p.G;
        }
      }
      if (tokens <= 0) {  // no second tile
        done();
        continue;
      }
      const bool row_ok = tr < tokens;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      const int pos0 = it.p0 + i * p.TQ, pos = pos0 + tr;
      const int h = it.g * p.G + hr;
      // the sink joins a whole item here, a divided one when its parts are joined
      const bool sunk = whole && p.sinks && row_ok;
      // a row of no token has a reference from the start, so that it never asks for one
      float m = sunk ? p.sinks[h] * 1.4426950408889634f : row_ok ? -INFINITY : 0.f;
      float l = sunk ? 1.f : 0.f;  // exact row sum (lse)
      float lr = l;                // sum of the bf16-rounded P that enter P.V (output)
      const int wrap = it.start + it.t1 * kPgKeys, span = it.count() * kPgKeys;
      int kpos0 = it.start + it.tile(0) * kPgKeys;  // first key of the tile
      bool later = false;                           // not the first tile to pass
      for (int j = it.count(); j > 0; --j, ++tg, later = true) {
        const int buf = kTiles == 1 ? (tg & 1) : i;
        const int phase = kTiles == 1 ? (tg >> 1) & 1 : tg & 1;
        const uint32_t tS = tbase + lane_off + buf * 128;
        if (!(ok = wait_lanes(&s_full[buf], phase, abort_flag))) break;
        tc_fence_after();
        if (warp_ok) {
          float s[128];
          tmem_load128_sync(tS, s);
          const bool full_tile = kpos0 + kPgKeys - 1 <= pos0 &&
                                 (p.window == 0 || pos0 + tokens - 1 - kpos0 <= p.window - 1);
          if (!full_tile) {
            const int hi_k = pos - kpos0;                                      // keys <= hi_k visible
            const int lo_k = p.window > 0 ? pos - p.window + 1 - kpos0 : -1;  // keys >= lo_k visible
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = (c <= hi_k && c >= lo_k) ? s[c] : -INFINITY;
          }
          // Moves the reference m up to the row max of this tile where need is
          // set (rescaling l, lr and, on later tiles, O by 2^(m_old - m_new)).
          // The whole warp takes part: the O rescale is a warp-wide TMEM access.
          auto move_max = [&](bool need) __attribute__((always_inline)) {
            float mx8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mx8[k] = -INFINITY;
#pragma unroll
            for (int c = 0; c < 64; ++c) mx8[c & 7] = fmax3(mx8[c & 7], s[2 * c], s[2 * c + 1]);
            const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                   fmaxf(mx8[6], mx8[7]));
            const float m_new = fmaxf(m, mx * p.scale_log2);
            float alpha = 1.f;
            bool rescale_o = false;
            if (need && m_new > m) {
              alpha = ex2(m - m_new);  // 0 when m was -inf
              l *= alpha;
              lr *= alpha;
              m = m_new;
              rescale_o = later;
            }
            if (__any_sync(0xffffffffu, rescale_o)) {
              // O must hold the previous key tile's product: with two tiles S(t) was
              // committed after it, with one it may still run
              if (kTiles == 1) {
                const int prev = tg - 1;
                wait_lanes(&v_empty[prev % kVStages], (prev / kVStages) & 1, abort_flag);
                tc_fence_after();
              }
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tmem_load32_sync(tO + c * 32, o);
                const float a_ = rescale_o ? alpha : 1.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a_);
                tmem_st32(tO + c * 32, o);
              }
            }
          };
          // P = 2^(s*scale - m), rounded to bf16 for the P.V product, written over
          // the first 64 columns of S, and its two row sums.
          float2 a, ar;
          auto exps = [&]() __attribute__((always_inline)) {
            const float neg_m = (m == -INFINITY) ? 0.f : -m;
            const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
            const float2 nm2 = make_float2(neg_m, neg_m);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            float2 acr[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t pk[32];
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float2 x = fma2(make_float2(s[64 * half + 2 * c], s[64 * half + 2 * c + 1]), sc2, nm2);
                const float2 e = make_float2(ex2(x.x), ex2(x.y));
                pk[c] = pack_bf16(e.x, e.y);
                acc[c & 1] = add2(acc[c & 1], e);
                add_bf16x2(acr[c & 1], pk[c]);
              }
              tmem_st32(tS + 32 * half, pk);
            }
            a = add2(acc[0], acc[1]);
            ar = add2(acr[0], acr[1]);
          };
          if (__any_sync(0xffffffffu, m == -INFINITY)) move_max(m == -INFINITY);
          exps();
          const auto unsafe = [&]() { return row_ok && !(a.x + a.y <= 0x1p64f); };  // also NaN
          if (__any_sync(0xffffffffu, unsafe())) {
            move_max(unsafe());
            tmem_wait_st();  // the first P stores are complete before they are overwritten
            exps();
          }
          l += a.x + a.y;
          lr += ar.x + ar.y;
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&p_full[buf]);
        kpos0 += kPgKeys;
        if (kpos0 == wrap) kpos0 -= span;
      }
      if (!ok) break;
      // ---------------- epilogue: O is read out of TMEM first and released, so
      // the next item's P.V can start at once.
      if (!(ok = wait_lanes(&o_full[i], n & 1, abort_flag))) break;
      tc_fence_after();
      float o[128];
      tmem_load128_sync(tO, o);
      const bool hidden = *const_cast<volatile int*>(&queue.dirty[item % kPgItems]);
      tc_fence_before();
      mbar_arrive(&o_empty[i]);
      ++n;
      if (hidden && row_ok) {
        float t[128];  // a copy: the call takes an address, and O stays in registers otherwise
#pragma unroll
        for (int e = 0; e < 128; ++e) t[e] = o[e];
        pg_add_hidden(p, it, it.start + it.t0 * kPgKeys, it.start + it.t1 * kPgKeys, it.tok0 + i * p.TQ + tr, h, pos, m,
                      0, t);
#pragma unroll
        for (int e = 0; e < 128; ++e) o[e] = t[e];
      }
      if (row_ok && !whole) {
        const size_t slot = (size_t)blockIdx.x * 2 + (it.t0 == 0 ? 1 : 0);
        const size_t row = slot * (kTiles * 128) + i * 128 + r;
        if (MIMO_ROW_OK(row, (long long)gridDim.x * 2 * kTiles * 128)) {
          p.ws_ml[row] = make_float4(m, l, lr, 0.f);
          float* dst = p.ws_o + row * 128;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            st_global_v8(dst + 8 * e, __float_as_uint(o[8 * e]), __float_as_uint(o[8 * e + 1]),
                         __float_as_uint(o[8 * e + 2]), __float_as_uint(o[8 * e + 3]), __float_as_uint(o[8 * e + 4]),
                         __float_as_uint(o[8 * e + 5]), __float_as_uint(o[8 * e + 6]), __float_as_uint(o[8 * e + 7]));
        }
      } else if (row_ok) {
        const int tok = it.tok0 + i * p.TQ + tr;
        if (MIMO_ROW_OK((long long)tok * p.Hq + h, (long long)p.pb.total_q * p.Hq)) {
          const float f = (lr > 0.f) ? p.v_scale / lr : 0.f;
          const size_t ob = ((size_t)tok * p.Hq + h) * 128;
          if (p.out_f32) {
            float* dst = reinterpret_cast<float*>(p.out) + ob;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              reinterpret_cast<float4*>(dst)[e] =
                  make_float4(o[4 * e] * f, o[4 * e + 1] * f, o[4 * e + 2] * f, o[4 * e + 3] * f);
          } else if (p.out_v8) {
            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.out) + ob;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              st_global_v8(dst + 16 * e, pack_bf16(o[16 * e + 0] * f, o[16 * e + 1] * f),
                           pack_bf16(o[16 * e + 2] * f, o[16 * e + 3] * f),
                           pack_bf16(o[16 * e + 4] * f, o[16 * e + 5] * f),
                           pack_bf16(o[16 * e + 6] * f, o[16 * e + 7] * f),
                           pack_bf16(o[16 * e + 8] * f, o[16 * e + 9] * f),
                           pack_bf16(o[16 * e + 10] * f, o[16 * e + 11] * f),
                           pack_bf16(o[16 * e + 12] * f, o[16 * e + 13] * f),
                           pack_bf16(o[16 * e + 14] * f, o[16 * e + 15] * f));
          } else {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + ob);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              uint4 u;
              u.x = pack_bf16(o[8 * e + 0] * f, o[8 * e + 1] * f);
              u.y = pack_bf16(o[8 * e + 2] * f, o[8 * e + 3] * f);
              u.z = pack_bf16(o[8 * e + 4] * f, o[8 * e + 5] * f);
              u.w = pack_bf16(o[8 * e + 6] * f, o[8 * e + 7] * f);
              dst[e] = u;
            }
          }
          if (p.lse)
            p.lse[(size_t)h * p.pb.total_q + tok] = (l != 0.f) ? (m * 0.6931471805599453f + logf(l)) : -INFINITY;
        }
      }
      done();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // a role gave up: the loads and MMAs still in flight land before the CTA
    // frees its TMEM and exits
    if (warp == 8 && lane == 0) {
      drain_armed(q_full, armed[0], never_flag);
      drain_armed(&k_full[0], (armed[1] + 1) / 2, never_flag);
      drain_armed(&k_full[1], armed[1] / 2, never_flag);
      if (kVStages == 2) {
        drain_armed(&v_full[0], (armed[2] + 1) / 2, never_flag);
        drain_armed(&v_full[1], armed[2] / 2, never_flag);
      } else {
        drain_armed(v_full, armed[2], never_flag);
      }
    }
    if (warp == 9 && lane == 0 && armed[3]) drain_mma(mma_drain, never_flag);  // MMAs may have been issued
    __syncthreads();
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Joins the parts of each divided item and folds the sink in:
//   M = max(sigma, max_c m_c),  Z = 2^(sigma-M) + sum_c 2^(m_c-M) l_c,
//   out = v_scale * sum_c 2^(m_c-M) o_c / Z~,   lse = ln Z + M ln 2
// where Z~ is Z over the parts' sums of the rounded P.  blockIdx.x: the CTA
// whose share ends inside the item; its later parts are slot 0 of the CTAs
// after it, up to the one where it ends.  One warp per row.
template <int kRows>  // of a slot
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedAttnParams p) {
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched before the parts are complete
  if (timed_out_before()) return;  // after a recorded timeout: write nothing
  // both loads at once: this CTA's descriptor, and whether the item ends in one of the next 32
  int k = c + 1 + lane;
  int open0 = k < (int)gridDim.x ? p.ws_desc[k].open0 : 0;
  const PgDesc d = p.ws_desc[c];
  if (!d.open1) return;
  int last = -1;  // the CTA where the item ends
  for (int k0 = c + 1;; k0 += 32) {
    const uint32_t ends = __ballot_sync(0xffffffffu, open0 == 2);
    if (ends) last = k0 + __ffs(ends) - 1;
    if (last >= 0 || k0 + 32 >= (int)gridDim.x) break;
    k = k0 + 32 + lane;
    open0 = k < (int)gridDim.x ? p.ws_desc[k].open0 : 0;
  }
  if (last < 0) return;  // a share gave up
  const int per_tile = p.TQ * p.G;  // valid rows of a full tile
  const int v = blockIdx.y * 8 + warp;
  if (v < d.rows) {
    const int tile = v / per_tile, r = tile * 128 + (v - tile * per_tile);
    const int tok = d.row0 + v / p.G, h = d.h0 + v % p.G;
    if (!MIMO_ROW_OK((long long)tok * p.Hq + h, (long long)p.pb.total_q * p.Hq)) return;
    const float sg = p.sinks ? p.sinks[h] * 1.4426950408889634f : -INFINITY;
    // a lane holds the statistics of one part; further parts come in rounds of 32
    const auto row_of = [&](int k) { return ((size_t)k * 2 + (k == c)) * kRows + r; };
    float M = sg;
    float4 ml = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    // O of the first parts beside the statistics, not after them
    constexpr int kAhead = 4;
    float4 ahead[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      if (c + e <= last) ahead[e] = reinterpret_cast<const float4*>(p.ws_o + row_of(c + e) * 128)[lane];
    for (int k0 = c; k0 <= last; k0 += 32) {
      if (k0 + lane <= last) {
        ml = p.ws_ml[row_of(k0 + lane)];
        M = fmaxf(M, ml.x);
      }
    }
#pragma unroll
    for (int e = 16; e > 0; e >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, e));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float Z = 0.f, Zr = 0.f;
    if (M != -INFINITY) {
      const bool one_round = last - c < 32;
      for (int k0 = c; k0 <= last; k0 += 32) {
        const int parts = min(32, last + 1 - k0);
        if (!one_round) ml = lane < parts ? p.ws_ml[row_of(k0 + lane)] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        const float w = (ml.x == -INFINITY) ? 0.f : ex2(ml.x - M);
        Z += w * ml.y;
        Zr += w * ml.z;
        const auto add = [&](int e, const float4& o) {
          const float we = __shfl_sync(0xffffffffu, w, e);
          acc.x += we * o.x;
          acc.y += we * o.y;
          acc.z += we * o.z;
          acc.w += we * o.w;
        };
        int e0 = 0;
        if (k0 == c) {
#pragma unroll
          for (int e = 0; e < kAhead; ++e)
            if (e < parts) add(e, ahead[e]);
          e0 = kAhead;
        }
#pragma unroll 4
        for (int e = e0; e < parts; ++e) add(e, reinterpret_cast<const float4*>(p.ws_o + row_of(k0 + e) * 128)[lane]);
      }
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) {
        Z += __shfl_xor_sync(0xffffffffu, Z, e);
        Zr += __shfl_xor_sync(0xffffffffu, Zr, e);
      }
      const float ps = (sg == -INFINITY) ? 0.f : ex2(sg - M);
      Z += ps;
      Zr += ps;
    }
    const float f = (Zr > 0.f) ? p.v_scale / Zr : 0.f;
    const size_t ob = ((size_t)tok * p.Hq + h) * 32 + lane;
    if (p.out_f32)
      reinterpret_cast<float4*>(p.out)[ob] = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    else
      reinterpret_cast<uint2*>(p.out)[ob] = make_uint2(pack_bf16(acc.x * f, acc.y * f), pack_bf16(acc.z * f, acc.w * f));
    if (p.lse && lane == 0)
      p.lse[(size_t)h * p.pb.total_q + tok] = (Z != 0.f) ? (M * 0.6931471805599453f + logf(Z)) : -INFINITY;
  }
}

}  // namespace mimo
