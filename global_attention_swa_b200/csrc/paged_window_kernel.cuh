// Attention of a chunk of new tokens over a paged cache under a window so
// short that all keys of an item fit one score tile (tcgen05).
//
// A block is TQ = 128 / G consecutive new tokens of one sequence times the G
// query heads of one key/value head: 128 rows that share their keys.  An item
// is kBlocks blocks.  Together they see at most window - 1 + kBlocks * TQ
// keys; loaded in boxes of 16 from the one that holds the first, that is at
// most kPwKeys = 160 (window 129, 16 heads to a key/value head: 2 blocks of 8
// tokens, 159).  So there is no online softmax, and the work of an item is one
// Q K^T and one P V per block.  The bytes of such a layer are its queries and
// outputs (80 KB a block, against 100 KB of keys and values from L2 for an item),
// so the roles run as a pipeline over blocks: while one block's softmax runs, the
// next one's scores are computed and the queries of the one after are on their way.
//
// Measured on one B200 (64 query heads, 4 key/value heads, window 129, 5197 new
// tokens of 9 sequences, 229 MB): 69.5 us, 3.3 TB/s, 50 % of a plain copy's rate, and
// up to 84 us from box to box (the general kernel: 159 us; one block to an item, at 72
// for two: 79 us).  A CTA passes 17.6 blocks, about 4 us each.  Two chains bind: of one
// block, scores (0.8 us), softmax (2.2), P V (0.6), with two blocks under way, since P
// lies over its scores; and of the one O, whose next P V waits until the epilogue has
// read both halves, the first of them stored before the second is read.  TMEM holds
// two score tiles of 160 columns beside one O.
//
//   warp 12     loads Q (two buffers, a block ahead) and K (once per item, a
//               lane per box of 16 keys; the page table is looked up here)
//   warp 13     MMA issuer: S(n) = Q K^T into score buffer n & 1, then O = P(n-1) V
//   warp 14     loads V (once per item, as K) and zeroes rows of it that
//               may never have been written
//   warp 15     works out the items of this CTA's share, ahead of the others
//   warps 0-7   softmax: warpgroup s takes the blocks with n & 1 == s, one row
//               per thread, one pass over its TMEM row
//   warps 8-11  epilogue: O / l -> out, lse
//
// The value operand carries a third 64-column block of ones and P V runs 144
// columns wide: columns 128..143 of O are the row sum of the bf16-rounded P,
// which normalises the output (P is rounded because the tensor cores take
// 16-bit operands beside bf16 V; the sums are fp32).
//
// TMEM: S_0 [0, 160), S_1 [160, 320), O [320, 448) + row sum [448, 464).
#pragma once

#include "paged_attention_kernel.cuh"

#undef MIMO_FILE_ID
#define MIMO_FILE_ID 15  // site numbers of the checked build

namespace mimo {

constexpr int kPwThreads = 512;
constexpr int kPwKeys = 160;
constexpr int kPwBoxRows = 16;
constexpr int kPwKBox = kPwKeys * 128;                // [keys][64 dims], 1024-aligned
constexpr int kPwOffQ = 0;                            // 2 buffers
constexpr int kPwOffK = 2 * kPgQBytes;                // 3 boxes
constexpr int kPwOffV = kPwOffK + 3 * kPwKBox;        // 2 boxes
constexpr int kPwOffOnes = kPwOffV + 2 * kPwKBox;     // the third value block: ones
constexpr int kPwOffML = kPwOffOnes + kPwKBox;        // [2][128] float4 (m, l, sink term, -)
constexpr int kPwOffBar = kPwOffML + 2 * 128 * 16;
constexpr int kPwOffItems = kPwOffBar + 512;            // barriers and plan before it
constexpr int kPwSmemBytes = kPwOffItems + 512 + 1024;  // the queue of items; alignment slack
constexpr int kPwReaders = 3 + 8 + 4;                   // warps 12, 13, 14, softmax, epilogue
constexpr uint32_t kPwColO = 2 * kPwKeys, kPwColSum = kPwColO + 128;
static_assert(kPwOffOnes % 1024 == 0 && kPwColSum + 16 <= 512 && kPwSmemBytes <= 227 * 1024, "window layout");

// An item's keys, all in one tile.
__device__ __forceinline__ PgTile pw_keys(const PgItem& it) { return pg_keys(it, it.start, kPwKeys); }

// Rows past the sequence's end, and before the first key that its chunk sees, may
// never have been written: they are zeroed before the product, with all that nothing
// of such an item sees.  Elsewhere such rows are seen by another item, and stay: what
// is not finite among them is met as in any hidden key (pw_row_again), and V goes to
// its products without a warp between (with an item fetched ahead by the issuer, 69.5
// against 72.5 us).
__device__ __forceinline__ bool pw_open(const PgItem& it) { return it.outer; }

// The row of the pool's keys and values (of the item's head) at position j; -1 without a page.
__device__ __forceinline__ long long pw_pool_row(const PagedAttnParams& p, const PgItem& it, int j) {
  const int e = p.pb.table[(size_t)it.b * p.pb.max_pages + j / p.pb.page_size];
  return e >= 0 && e < p.pb.num_pages ? ((long long)e * p.pb.page_size + j % p.pb.page_size) * p.Hkv + it.g : -1;
}

// Of the 32 keys from k on, those that enter the item's product with a value that is
// not finite (bit i: key k + i).  By a whole warp.
__device__ __forceinline__ uint32_t pw_not_finite(const PagedAttnParams& p, const PgItem& it, const PgTile& keys, int k) {
  const int lane = threadIdx.x & 31, j = k + lane;
  const bool in = pw_open(it) ? j >= it.lo && j <= it.hi : j < keys.k0 + keys.n;
  const long long row = in ? pw_pool_row(p, it, j) : -1;
  uint32_t found = 0;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    const long long r = __shfl_sync(0xffffffffu, row, i);
    const uint2 v = r >= 0 ? reinterpret_cast<const uint2*>(p.v + r * 128)[lane] : make_uint2(0u, 0u);
    if (__any_sync(0xffffffffu, bf16x2_not_finite(v.x) || bf16x2_not_finite(v.y))) found |= 1u << i;
  }
  return found;
}

// One row (packed row tok, head h, position pos) from the definition, its output
// only: keys that it does not see take no part at all.  For rows whose product over
// the item's keys is not finite, where that of a key they do not see is to blame.  By
// a whole warp: 32 keys at a time, a lane to each for its score, then four value
// columns to a lane.  (Looking the values over as they come instead, one warp ahead of
// the products, cost 23 us of a 69 us call; a test of the products, 2 at most.)  One
// NaN in a chunk of 165 tokens takes a 77 us call to 2.4 ms: 128 rows to a block, 20 us
// each, 32 one after the other; by one thread a row, and for seen values too, 26 ms.
__device__ __forceinline__ void pw_row_again(const PagedAttnParams& p, const PgItem& it, int tok, int h, int pos) {
  if (!MIMO_ROW_OK((long long)tok * p.Hq + h, (long long)p.pb.total_q * p.Hq)) return;
  const int lane = threadIdx.x & 31;
  const uint4* q = reinterpret_cast<const uint4*>(p.q + ((size_t)tok * p.Hq + h) * 192);
  float m = p.sinks ? p.sinks[h] * 1.4426950408889634f : -INFINITY;
  float l = p.sinks ? 1.f : 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int j0 = max(0, pos - p.window + 1); j0 <= pos; j0 += 32) {
    const int j = j0 + lane;
    const long long row = j <= pos ? pw_pool_row(p, it, j) : -1;  // without a page: zero key and value
    float s = 0.f;
    if (row >= 0) {
      const uint4* k = reinterpret_cast<const uint4*>(p.k + row * 192);
#pragma unroll 8
      for (int i = 0; i < 24; ++i) {
        const uint4 a = q[i], b = k[i];
        s += bf16_lo(a.x) * bf16_lo(b.x) + bf16_hi(a.x) * bf16_hi(b.x);
        s += bf16_lo(a.y) * bf16_lo(b.y) + bf16_hi(a.y) * bf16_hi(b.y);
        s += bf16_lo(a.z) * bf16_lo(b.z) + bf16_hi(a.z) * bf16_hi(b.z);
        s += bf16_lo(a.w) * bf16_lo(b.w) + bf16_hi(a.w) * bf16_hi(b.w);
      }
    }
    s = j <= pos ? s * p.scale_log2 : -INFINITY;
    float up = fmaxf(m, s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, d));
    const float neg = up == -INFINITY ? 0.f : -up;
    const float f = ex2(m + neg), pe = ex2(s + neg);
    float sum = pe;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    m = up;
    l = l * f + sum;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll 16
    for (int i = 0; i < 32; ++i) {  // past the last key: weight 0, no row
      const float w = __shfl_sync(0xffffffffu, pe, i);
      const long long r = __shfl_sync(0xffffffffu, row, i);
      const uint2 v = r >= 0 ? reinterpret_cast<const uint2*>(p.v + r * 128)[lane] : make_uint2(0u, 0u);
      o.x += w * bf16_lo(v.x);
      o.y += w * bf16_hi(v.x);
      o.z += w * bf16_lo(v.y);
      o.w += w * bf16_hi(v.y);
    }
  }
  const float f = l != 0.f ? p.v_scale / l : 0.f;
  const size_t ob = ((size_t)tok * p.Hq + h) * 32 + lane;
  if (p.out_f32)
    reinterpret_cast<float4*>(p.out)[ob] = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  else
    reinterpret_cast<uint2*>(p.out)[ob] = make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
}

// The rows of a warp (token a of block blk, head hh of the item's) whose product is not
// finite: done again where a key that the row does not see is to blame.
__device__ __noinline__ void pw_rows_again(const PagedAttnParams& p, const PgItem& it, int blk, int a, int hh, bool odd) {
  const PgTile keys = pw_keys(it);
  const int pos0 = it.p0 + blk * p.TQ, pos = pos0 + a;
  const int c_lo = max(pos - p.window + 1, 0) - keys.k0, c_hi = pos - keys.k0;  // what the row sees
  bool hidden = false;
#pragma unroll 1
  for (int c = 0; c < keys.n; c += 32) {
#pragma unroll 1
    for (uint32_t left = pw_not_finite(p, it, keys, keys.k0 + c); left; left &= left - 1) {
      const int k = c + __ffs(left) - 1;
      hidden |= k < c_lo || k > c_hi;
    }
  }
#pragma unroll 1
  for (uint32_t again = __ballot_sync(0xffffffffu, hidden && odd); again; again &= again - 1) {
    const int src = __ffs(again) - 1;
    const int a_ = __shfl_sync(0xffffffffu, a, src), h = it.g * p.G + __shfl_sync(0xffffffffu, hh, src);
    pw_row_again(p, it, it.tok0 + blk * p.TQ + a_, h, pos0 + a_);
  }
}

template <int kBlocks>
__global__ void __launch_bounds__(kPwThreads, 1)
    paged_window_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttnParams p) {
  extern __shared__ __align__(1024) uint8_t pwsmem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pwsmem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kPwOffBar);
  uint64_t* q_full = bars + 0;     // [2]
  uint64_t* q_empty = bars + 2;    // [2]
  uint64_t* k_full = bars + 4;
  uint64_t* k_empty = bars + 5;
  uint64_t* v_full = bars + 6;
  uint64_t* v_empty = bars + 7;
  uint64_t* v_ready = bars + 8;
  uint64_t* s_full = bars + 10;    // [2]
  uint64_t* p_full = bars + 12;    // [2]
  uint64_t* o_full = bars + 14;
  uint64_t* o_empty = bars + 15;
  uint64_t* ml_full = bars + 16;   // [2]
  uint64_t* ml_empty = bars + 18;  // [2]
  uint64_t* mma_drain = bars + 20;  // teardown after a timed-out wait only
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 21);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 22);
  volatile int* never_flag = reinterpret_cast<volatile int*>(bars + 23);  // never raised
  PgPlace* plan = reinterpret_cast<PgPlace*>(bars + 26);          // [2]
  uint64_t* i_full = bars + 30;                                   // [kPgItems]
  uint64_t* i_empty = bars + 34;                                  // [kPgItems]
  long long* warp_sum = reinterpret_cast<long long*>(bars + 38);  // [16]
  PgQueue& queue = *reinterpret_cast<PgQueue*>(smem + kPwOffItems);
  float4* ml = reinterpret_cast<float4*>(smem + kPwOffML);  // [2][128] (m, l, sink term) per row

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // phases armed: Q for blocks 0, 1, ... (buffer n & 1), K and V per item
  int armed_q = 0, armed_k = 0, armed_v = 0;
  for (int i = threadIdx.x; i < kPwKBox / 4; i += kPwThreads)
    reinterpret_cast<uint32_t*>(smem + kPwOffOnes)[i] = 0x3F803F80u;  // bf16 1.0
  fence_proxy_async_smem();
  if (warp == 12) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&q_full[i], 1);
        mbar_init(&q_empty[i], 1);
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], 128);
        mbar_init(&ml_full[i], 128);
        mbar_init(&ml_empty[i], 128);
      }
      mbar_init(k_full, 1);
      mbar_init(k_empty, 1);
      mbar_init(v_full, 1);
      mbar_init(v_empty, 1);
      mbar_init(v_ready, 1);
      mbar_init(o_full, 1);
      mbar_init(o_empty, 128);
      for (int i = 0; i < kPgItems; ++i) {
        mbar_init(&i_full[i], 1);
        mbar_init(&i_empty[i], kPwReaders);
      }
      mbar_init(mma_drain, 1);
      *never_flag = 0;
      *abort_flag = timed_out_before() ? 1 : 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const bool share = pg_plan<kBlocks, kPwThreads>(p, plan, warp_sum);  // has the barriers the set-up needs
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  const bool work = share && !*abort_flag;

  // Each role takes the same items in turn, and the blocks of each: block n of the
  // CTA's uses buffer n & 1.
  int items = 0;  // taken by this role
  PgItem it;
  const auto next = [&](bool warp_wide) {  // the item is copied and released at once
    if (!(warp_wide ? pg_item<true>(queue, i_full, items, abort_flag) : pg_item<false>(queue, i_full, items, abort_flag)))
      return false;
    it = queue.it[items % kPgItems];
    if (warp_wide) __syncwarp();
    if (!warp_wide || lane == 0) mbar_arrive(&i_empty[items % kPgItems]);
    ++items;
    return true;
  };
  const auto blocks_of = [&](const PgItem& x) { return kBlocks == 2 && x.tokens > p.TQ ? 2 : 1; };

  if (!work) {
    // no share, or a time-out elsewhere
  } else if (warp == 12) {
    // ------------------------------------------------------------ loads
    const auto load_q = [&](const PgItem& x, int blk, int b) {
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[b], p.TQ * p.G * 384);
#pragma unroll
        for (int c = 0; c < 3; ++c)
          tma_load_3d(smem + kPwOffQ + b * kPgQBytes + c * 16384, &tm_q, &q_full[b], c * 64, x.g * p.G,
                      x.tok0 + blk * p.TQ);
      }
      ++armed_q;
    };
    bool ok = true, have = next(true);
    int n = 0, kp = 0;
    if (have) load_q(it, 0, 0);
    PgTile keys = pw_keys(it);
    int boxes = keys.n / kPwBoxRows;
    int row = have && lane < boxes ? pg_box_row(p, it, keys, lane) : 0;
    while (ok && have) {
      const int nblk = blocks_of(it), bytes = boxes * kPwBoxRows * 384, row_now = row, boxes_now = boxes;
      const int g = it.g;
      for (int blk = 0; ok && blk < nblk; ++blk, ++n) {
        if (blk == 0) {
          if (kp >= 1 && !(ok = wait_warp(k_empty, (kp - 1) & 1, abort_flag))) break;
          if (lane == 0) mbar_arrive_expect_tx(k_full, bytes);
          ++armed_k;
          __syncwarp();
          if (lane < boxes_now) {
#pragma unroll
            for (int c = 0; c < 3; ++c)
              tma_load_3d(smem + kPwOffK + c * kPwKBox + lane * kPwBoxRows * 128, &tm_k, k_full, c * 64, g, row_now);
          }
          ++kp;
        }
        // the next block's Q, one block ahead (its buffer was freed by S(n-1));
        // with the item's last block, the next item's pages too
        const int bn = (n + 1) & 1;
        const bool in_item = blk + 1 < nblk;
        if (!in_item) {
          have = next(true);
          if (!have) continue;
          keys = pw_keys(it);
          boxes = keys.n / kPwBoxRows;
          row = lane < boxes ? pg_box_row(p, it, keys, lane) : 0;
        }
        if (n + 1 >= 2 && !(ok = wait_warp(&q_empty[bn], (((n + 1) >> 1) - 1) & 1, abort_flag))) break;
        load_q(it, in_item ? blk + 1 : 0, bn);
      }
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, 144, false, true);  // 128 value dims + 16 ones
      const uint32_t tO = tbase + kPwColO;
      // One low descriptor word per operand, compile-time offsets to it: the one
      // issuing thread is what a block's two products wait for.
      constexpr uint32_t dhi = desc_hi_sw128(1024);
      const uint32_t dQ0 = desc_lo_sw128(sbase + kPwOffQ, 16), dK = desc_lo_sw128(sbase + kPwOffK, 16);
      const uint32_t dV = desc_lo_sw128(sbase + kPwOffV, kPwKBox);
      bool ok = true;
      // O = P(m) V over k keys: 16 to an MMA (P: 8 TMEM columns; V: 16 rows = 2 KB)
      int opened = 0;  // items whose V was zeroed in part: phases of v_ready
      const auto do_pv = [&](int m, int item, int k, bool first_of_item, bool last_of_item, bool open) {
        const int bm = m & 1;
        if (!(ok = wait_bounded(&p_full[bm], (m >> 1) & 1, abort_flag))) return;
        if (first_of_item) {
          if (!(ok = wait_bounded(v_full, item & 1, abort_flag))) return;
          if (open && !(ok = wait_bounded(v_ready, opened++ & 1, abort_flag))) return;
        }
        if (m >= 1 && !(ok = wait_bounded(o_empty, (m - 1) & 1, abort_flag))) return;
        tc_fence_after();
        const uint32_t tP = tbase + bm * kPwKeys;
#pragma unroll
        for (int kk = 0; kk < kPwKeys / 16; ++kk)
          if (kk * 16 < k) umma_ts_lo(tO, tP + kk * 8, dV + ((kk * 2048) >> 4), dhi, idesc_o, kk > 0 ? 1u : 0u);
        if (last_of_item) umma_commit(v_empty);
        umma_commit(o_full);
      };
      int n = 0, kp = 0;
      int pm = -1, pkp = 0, pk = 0;  // previous block: number, item, keys
      bool pfirst = false, plast = false, popen = false;
      bool have = next(false);
      while (ok && have) {
        const int nblk = blocks_of(it);
        const PgTile keys = pw_keys(it);
        const int k = keys.n;
        const bool open = pw_open(it);
        const uint32_t idesc_s = idesc_bf16_f32(128, 0, false, false) | (static_cast<uint32_t>(k >> 3) << 17);
        for (int blk = 0; ok && blk < nblk; ++blk, ++n) {
          const int b = n & 1;
          if (!(ok = wait_bounded(&q_full[b], (n >> 1) & 1, abort_flag))) break;
          if (blk == 0 && !(ok = wait_bounded(k_full, kp & 1, abort_flag))) break;
          tc_fence_after();
          const uint32_t dQ = dQ0 + b * (kPgQBytes >> 4), tS = tbase + b * kPwKeys;
#pragma unroll
          for (int kk = 0; kk < 12; ++kk) {
            const uint32_t off = (kk & 3) * 32;
            umma_ss_lo(tS, dQ + (((kk >> 2) * 16384 + off) >> 4), dK + (((kk >> 2) * kPwKBox + off) >> 4), dhi, idesc_s,
                       kk > 0 ? 1u : 0u);
          }
          umma_commit(&s_full[b]);
          umma_commit(&q_empty[b]);
          if (blk == nblk - 1) {
            umma_commit(k_empty);
            have = next(false);  // here, where the thread would wait for P
          }
          if (pm >= 0) do_pv(pm, pkp, pk, pfirst, plast, popen);
          pm = n;
          pkp = kp;
          pk = k;
          pfirst = blk == 0;
          plast = blk == nblk - 1;
          popen = open;
        }
        ++kp;
      }
      if (ok && pm >= 0) do_pv(pm, pkp, pk, pfirst, plast, popen);
    }
  } else if (warp == 14) {
    // ------------------------------------------------------------ V, and its rows nothing sees
    int kp = 0;
    while (pg_item<true>(queue, i_full, kp, abort_flag)) {
      const PgItem it = queue.it[kp % kPgItems];
      const PgTile keys = pw_keys(it);
      const int boxes = keys.n / kPwBoxRows;
      const int row = lane < boxes ? pg_box_row(p, it, keys, lane) : 0;
      if (kp >= 1 && !wait_warp(v_empty, (kp - 1) & 1, abort_flag)) break;
      if (lane == 0) mbar_arrive_expect_tx(v_full, boxes * kPwBoxRows * 256);
      ++armed_v;
      __syncwarp();
      if (lane < boxes) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          tma_load_3d(smem + kPwOffV + c * kPwKBox + lane * kPwBoxRows * 128, &tm_v, v_full, c * 64, it.g, row);
      }
      if (pw_open(it)) {
        if (!wait_warp(v_full, kp & 1, abort_flag)) break;
        pg_zero_unseen(keys, sbase + kPwOffV, kPwKBox);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_ready);
      }
      if (lane == 0) mbar_arrive(&i_empty[kp % kPgItems]);
      ++kp;
    }
  } else if (warp == 15) {
    if (lane == 0) pg_schedule<kBlocks>(p, plan, queue, i_full, i_empty, abort_flag);
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int s = warp >> 2;               // this warpgroup's blocks: n & 1 == s
    const int r = (warp & 3) * 32 + lane;  // TMEM lane = row = token * G + head
    const int a = r / p.G, hh = r - a * p.G;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int n = 0;
    bool ok = true;
    while (ok && next(true)) {
      const int nblk = blocks_of(it);
      const PgTile keys = pw_keys(it);
      const int N = keys.n;
      for (int blk = 0; ok && blk < nblk; ++blk, ++n) {
        const int b = n & 1;
        if (b != s) continue;
        const int tokens = min(p.TQ, it.tokens - blk * p.TQ);
        // rows 32 and up of this warp's quarter may hold no token at all
        const bool warp_ok = __any_sync(0xffffffffu, a < tokens);
        const int hg = it.g * p.G + hh;
        const int qpos = it.p0 + blk * p.TQ + a;
        const int c_hi = qpos - keys.k0;                              // keys <= qpos
        const int c_lo = max(qpos - p.window + 1, 0) - keys.k0;       // keys in window, >= 0
        const float sg2 = p.sinks && a < tokens ? p.sinks[hg] * 1.4426950408889634f : -INFINITY;
        if (!(ok = wait_lanes(&s_full[b], (n >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        const uint32_t tS = tbase + lane_off + b * kPwKeys;
        float m = sg2, l = 0.f;
        if (warp_ok) {
          // Rows go by token, so a warp's masks lie between its first and its last
          // row's: a run of 16 columns is visible to all rows, to none, or masked, and
          // the warp takes one way.
          const int lo_min = __shfl_sync(0xffffffffu, c_lo, 0), lo_max = __shfl_sync(0xffffffffu, c_lo, 31);
          const int hi_min = __shfl_sync(0xffffffffu, c_hi, 0), hi_max = __shfl_sync(0xffffffffu, c_hi, 31);
          const auto all_see = [&](int c) { return c >= lo_max && c + 15 <= hi_min; };
          const auto none_sees = [&](int c) { return c > hi_max || c + 15 < lo_min; };
          // One pass: P = 2^(s*scale - m) (0 outside the window), bf16 over the same
          // columns (P of columns [c0, c0 + 32) lands in [c0 / 2, c0 / 2 + 16), behind
          // the read position).  The reference m is the sink's logit, or the first
          // visible columns' maximum, and stands while no column exceeds it by more than
          // 64: P is as exact against any reference that neither overflows nor vanishes.
          // Else it moves up by a whole number, by which the P stored so far are scaled
          // exactly; or by more than 256 to the maximum itself, where nothing is left of
          // them (and the rounding of a sum with a far m would be the scores' loss).
          float2 l2 = make_float2(0.f, 0.f);
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll 1
          for (int c0 = 0; c0 < N; c0 += 32) {
            uint32_t v[32], pk[16];
            tmem_load32_sync(tS + c0, v);
            if (!(all_see(c0) && all_see(c0 + 16))) {  // columns at or past N are masked too
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = c0 + e >= c_lo && c0 + e <= c_hi ? v[e] : 0xff800000u;  // -inf
            }
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              mx0 = fmax3(mx0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              mx1 = fmax3(mx1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
            }
            const float mx = fmaxf(mx0, mx1) * p.scale_log2;
            const bool low = mx > m + 64.f;
            if (__any_sync(0xffffffffu, low)) {
              const float up = mx - m > 256.f ? mx : m + ceilf(mx - m);  // infinity too
              const float f = !low || m == -INFINITY ? 1.f : ex2(m - up);  // without a reference all P are 0
              if (low) m = up;
              if (c0 > 0 && __any_sync(0xffffffffu, f != 1.f)) {
                tmem_wait_st();
#pragma unroll 1
                for (int c = 0; c < c0 / 2; c += 16) {
                  tmem_load16_sync(tS + c, pk);
#pragma unroll
                  for (int e = 0; e < 16; ++e) pk[e] = pack_bf16(bf16_lo(pk[e]) * f, bf16_hi(pk[e]) * f);
                  tmem_st16(tS + c, pk);
                }
              }
              l2 = make_float2(l2.x * f, l2.y * f);
            }
            const float neg_m = (m == -INFINITY) ? 0.f : -m;
            const float2 nm2 = make_float2(neg_m, neg_m);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y = fma2(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sc2, nm2);
              const float2 pe = make_float2(ex2(y.x), ex2(y.y));
              pk[e] = pack_bf16(pe.x, pe.y);
              l2 = add2(l2, pe);
            }
            tmem_st16(tS + c0 / 2, pk);
          }
          l = l2.x + l2.y;
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&p_full[b]);
        const float ps = (sg2 != -INFINITY) ? ex2(sg2 - m) : 0.f;  // the sink's term
        if (n >= 2 && !(ok = wait_lanes(&ml_empty[b], ((n >> 1) - 1) & 1, abort_flag))) break;
        ml[b * 128 + r] = make_float4(m, l + ps, ps, 0.f);
        mbar_arrive(&ml_full[b]);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int r = threadIdx.x - 256;
    const int a = r / p.G, hh = r - a * p.G;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tbase + lane_off + kPwColO;
    int n = 0;
    bool ok = true;
    for (int item = 0; ok && pg_item<true>(queue, i_full, item, abort_flag); ++item) {
      const PgItem& it = queue.it[item % kPgItems];
      const int nblk = blocks_of(it);
      for (int blk = 0; ok && blk < nblk; ++blk, ++n) {
        const int b = n & 1;
        if (!(ok = wait_lanes(o_full, n & 1, abort_flag))) break;
        tc_fence_after();
        if (!(ok = wait_lanes(&ml_full[b], (n >> 1) & 1, abort_flag))) break;
        const float4 mlv = ml[b * 128 + r];  // m (base 2), unrounded sum with the sink, the sink's term
        mbar_arrive(&ml_empty[b]);
        float rs[16];
        tmem_load16_sync(tbase + lane_off + kPwColSum, rs);  // rounded-P row sum (16 equal columns)
        const float lr = rs[0] + mlv.z;
        const int tok = it.tok0 + blk * p.TQ + a;
        const int hg = it.g * p.G + hh;
        const bool live = a < min(p.TQ, it.tokens - blk * p.TQ) &&
                          MIMO_ROW_OK((long long)tok * p.Hq + hg, (long long)p.pb.total_q * p.Hq);
        const float f = (lr > 0.f) ? p.v_scale / lr : 0.f;
        const size_t ob = ((size_t)tok * p.Hq + hg) * 128;
        float odd = 0.f;  // NaN once a value of O is not finite
        // O in two 64-column halves (512 threads leave 128 registers each); it is
        // released to the next P V after the second half is in registers
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float o[64];
          tmem_load64_sync(tO + h * 64, o);
          if (h == 1) {
            tc_fence_before();
            mbar_arrive(o_empty);
          }
          if (live) {
#pragma unroll
            for (int e = 0; e < 64; ++e) odd = fmaf(o[e], 0.f, odd);
            if (p.out_f32) {
              float* dst = reinterpret_cast<float*>(p.out) + ob + h * 64;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                reinterpret_cast<float4*>(dst)[e] =
                    make_float4(o[4 * e] * f, o[4 * e + 1] * f, o[4 * e + 2] * f, o[4 * e + 3] * f);
            } else if (p.out_v8) {
              __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.out) + ob + h * 64;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                st_global_v8(dst + 16 * e, pack_bf16(o[16 * e + 0] * f, o[16 * e + 1] * f),
                             pack_bf16(o[16 * e + 2] * f, o[16 * e + 3] * f),
                             pack_bf16(o[16 * e + 4] * f, o[16 * e + 5] * f),
                             pack_bf16(o[16 * e + 6] * f, o[16 * e + 7] * f),
                             pack_bf16(o[16 * e + 8] * f, o[16 * e + 9] * f),
                             pack_bf16(o[16 * e + 10] * f, o[16 * e + 11] * f),
                             pack_bf16(o[16 * e + 12] * f, o[16 * e + 13] * f),
                             pack_bf16(o[16 * e + 14] * f, o[16 * e + 15] * f));
            } else {
              uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + ob + h * 64);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                uint4 u;
                u.x = pack_bf16(o[8 * e + 0] * f, o[8 * e + 1] * f);
                u.y = pack_bf16(o[8 * e + 2] * f, o[8 * e + 3] * f);
                u.z = pack_bf16(o[8 * e + 4] * f, o[8 * e + 5] * f);
                u.w = pack_bf16(o[8 * e + 6] * f, o[8 * e + 7] * f);
                dst[e] = u;
              }
            }
          }
          __syncwarp();  // TMEM is read by the whole warp
        }
        // 0 * v is NaN where v is not finite, so such a value of a key that the row
        // does not see, and another row of the item does, is in its sum
        if (__any_sync(0xffffffffu, odd != 0.f)) pw_rows_again(p, it, blk, a, hh, odd != 0.f);
        if (live && p.lse)
          p.lse[(size_t)hg * p.pb.total_q + tok] =
              (mlv.y != 0.f) ? (mlv.x * 0.6931471805599453f + logf(mlv.y)) : -INFINITY;
        __syncwarp();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[item % kPgItems]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // a role gave up: the loads and MMAs still in flight land before the CTA
    // frees its TMEM and exits
    if (warp == 12 && lane == 0) {
      drain_armed(&q_full[0], (armed_q + 1) / 2, never_flag);
      drain_armed(&q_full[1], armed_q / 2, never_flag);
      drain_armed(k_full, armed_k, never_flag);
    }
    if (warp == 14 && lane == 0) drain_armed(v_full, armed_v, never_flag);
    if (warp == 13 && lane == 0 && work) drain_mma(mma_drain, never_flag);  // MMAs may have been issued
    __syncthreads();
  }
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace mimo
