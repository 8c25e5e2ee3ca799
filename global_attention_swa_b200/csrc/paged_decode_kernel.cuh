// The decode step over a paged cache: one new token per sequence and at most 16
// query heads to a key/value head.
//
// Bound by the cache's bytes: 16 rows do 16 flop for a byte of K and V, which
// the warp-level mma.sync.m16n8k16 carries while the bytes stream in; a
// tcgen05 tile would spend its 128 rows on them.  So a CTA is small, two share
// an SM (2 x 80 KB of keys and values in flight), and one's merge and epilogue
// overlap the other's loads.
//
// The items, their cuts and the combine kernel are those of
// paged_attention_kernel with a tile of one token's rows: an item is one
// key/value head of one sequence.
//
//   warp 4      loads: K and V in tiles of 64 keys through two stages (TMA, a
//               lane per box; the page table is looked up here), Q rows ahead
//   warps 0-3   16 keys of every tile each: scores, online softmax (base 2),
//               P V in registers; joined at an item's end
//
// Measured on one B200 (64 query heads, 4 key/value heads): 64 sequences of 1024
// to 32768 keys, 3.27 GB in 514 to 527 us, 6.3 TB/s, 95 to 97 % of a plain copy's
// rate; under a window of 129, 23.8 MB in 12 us, where latency binds: the share is
// found (2 us), its pages and loads (2), three tiles (3), the join (2), one after the
// other.  The general kernel takes 536 and 21 to 24 us; three sequences of up to
// 700 keys 15.3 here, 1 us more there.
//
// P is rounded to bf16 for the P V product (bf16 V) and the output normalised
// by the sum of the rounded values; everything else is fp32.
#pragma once

#include "paged_attention_kernel.cuh"

#undef MIMO_FILE_ID
#define MIMO_FILE_ID 16  // site numbers of the checked build

namespace mimo {

constexpr int kPdThreads = 160;
constexpr int kPdRows = 16;
constexpr int kPdKeys = 64;
constexpr int kPdStages = 2;
constexpr int kPdBox = kPdKeys * 128;           // [keys][64 dims]
constexpr int kPdStageBytes = 5 * kPdBox;       // K: 3 boxes, V: 2 boxes
constexpr int kPdQBox = kPdRows * 128;          // [heads][64 dims]
constexpr int kPdQBytes = 3 * kPdQBox;
constexpr int kPdORow = 136;                    // padded row of the merge buffers
constexpr int kPdOffQ = kPdStages * kPdStageBytes;          // 2 buffers
constexpr int kPdOffO = kPdOffQ + 2 * kPdQBytes;            // 2 x [16][kPdORow] fp32
constexpr int kPdOffML = kPdOffO + 2 * kPdRows * kPdORow * 4;  // 3 x [4][16]: max, sum, rounded sum
constexpr int kPdOffBar = kPdOffML + 3 * 4 * kPdRows * 4;
constexpr int kPdSmemBytes = kPdOffBar + 256 + 1024;  // barriers, plan; alignment slack
static_assert(2 * (kPdSmemBytes + 1024) <= 228 * 1024, "two CTAs to an SM");

__global__ void __launch_bounds__(kPdThreads, 2)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttnParams p) {
  extern __shared__ __align__(1024) uint8_t pdsmem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pdsmem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kPdOffBar);
  uint64_t* full = bars + 0;     // [2]
  uint64_t* empty = bars + 2;    // [2]
  uint64_t* q_full = bars + 4;   // [2]
  uint64_t* q_empty = bars + 6;  // [2]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 8);
  volatile int* never_flag = reinterpret_cast<volatile int*>(bars + 9);  // never raised
  volatile int* fine = reinterpret_cast<volatile int*>(bars + 10);       // [2][4]: a consumer warp saw no time-out
  PgPlace* plan = reinterpret_cast<PgPlace*>(bars + 14);                 // [2]
  long long* warp_sum = reinterpret_cast<long long*>(bars + 18);         // [5]
  float* so = reinterpret_cast<float*>(smem + kPdOffO);
  float* sm = reinterpret_cast<float*>(smem + kPdOffML);
  float* sl = sm + 4 * kPdRows;
  float* slr = sl + 4 * kPdRows;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 128) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 4);
    }
    *never_flag = 0;
    // sampled once, so every thread of the CTA sees the same decision
    *abort_flag = timed_out_before() ? 1 : 0;
    fence_mbar_init();
  }
  const bool share = pg_plan<1, kPdThreads>(p, plan, warp_sum);  // has the barriers the set-up needs
  const bool work = share && !*abort_flag;
  if (threadIdx.x == 0 && p.split) p.ws_desc[blockIdx.x] = PgDesc{};
  // the combine kernel may be set up while this one runs; it waits for its end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!work) return;

  PgWalk<1> walk(p, plan);
  PgItem it;
  if (warp == 4) {
    // ------------------------------------------------------------ loads
    int n = 0, kt = 0;  // items, tiles
    bool ok = true;
    while (ok && walk.next(p, it)) {
      const int end = min(it.hi + 1, it.start + it.t1 * kPgKeys);
      int k0 = it.start + it.t0 * kPgKeys;
      // a tile's boxes and the lanes' pool rows, looked up a tile ahead of its loads
      int boxes, row;
      const auto look_up = [&]() {
        PgTile tl;
        tl.k0 = k0;
        boxes = (min(kPdKeys, end - k0) + p.box_rows - 1) / p.box_rows;
        row = lane < boxes ? pg_box_row(p, it, tl, lane) : 0;
      };
      look_up();
      const int qb = n & 1;
      if (n >= 2 && !(ok = wait_warp(&q_empty[qb], ((n >> 1) - 1) & 1, abort_flag))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[qb], p.G * 384);
#pragma unroll
        for (int c = 0; c < 3; ++c)
          tma_load_3d(smem + kPdOffQ + qb * kPdQBytes + c * kPdQBox, &tm_q, &q_full[qb], c * 64, it.g * p.G, it.tok0);
      }
      ++n;
      while (k0 < end) {
        const int st = kt & 1;
        if (kt >= kPdStages && !(ok = wait_warp(&empty[st], ((kt >> 1) - 1) & 1, abort_flag))) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], boxes * p.box_rows * 640);
        __syncwarp();
        if (lane < boxes) {
          uint8_t* kb = smem + st * kPdStageBytes + lane * p.box_rows * 128;
#pragma unroll
          for (int c = 0; c < 3; ++c) tma_load_3d(kb + c * kPdBox, &tm_k, &full[st], c * 64, it.g, row);
#pragma unroll
          for (int c = 0; c < 2; ++c) tma_load_3d(kb + (3 + c) * kPdBox, &tm_v, &full[st], c * 64, it.g, row);
        }
        ++kt;
        k0 += kPdKeys;
        if (k0 < end) look_up();
      }
    }
    // the CTA never exits with copies in flight (after a timed-out wait the
    // consumers may have stopped waiting for them); every item counted had its
    // Q armed, and every tile counted its K and V
    drain_armed(&full[0], (kt + 1) / 2, never_flag);
    drain_armed(&full[1], kt / 2, never_flag);
    drain_armed(&q_full[0], (n + 1) / 2, never_flag);
    drain_armed(&q_full[1], n / 2, never_flag);
    return;
  }
  // -------------------------------------------------------------- consumers
  const int r0 = lane >> 2;       // rows (heads) r0 and r0 + 8
  const int cq = (lane & 3) * 2;  // column pair within an 8-wide block
  const int kw = warp * 16;       // this warp's 16 keys of each tile
  const uint32_t sbase = smem_u32(smem);
  int n = 0, kt = 0;
  bool ok = true;
  while (ok && walk.next(p, it)) {
    const int rows = p.G;
    const int qb = n & 1;
    // the sink of the row that this thread writes: here, a load off the item's end
    const int row = threadIdx.x >> 3;
    const float sg = p.sinks && row < rows ? p.sinks[it.g * p.G + row] * 1.4426950408889634f : -INFINITY;
    uint32_t qa[12][4];
    if ((ok = wait_lanes(&q_full[qb], (n >> 1) & 1, abort_flag))) {
      // fragments of all 12 k-steps of 16 dims; rows that hold nothing are zero
      const uint32_t qs = sbase + kPdOffQ + qb * kPdQBytes;
#pragma unroll
      for (int kk = 0; kk < 12; ++kk) {
        ldsm_x4(qs + (kk >> 2) * kPdQBox + sw128_offset(lane & 15, (kk & 3) * 16 + (lane >> 4) * 8), qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3]);
        if (r0 >= rows) qa[kk][0] = qa[kk][2] = 0u;
        if (r0 + 8 >= rows) qa[kk][1] = qa[kk][3] = 0u;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[qb]);
    }
    float o[16][4];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY;  // running max (base 2)
    float l0 = 0.f, l1 = 0.f;              // per-thread partial sums (lse)
    float lr0 = 0.f, lr1 = 0.f;            // the same over the rounded P (output normaliser)
    const int end = min(it.hi + 1, it.start + it.t1 * kPgKeys);
    for (int k0 = it.start + it.t0 * kPgKeys; ok && k0 < end; k0 += kPdKeys, ++kt) {
      const int st = kt & 1;
      if (!(ok = wait_lanes(&full[st], (kt >> 1) & 1, abort_flag))) break;
      const int kpos = k0 + kw;  // this warp's first key
      if (kpos < end && kpos + 15 >= it.lo) {
        const uint32_t kb = sbase + st * kPdStageBytes;
        const uint32_t vb = kb + 3 * kPdBox;
        // ---- S = Q K^T for 16 keys (two n-blocks of 8).  ldmatrix.x4 rows: lanes 0-7
        // keys 0..7 dims +0; 8-15 the same dims +8; 16-31 keys 8..15.
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        float s1[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // odd steps: two shorter chains
        {
          const int krow = kw + (lane & 7) + ((lane >> 4) << 3);
          const int kcol = ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int kk = 0; kk < 12; ++kk) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kb + (kk >> 2) * kPdBox + sw128_offset(krow, (kk & 3) * 16 + kcol), b0, b1, b2, b3);
            mma_bf16_16816(kk & 1 ? s1[0] : s[0], qa[kk], b0, b1);
            mma_bf16_16816(kk & 1 ? s1[1] : s[1], qa[kk], b2, b3);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e >> 2][e & 3] += s1[e >> 2][e & 3];
        }
        // ---- scale to base 2, mask, running max
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = kpos + (e >> 1) * 8 + cq + (e & 1);
          const bool seen = key < end && key >= it.lo;  // all rows are the same token's
          float& a = s[e >> 1][e & 1];
          float& b = s[e >> 1][2 + (e & 1)];
          a = seen ? a * p.scale_log2 : -INFINITY;
          b = seen ? b * p.scale_log2 : -INFINITY;
          mx0 = fmaxf(mx0, a);
          mx1 = fmaxf(mx1, b);
        }
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
        const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
        // a row that has seen no key yet has no reference: any will do for its zeros
        const float ref0 = mn0 == -INFINITY ? 0.f : mn0, ref1 = mn1 == -INFINITY ? 0.f : mn1;
        const float a0 = ex2(m0 - ref0), a1 = ex2(m1 - ref1);
        m0 = mn0;
        m1 = mn1;
        uint32_t pa[4];
        {
          const float p00 = ex2(s[0][0] - ref0), p01 = ex2(s[0][1] - ref0);
          const float p02 = ex2(s[0][2] - ref1), p03 = ex2(s[0][3] - ref1);
          const float p10 = ex2(s[1][0] - ref0), p11 = ex2(s[1][1] - ref0);
          const float p12 = ex2(s[1][2] - ref1), p13 = ex2(s[1][3] - ref1);
          pa[0] = pack_bf16(p00, p01);
          pa[1] = pack_bf16(p02, p03);
          pa[2] = pack_bf16(p10, p11);
          pa[3] = pack_bf16(p12, p13);
          l0 = l0 * a0 + ((p00 + p01) + (p10 + p11));
          l1 = l1 * a1 + ((p02 + p03) + (p12 + p13));
          lr0 = lr0 * a0 + ((bf16_lo(pa[0]) + bf16_hi(pa[0])) + (bf16_lo(pa[2]) + bf16_hi(pa[2])));
          lr1 = lr1 * a1 + ((bf16_lo(pa[1]) + bf16_hi(pa[1])) + (bf16_lo(pa[3]) + bf16_hi(pa[3])));
        }
        // rescale O only when some row's running max moved (2^0 is exactly 1)
        if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            o[e][0] *= a0;
            o[e][1] *= a0;
            o[e][2] *= a1;
            o[e][3] *= a1;
          }
        }
        // ---- O += P V.  ldmatrix.trans rows: lanes 0-7 keys 0..7, 8-15 keys 8..15
        // (dims +0), 16-31 the same at dims +8.
        const int vrow = kw + (lane & 7) + (((lane >> 3) & 1) << 3);
        const int vcol = (lane >> 4) * 8;
        // values that nothing sees may be anything: zeroed.  This thread holds keys
        // cq + {0, 1} (b0, b2) and 8 + cq + {0, 1} (b1, b3).
        const bool partial = kpos + 16 > end || kpos < it.lo;
        const auto seen = [&](int key) { return key < end && key >= it.lo; };
        const uint32_t mk0 = (seen(kpos + cq) ? 0x0000FFFFu : 0u) | (seen(kpos + cq + 1) ? 0xFFFF0000u : 0u);
        const uint32_t mk1 = (seen(kpos + 8 + cq) ? 0x0000FFFFu : 0u) | (seen(kpos + 9 + cq) ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int n2 = 0; n2 < 8; ++n2) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(vb + (n2 >> 2) * kPdBox + sw128_offset(vrow, (n2 & 3) * 16 + vcol), b0, b1, b2, b3);
          if (partial) {
            b0 &= mk0; b1 &= mk1; b2 &= mk0; b3 &= mk1;
          }
          mma_bf16_16816(o[2 * n2], pa, b0, b1);
          mma_bf16_16816(o[2 * n2 + 1], pa, b2, b3);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    // ---- join the four warps: a common reference, then two warps' O at a time
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    lr0 += __shfl_xor_sync(0xffffffffu, lr0, 1);
    lr0 += __shfl_xor_sync(0xffffffffu, lr0, 2);
    lr1 += __shfl_xor_sync(0xffffffffu, lr1, 1);
    lr1 += __shfl_xor_sync(0xffffffffu, lr1, 2);
    if ((lane & 3) == 0) {
      sm[warp * kPdRows + r0] = m0;
      sm[warp * kPdRows + r0 + 8] = m1;
      sl[warp * kPdRows + r0] = l0;
      sl[warp * kPdRows + r0 + 8] = l1;
      slr[warp * kPdRows + r0] = lr0;
      slr[warp * kPdRows + r0 + 8] = lr1;
    }
    if (lane == 0) fine[(n & 1) * 4 + warp] = ok;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    {
      float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        M0 = fmaxf(M0, sm[w * kPdRows + r0]);
        M1 = fmaxf(M1, sm[w * kPdRows + r0 + 8]);
      }
      const float w0 = M0 == -INFINITY ? 0.f : ex2(m0 - M0), w1 = M1 == -INFINITY ? 0.f : ex2(m1 - M1);
      float* mine = so + (warp & 1) * kPdRows * kPdORow;
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {
        if ((warp >> 1) == turn) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2* a = reinterpret_cast<float2*>(mine + r0 * kPdORow + e * 8 + cq);
            float2* b = reinterpret_cast<float2*>(mine + (r0 + 8) * kPdORow + e * 8 + cq);
            float2 x = make_float2(o[e][0] * w0, o[e][1] * w0), y = make_float2(o[e][2] * w1, o[e][3] * w1);
            if (turn == 1) {
              x = make_float2(a->x + x.x, a->y + x.y);
              y = make_float2(b->x + y.x, b->y + y.y);
            }
            *a = x;
            *b = y;
          }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
      }
    }
    // every warp comes to the same decision: the flags change only two items on
    ok = fine[(n & 1) * 4] && fine[(n & 1) * 4 + 1] && fine[(n & 1) * 4 + 2] && fine[(n & 1) * 4 + 3];
    // ---- 128 threads: row tid / 8, columns 4 (tid & 7) + 32 j
    const int tid = threadIdx.x, cb = (tid & 7) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sm[w * kPdRows + row]);
    float L = 0.f, Lr = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float wgt = M == -INFINITY ? 0.f : ex2(sm[w * kPdRows + row] - M);
      L += wgt * sl[w * kPdRows + row];
      Lr += wgt * slr[w * kPdRows + row];
    }
    float4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 a = *reinterpret_cast<const float4*>(so + row * kPdORow + cb + 32 * j);
      const float4 b = *reinterpret_cast<const float4*>(so + (kPdRows + row) * kPdORow + cb + 32 * j);
      acc[j] = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
    }
    const bool whole = it.t0 == 0 && it.t1 == it.n_kt;
    if (ok && !whole && tid == 0) {
      PgDesc* desc = p.ws_desc + blockIdx.x;
      if (it.t0 > 0) {
        desc->open0 = it.t1 == it.n_kt ? 2 : 1;
      } else {
        desc->open1 = 1;
        desc->row0 = it.tok0;
        desc->h0 = it.g * p.G;
        desc->rows = rows;
      }
    }
    if (ok && row < rows) {
      const int tok = it.tok0, h = it.g * p.G + row;
      if (!whole) {
        const size_t at = ((size_t)blockIdx.x * 2 + (it.t0 == 0 ? 1 : 0)) * kPdRows + row;
        if (MIMO_ROW_OK(at, (long long)gridDim.x * 2 * kPdRows)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) *reinterpret_cast<float4*>(p.ws_o + at * 128 + cb + 32 * j) = acc[j];
          if ((tid & 7) == 0) p.ws_ml[at] = make_float4(M, L, Lr, 0.f);
        }
      } else if (MIMO_ROW_OK((long long)tok * p.Hq + h, (long long)p.pb.total_q * p.Hq)) {
        // fold the sink: it joins the normaliser only
        const float Mf = fmaxf(M, sg);
        const float scl = M == -INFINITY ? 0.f : ex2(M - Mf), ps = sg == -INFINITY ? 0.f : ex2(sg - Mf);
        const float Lf = L * scl + ps, Lrf = Lr * scl + ps;
        const float f = (Lrf > 0.f) ? p.v_scale * scl / Lrf : 0.f;
        const size_t ob = ((size_t)tok * p.Hq + h) * 128 + cb;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (p.out_f32)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + ob + 32 * j) =
                make_float4(acc[j].x * f, acc[j].y * f, acc[j].z * f, acc[j].w * f);
          else
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + ob + 32 * j) =
                make_uint2(pack_bf16(acc[j].x * f, acc[j].y * f), pack_bf16(acc[j].z * f, acc[j].w * f));
        }
        if (p.lse && (tid & 7) == 0)
          p.lse[(size_t)h * p.pb.total_q + tok] = (Lf != 0.f) ? (Mf * 0.6931471805599453f + logf(Lf)) : -INFINITY;
      }
    }
    ++n;
    // the next item's join writes what this one's threads still read
    asm volatile("bar.sync 1, 128;" ::: "memory");
  }
}

}  // namespace mimo
