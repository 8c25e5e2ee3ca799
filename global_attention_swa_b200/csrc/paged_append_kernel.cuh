// Rotary position embedding of a chunk of new tokens' queries and keys, and
// the write of their keys and values into the pages of the cache.
//
// The paged counterpart of rope_append_kernel: the same rotation (rotate-half,
// angles formed in double precision) at position p = L - n + i of token i of
// the chunk; the key and value go to slot p % page_size of page
// block_table[b][p / page_size].
//
// One CTA per token: the angles of a position are formed once and used by its
// Hq + Hkv rows.  The step moves bytes and little else, so the CTA asks for the
// token's queries first, all of them at once (16-byte vectors), and finds the
// token's sequence, page and angles while they are on their way.
#pragma once

#include "paged_common.cuh"
#include "rope_append_kernel.cuh"

#undef MIMO_FILE_ID
#define MIMO_FILE_ID 12  // site numbers of the checked build

namespace mimo {

constexpr int kPaThreads = 256;
constexpr int kPaBatch = 6;  // units in flight per thread: 64 heads' worth in a CTA

struct PagedAppendParams {
  PagedBatch pb;
  const __nv_bfloat16* q;       // [total_q, Hq, 192]
  __nv_bfloat16* q_out;         // the same shape; may be q
  const __nv_bfloat16* k_new;   // [total_q, Hkv, 192], before rotation
  const __nv_bfloat16* v_new;   // [total_q, Hkv, 128]
  __nv_bfloat16* k_pages;       // [num_pages, page_size, Hkv, 192]
  __nv_bfloat16* v_pages;       // [num_pages, page_size, Hkv, 128]
  int Hq, Hkv;
  int rotary_dim;               // even, <= 192
  double inv_freq[kRaMaxHalf];  // theta^(-2 i / rotary_dim)
};

// The rows of one token in units of 16 bytes: `turn` pairs of vectors that
// rotate into each other (dimensions 8j.. and half + 8j..), then `keep` vectors
// that are copied (none where the destination is the source).
struct PaRows {
  int turn, keep, each;
  uint32_t magic;  // w / each = w * magic >> 32 for w < 2^22
  __device__ __forceinline__ PaRows(int half, bool in_place)
      : turn(half / 8), keep(in_place ? 0 : 24 - 2 * (half / 8)), each(turn + keep) {
    magic = each > 0 ? 0xffffffffu / each + 1 : 0;
  }
};
struct PaUnit {
  uint4 a, b;
};
__device__ __forceinline__ void pa_place(const PaRows& s, int half, uint32_t w, int& row, int& j, int& x, int& y) {
  row = s.each == 1 ? (int)w : (int)__umulhi(w, s.magic);
  j = (int)w - row * s.each;
  x = j < s.turn ? 8 * j : 2 * half + 8 * (j - s.turn);
  y = j < s.turn ? half + 8 * j : -1;
}
__device__ __forceinline__ PaUnit pa_load(const PaRows& s, int half, const __nv_bfloat16* src, uint32_t w) {
  int row, j, x, y;
  pa_place(s, half, w, row, j, x, y);
  PaUnit u;
  u.a = *reinterpret_cast<const uint4*>(src + row * 192 + x);
  u.b = y >= 0 ? *reinterpret_cast<const uint4*>(src + row * 192 + y) : make_uint4(0, 0, 0, 0);
  return u;
}
__device__ __forceinline__ void pa_store(const PaRows& s, int half, __nv_bfloat16* dst, uint32_t w, const PaUnit& u,
                                         const float2* cs) {
  int row, j, x, y;
  pa_place(s, half, w, row, j, x, y);
  if (y < 0) {
    *reinterpret_cast<uint4*>(dst + row * 192 + x) = u.a;
    return;
  }
  const uint32_t av[4] = {u.a.x, u.a.y, u.a.z, u.a.w}, bv[4] = {u.b.x, u.b.y, u.b.z, u.b.w};
  uint32_t ra[4], rb[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 lo = rope_pair(bf16_lo(av[e]), bf16_lo(bv[e]), cs[8 * j + 2 * e]);
    const float2 hi = rope_pair(bf16_hi(av[e]), bf16_hi(bv[e]), cs[8 * j + 2 * e + 1]);
    ra[e] = pack_bf16(lo.x, hi.x);
    rb[e] = pack_bf16(lo.y, hi.y);
  }
  *reinterpret_cast<uint4*>(dst + row * 192 + x) = make_uint4(ra[0], ra[1], ra[2], ra[3]);
  *reinterpret_cast<uint4*>(dst + row * 192 + y) = make_uint4(rb[0], rb[1], rb[2], rb[3]);
}

__global__ void __launch_bounds__(kPaThreads) paged_append_kernel(const PagedAppendParams p) {
  __shared__ float2 cs[kRaMaxHalf];
  const int t = blockIdx.x;
  const int half = p.rotary_dim / 2;
  const bool vec = half % 8 == 0;
  const __nv_bfloat16* qs = p.q + (size_t)t * p.Hq * 192;
  __nv_bfloat16* qd = p.q_out + (size_t)t * p.Hq * 192;
  const PaRows qr(half, p.q == p.q_out), kr(half, false);
  const uint32_t qn = p.Hq * qr.each;
  if (!MIMO_ROW_OK(t, p.pb.total_q)) return;
  PaUnit u[kPaBatch];
  if (vec) {
#pragma unroll
    for (int i = 0; i < kPaBatch; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qn) u[i] = pa_load(qr, half, qs, w);
    }
  }
  const int b = paged_seq_of_row(p.pb, t);  // the whole CTA takes the same branches
  if (b < 0) return;
  const PagedSeq s = paged_seq(p.pb, b);
  if (!s.ok || t < s.b0 || t >= s.b0 + s.n) {
    if (!s.ok && threadIdx.x == 0) record_status(1 /* MIMO_ERR_INVALID_ARG */);
    return;
  }
  const int pos = s.len - s.n + (t - s.b0);
  const int page = paged_page(p.pb, b, pos / p.pb.page_size);
  const long long slot = (long long)page * p.pb.page_size + pos % p.pb.page_size;
  const bool kv = page >= 0 && MIMO_ROW_OK(slot, (long long)p.pb.num_pages * p.pb.page_size);
  if (threadIdx.x < half) {
    // the angle in double, reduced to [-pi, pi] before the fp32 sine and cosine
    const double a = (double)pos * p.inv_freq[threadIdx.x];
    const float r = (float)fma(-6.283185307179586476925286766559, rint(a * 0.15915494309189533576888376337251), a);
    float sn, c;
    sincosf(r, &sn, &c);
    cs[threadIdx.x] = make_float2(c, sn);
  }
  __syncthreads();
  const __nv_bfloat16* ks = p.k_new + (size_t)t * p.Hkv * 192;
  __nv_bfloat16* kd = p.k_pages + (kv ? slot : 0) * p.Hkv * 192;
  if (vec) {
#pragma unroll
    for (int i = 0; i < kPaBatch; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qn) pa_store(qr, half, qd, w, u[i], cs);
    }
    for (uint32_t w = threadIdx.x + kPaBatch * kPaThreads; w < qn; w += kPaThreads)
      pa_store(qr, half, qd, w, pa_load(qr, half, qs, w), cs);
    if (kv)
      for (uint32_t w = threadIdx.x; w < (uint32_t)(p.Hkv * kr.each); w += kPaThreads)
        pa_store(kr, half, kd, w, pa_load(kr, half, ks, w), cs);
  } else {
    // a pair at a time
    const int rows = p.Hq + (kv ? p.Hkv : 0);
    const int tail = 192 - 2 * half, each = half + tail;
    for (int w = threadIdx.x; w < rows * each; w += kPaThreads) {
      const int r = w / each, j = w % each;
      const __nv_bfloat16* src = r < p.Hq ? qs + r * 192 : ks + (r - p.Hq) * 192;
      __nv_bfloat16* dst = r < p.Hq ? qd + r * 192 : kd + (r - p.Hq) * 192;
      if (j < half) {
        const float2 x = rope_pair(__bfloat162float(src[j]), __bfloat162float(src[j + half]), cs[j]);
        dst[j] = __float2bfloat16_rn(x.x);
        dst[j + half] = __float2bfloat16_rn(x.y);
      } else {
        dst[half + j] = src[half + j];
      }
    }
  }
  if (kv) {
    const uint4* vs = reinterpret_cast<const uint4*>(p.v_new + (size_t)t * p.Hkv * 128);
    uint4* vd = reinterpret_cast<uint4*>(p.v_pages + slot * p.Hkv * 128);
    for (int w = threadIdx.x; w < p.Hkv * 16; w += kPaThreads) vd[w] = vs[w];
  }
}

}  // namespace mimo
