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
constexpr int kPaPairs = 3;  // vectors in flight per thread: 64 heads' worth at rotary_dim 192,
constexpr int kPaKept = 4;   // and at 64

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

// A row of one token in 16-byte vectors: `turn` pairs of them rotate into each
// other (dimensions 8j.. and half + 8j..), then `keep` are copied (none where
// the destination is the source).
struct PaSplit {
  uint32_t each, magic;  // w / each = w * magic >> 32 for w < 2^22
  __device__ __forceinline__ explicit PaSplit(int n) : each(n), magic(n > 1 ? 0xffffffffu / n + 1 : 0) {}
  __device__ __forceinline__ int row(uint32_t w) const { return each == 1 ? (int)w : (int)__umulhi(w, magic); }
};
struct PaPair {
  uint4 a, b;
};
__device__ __forceinline__ PaPair pa_load(const PaSplit& s, int half, const __nv_bfloat16* src, uint32_t w) {
  const int r = s.row(w), j = w - r * s.each;
  PaPair u;
  u.a = *reinterpret_cast<const uint4*>(src + r * 192 + 8 * j);
  u.b = *reinterpret_cast<const uint4*>(src + r * 192 + half + 8 * j);
  return u;
}
__device__ __forceinline__ void pa_store(const PaSplit& s, int half, __nv_bfloat16* dst, uint32_t w, const PaPair& u,
                                         const float2* cs) {
  const int r = s.row(w), j = w - r * s.each;
  const uint32_t av[4] = {u.a.x, u.a.y, u.a.z, u.a.w}, bv[4] = {u.b.x, u.b.y, u.b.z, u.b.w};
  uint32_t ra[4], rb[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 lo = rope_pair(bf16_lo(av[e]), bf16_lo(bv[e]), cs[8 * j + 2 * e]);
    const float2 hi = rope_pair(bf16_hi(av[e]), bf16_hi(bv[e]), cs[8 * j + 2 * e + 1]);
    ra[e] = pack_bf16(lo.x, hi.x);
    rb[e] = pack_bf16(lo.y, hi.y);
  }
  *reinterpret_cast<uint4*>(dst + r * 192 + 8 * j) = make_uint4(ra[0], ra[1], ra[2], ra[3]);
  *reinterpret_cast<uint4*>(dst + r * 192 + half + 8 * j) = make_uint4(rb[0], rb[1], rb[2], rb[3]);
}
// Offset of copied vector w of rows that keep s.each vectors from dimension 2 half on.
__device__ __forceinline__ int pa_kept(const PaSplit& s, int half, uint32_t w) {
  const int r = s.row(w);
  return r * 192 + 2 * half + 8 * (w - r * s.each);
}

__global__ void __launch_bounds__(kPaThreads, 4) paged_append_kernel(const PagedAppendParams p) {
  __shared__ float2 cs[kRaMaxHalf];
  const int t = blockIdx.x;
  const int half = p.rotary_dim / 2;
  const bool vec = half % 8 == 0;
  const __nv_bfloat16* qs = p.q + (size_t)t * p.Hq * 192;
  __nv_bfloat16* qd = p.q_out + (size_t)t * p.Hq * 192;
  const PaSplit turn(half / 8), keep(24 - 2 * (half / 8));
  const uint32_t qt = p.Hq * turn.each, qk = p.q == p.q_out ? 0 : p.Hq * keep.each;
  if (!MIMO_ROW_OK(t, p.pb.total_q)) return;
  PaPair u[kPaPairs];
  uint4 c[kPaKept];
  if (vec) {
#pragma unroll
    for (int i = 0; i < kPaPairs; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qt) u[i] = pa_load(turn, half, qs, w);
    }
#pragma unroll
    for (int i = 0; i < kPaKept; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qk) c[i] = *reinterpret_cast<const uint4*>(qs + pa_kept(keep, half, w));
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
    float sn, co;
    sincosf(r, &sn, &co);
    cs[threadIdx.x] = make_float2(co, sn);
  }
  __syncthreads();
  const __nv_bfloat16* ks = p.k_new + (size_t)t * p.Hkv * 192;
  __nv_bfloat16* kd = p.k_pages + (kv ? slot : 0) * p.Hkv * 192;
  if (vec) {
#pragma unroll
    for (int i = 0; i < kPaPairs; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qt) pa_store(turn, half, qd, w, u[i], cs);
    }
#pragma unroll
    for (int i = 0; i < kPaKept; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qk) *reinterpret_cast<uint4*>(qd + pa_kept(keep, half, w)) = c[i];
    }
    // what a CTA of this size does not hold at once
    for (uint32_t w = threadIdx.x + kPaPairs * kPaThreads; w < qt; w += kPaThreads)
      pa_store(turn, half, qd, w, pa_load(turn, half, qs, w), cs);
    for (uint32_t w = threadIdx.x + kPaKept * kPaThreads; w < qk; w += kPaThreads)
      *reinterpret_cast<uint4*>(qd + pa_kept(keep, half, w)) = *reinterpret_cast<const uint4*>(qs + pa_kept(keep, half, w));
    if (kv) {
      for (uint32_t w = threadIdx.x; w < p.Hkv * turn.each; w += kPaThreads)
        pa_store(turn, half, kd, w, pa_load(turn, half, ks, w), cs);
      for (uint32_t w = threadIdx.x; w < p.Hkv * keep.each; w += kPaThreads)
        *reinterpret_cast<uint4*>(kd + pa_kept(keep, half, w)) = *reinterpret_cast<const uint4*>(ks + pa_kept(keep, half, w));
    }
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
