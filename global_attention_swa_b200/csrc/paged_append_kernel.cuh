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
// token's queries, keys and values first, all at once (16-byte vectors), and
// finds the token's sequence, page and angles while they are on their way.
//
// Measured on one B200 (64 query heads, 4 key/value heads): 4375 tokens, rotary
// dimension 64, 237 MB in 39.4 us, 6.0 TB/s, 92 % of a plain copy's rate (46.5
// when the loads waited for the page); 48 tokens in 4.8 us, a launch and one
// chain of loads.
#pragma once

#include "paged_common.cuh"
#include "rope_append_kernel.cuh"

#undef MIMO_FILE_ID
#define MIMO_FILE_ID 12  // site numbers of the checked build

namespace mimo {

constexpr int kPaThreads = 256;

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

// kPairs pairs and kKept vectors of the queries per thread are held at once, six
// vectors in all: the 64 heads of a token at any rotary_dim that is a multiple
// of 64 (kPairs 3 at 192, 2 at 128, 1 at 64).
template <int kPairs, int kKept>
__global__ void __launch_bounds__(kPaThreads, 4) paged_append_kernel(const PagedAppendParams p) {
  __shared__ float2 cs[kRaMaxHalf];
  const int t = blockIdx.x;
  const int half = p.rotary_dim / 2;
  const bool vec = half % 8 == 0;
  const __nv_bfloat16* qs = p.q + (size_t)t * p.Hq * 192;
  __nv_bfloat16* qd = p.q_out + (size_t)t * p.Hq * 192;
  const __nv_bfloat16* ks = p.k_new + (size_t)t * p.Hkv * 192;
  const uint4* vs = reinterpret_cast<const uint4*>(p.v_new + (size_t)t * p.Hkv * 128);
  const PaSplit turn(half / 8), keep(24 - 2 * (half / 8));
  const uint32_t qt = p.Hq * turn.each, qk = p.q == p.q_out ? 0 : p.Hq * keep.each;
  const uint32_t kt = p.Hkv * turn.each, kk = p.Hkv * keep.each, vn = p.Hkv * 16;
  if (!MIMO_ROW_OK(t, p.pb.total_q)) return;
  PaPair u[kPairs > 0 ? kPairs : 1], ku;
  uint4 c[kKept > 0 ? kKept : 1], kc, vc;
  if (vec) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qt) u[i] = pa_load(turn, half, qs, w);
    }
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qk) c[i] = *reinterpret_cast<const uint4*>(qs + pa_kept(keep, half, w));
    }
    if (threadIdx.x < kt) ku = pa_load(turn, half, ks, threadIdx.x);
    if (threadIdx.x < kk) kc = *reinterpret_cast<const uint4*>(ks + pa_kept(keep, half, threadIdx.x));
  }
  if (threadIdx.x < vn) vc = vs[threadIdx.x];
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
  __nv_bfloat16* kd = p.k_pages + (kv ? slot : 0) * p.Hkv * 192;
  uint4* vd = reinterpret_cast<uint4*>(p.v_pages + (kv ? slot : 0) * p.Hkv * 128);
  if (vec) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qt) pa_store(turn, half, qd, w, u[i], cs);
    }
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const uint32_t w = threadIdx.x + i * kPaThreads;
      if (w < qk) *reinterpret_cast<uint4*>(qd + pa_kept(keep, half, w)) = c[i];
    }
    if (kv && threadIdx.x < kt) pa_store(turn, half, kd, threadIdx.x, ku, cs);
    if (kv && threadIdx.x < kk) *reinterpret_cast<uint4*>(kd + pa_kept(keep, half, threadIdx.x)) = kc;
    // what a CTA of this size does not hold at once
    for (uint32_t w = threadIdx.x + kPairs * kPaThreads; w < qt; w += kPaThreads)
      pa_store(turn, half, qd, w, pa_load(turn, half, qs, w), cs);
    for (uint32_t w = threadIdx.x + kKept * kPaThreads; w < qk; w += kPaThreads)
      *reinterpret_cast<uint4*>(qd + pa_kept(keep, half, w)) = *reinterpret_cast<const uint4*>(qs + pa_kept(keep, half, w));
    if (kv) {
      for (uint32_t w = threadIdx.x + kPaThreads; w < kt; w += kPaThreads)
        pa_store(turn, half, kd, w, pa_load(turn, half, ks, w), cs);
      for (uint32_t w = threadIdx.x + kPaThreads; w < kk; w += kPaThreads)
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
    if (threadIdx.x < vn) vd[threadIdx.x] = vc;
    for (uint32_t w = threadIdx.x + kPaThreads; w < vn; w += kPaThreads) vd[w] = vs[w];
  }
}

}  // namespace mimo
