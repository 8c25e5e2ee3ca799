// Rotary position embedding of a chunk of new tokens' queries and keys, and
// the write of their keys and values into the pages of the cache.
//
// The paged counterpart of rope_append_kernel: the same rotation (rotate-half,
// angles formed in double precision) at position p = L - n + i of token i of
// the chunk; the key and value go to slot p % page_size of page
// block_table[b][p / page_size].
//
// One CTA per token: the angles of a position are formed once and used by its
// Hq + Hkv rows.
#pragma once

#include "paged_common.cuh"
#include "rope_append_kernel.cuh"

#undef MIMO_FILE_ID
#define MIMO_FILE_ID 12  // site numbers of the checked build

namespace mimo {

constexpr int kPaThreads = 192;

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

__global__ void __launch_bounds__(kPaThreads) paged_append_kernel(const PagedAppendParams p) {
  __shared__ float2 cs[kRaMaxHalf];
  const int t = blockIdx.x;
  const int b = paged_seq_of_row(p.pb, t);  // the whole CTA takes the same branches
  if (b < 0) return;
  const PagedSeq s = paged_seq(p.pb, b);
  if (!s.ok || t < s.b0 || t >= s.b0 + s.n) {
    if (!s.ok && threadIdx.x == 0) record_status(1 /* MIMO_ERR_INVALID_ARG */);
    return;
  }
  const int pos = s.len - s.n + (t - s.b0);
  const int half = p.rotary_dim / 2;
  if (threadIdx.x < half) {
    const double a = (double)pos * p.inv_freq[threadIdx.x];
    const double twopi = 6.283185307179586476925286766559;
    const float r = (float)(a - twopi * rint(a / twopi));  // in [-pi, pi]
    float sn, c;
    sincosf(r, &sn, &c);
    cs[threadIdx.x] = make_float2(c, sn);
  }
  __syncthreads();
  const int page = paged_page(p.pb, b, pos / p.pb.page_size);
  const long long slot = (long long)page * p.pb.page_size + pos % p.pb.page_size;
  const bool kv = page >= 0 && MIMO_ROW_OK(slot, (long long)p.pb.num_pages * p.pb.page_size);
  const __nv_bfloat16* qs = p.q + (size_t)t * p.Hq * 192;
  __nv_bfloat16* qd = p.q_out + (size_t)t * p.Hq * 192;
  const __nv_bfloat16* ks = p.k_new + (size_t)t * p.Hkv * 192;
  __nv_bfloat16* kd = p.k_pages + (kv ? slot : 0) * p.Hkv * 192;
  const int rows = p.Hq + (kv ? p.Hkv : 0);  // rows to rotate: the query heads, then the keys
  if (!MIMO_ROW_OK(t, p.pb.total_q)) return;
  if (half % 8 == 0) {
    const int tasks = half / 8, tail = (192 - 2 * half) / 8, each = tasks + tail;
    for (int w = threadIdx.x; w < rows * each; w += kPaThreads) {
      const int r = w / each, j = w % each;
      const __nv_bfloat16* src = r < p.Hq ? qs + r * 192 : ks + (r - p.Hq) * 192;
      __nv_bfloat16* dst = r < p.Hq ? qd + r * 192 : kd + (r - p.Hq) * 192;
      if (j < tasks) {
        rope_row8(src, dst, half, j, cs);
      } else {
        const int d = 2 * half + (j - tasks) * 8;
        *reinterpret_cast<uint4*>(dst + d) = *reinterpret_cast<const uint4*>(src + d);
      }
    }
  } else {
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
