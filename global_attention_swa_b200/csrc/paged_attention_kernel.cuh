// Attention of a chunk of new tokens over a paged cache.
//
// Row (token i of the chunk, query head h) at position p = L - n + i sees the
// keys j with 0 <= p - j and, in a window, p - j <= window - 1:
//   m = max(sigma_h, max_j S_j),  Z = exp(sigma_h - m) + sum_j exp(S_j - m),
//   out = v_scale * sum_j exp(S_j - m) v_j / Z,  lse = m + ln Z.
//
// One warp per row: a lane holds 6 of the 192 query dimensions and 4 of the
// 128 value columns, and the keys pass one at a time through an online softmax.
#pragma once

#include "paged_common.cuh"

#undef MIMO_FILE_ID
#define MIMO_FILE_ID 11  // site numbers of the checked build

namespace mimo {

struct PagedAttnParams {
  PagedBatch pb;
  const __nv_bfloat16* q;  // [total_q, Hq, 192]
  const __nv_bfloat16* k;  // [num_pages, page_size, Hkv, 192]
  const __nv_bfloat16* v;  // [num_pages, page_size, Hkv, 128]
  const float* sinks;      // [Hq] or null
  void* out;               // [total_q, Hq, 128]
  float* lse;              // [Hq, total_q] or null
  int Hq, Hkv, G;
  int window;
  float scale_log2, v_scale;
  int out_f32;
};

__global__ void __launch_bounds__(256) paged_attention_kernel(const PagedAttnParams p) {
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)p.pb.total_q * p.Hq;
  for (long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); w < rows; w += (long long)gridDim.x * 8) {
    const int t = (int)(w / p.Hq), h = (int)(w % p.Hq), g = h / p.G;
    const int b = paged_seq_of_row(p.pb, t);
    if (b < 0) continue;
    const PagedSeq s = paged_seq(p.pb, b);
    if (!s.ok || t < s.b0 || t >= s.b0 + s.n) {
      if (!s.ok) record_status(1 /* MIMO_ERR_INVALID_ARG */);
      continue;
    }
    const int pos = s.len - s.n + (t - s.b0);
    const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    float2 q[3];
#pragma unroll
    for (int c = 0; c < 3; ++c)
      q[c] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p.q + w * 192 + 64 * c + 2 * lane));
    float m = p.sinks ? p.sinks[h] * 1.4426950408889634f : -INFINITY;
    float l = p.sinks ? 1.f : 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    int page = -1;
    for (int j = lo; j <= pos; ++j) {
      const int slot = j % p.pb.page_size;
      if (j == lo || slot == 0) page = paged_page(p.pb, b, j / p.pb.page_size);
      float x = 0.f;  // a key without a page reads as zeros
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const long long row = ((long long)page * p.pb.page_size + slot) * p.Hkv + g;
      if (page >= 0 && MIMO_ROW_OK(row, (long long)p.pb.num_pages * p.pb.page_size * p.Hkv)) {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const float2 k = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p.k + row * 192 + 64 * c + 2 * lane));
          x += q[c].x * k.x + q[c].y * k.y;
        }
        const uint2 u = *reinterpret_cast<const uint2*>(p.v + row * 128 + 4 * lane);
        v = make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x *= p.scale_log2;
      const float mn = fmaxf(m, x);
      const float a = (m == -INFINITY) ? 0.f : ex2(m - mn), e = ex2(x - mn);
      m = mn;
      l = l * a + e;
      o = make_float4(o.x * a + e * v.x, o.y * a + e * v.y, o.z * a + e * v.z, o.w * a + e * v.w);
    }
    if (!MIMO_ROW_OK(w, rows)) continue;
    const float f = l > 0.f ? p.v_scale / l : 0.f;
    if (p.out_f32)
      reinterpret_cast<float4*>(p.out)[w * 32 + lane] = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    else
      reinterpret_cast<uint2*>(p.out)[w * 32 + lane] = make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
    if (p.lse && lane == 0)
      p.lse[(size_t)h * p.pb.total_q + t] = l > 0.f ? m * 0.6931471805599453f + logf(l) : -INFINITY;
  }
}

}  // namespace mimo
