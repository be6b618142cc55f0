// Attention of one new token per sequence over a paged cache.
#pragma once

#include "attn_row.cuh"

namespace convrot {

struct DecodeArgs {
  const uint16_t* q;              // bf16 [seqs, q_heads, D]
  int64_t q_stride, o_stride;     // elements per sequence
  uint16_t* o;
  const void *k_cache, *v_cache;  // [pages, kv_heads, page_size, D], bf16 or int8
  const float *k_scale, *v_scale; // [pages, kv_heads, page_size] (int8)
  const int32_t* table;           // [seqs, table_cols]
  int64_t table_stride;
  const int32_t* lens;            // [seqs]
  int seqs, q_heads, kv_heads, pages, page_size, table_cols;
  float scale_log2;
};

// One warp per (sequence, head); a lane holds D / 32 dimensions.
template <int D, bool I8>
__global__ void __launch_bounds__(128) decode_rows_kernel(const DecodeArgs a) {
  constexpr int E = D / 32;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int b = static_cast<int>(w / a.q_heads), h = static_cast<int>(w - static_cast<int64_t>(b) * a.q_heads);
  if (b >= a.seqs) return;
  const int lane = threadIdx.x & 31, kh = h / (a.q_heads / a.kv_heads);
  int n = a.lens[b];
  if (n < 0 || n > static_cast<int64_t>(a.table_cols) * a.page_size) {
    if (lane == 0) report_error(ERR_BAD_ARGUMENT);
    n = 0;
  }
  float qe[E], acc[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) qe[e] = bf16_at(a.q + b * a.q_stride + static_cast<int64_t>(h) * D, e * 32 + lane);
  for (int j = 0; j < n; ++j) {
    const int page = a.table[b * a.table_stride + j / a.page_size];
    if (page < 0 || page >= a.pages) {
      if (lane == 0) report_error(ERR_BAD_ARGUMENT);
      continue;
    }
    const int64_t at = (static_cast<int64_t>(page) * a.kv_heads + kh) * a.page_size + j % a.page_size;
    float s = 0.f, ve[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t i = at * D + e * 32 + lane;
      float ke;
      if (I8) {
        ke = static_cast<const int8_t*>(a.k_cache)[i] * a.k_scale[at];
        ve[e] = static_cast<const int8_t*>(a.v_cache)[i] * a.v_scale[at];
      } else {
        ke = bf16_at(static_cast<const uint16_t*>(a.k_cache) + i, 0);
        ve[e] = bf16_at(static_cast<const uint16_t*>(a.v_cache) + i, 0);
      }
      s = fmaf(qe[e], ke, s);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    s *= a.scale_log2;
    const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top;
    const float old = exp2f(m - base), p = exp2f(s - base);
    m = top;
    l = l * old + p;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], old, p * ve[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.o[b * a.o_stride + static_cast<int64_t>(h) * D + e * 32 + lane] =
        __bfloat16_as_ushort(__float2bfloat16(n > 0 ? acc[e] / l : 0.f));
}

}  // namespace convrot
