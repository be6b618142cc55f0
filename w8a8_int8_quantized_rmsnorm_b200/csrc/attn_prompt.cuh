// Attention over whole prompts, packed one after another.
#pragma once

#include "attn_row.cuh"

namespace convrot {

struct PromptArgs {
  const uint16_t *q, *k, *v;                       // bf16 [tokens, heads, D]
  int64_t q_stride, k_stride, v_stride, o_stride;  // elements per token
  uint16_t* o;
  const int32_t *cu_q, *cu_k;                      // [seqs + 1]
  int tokens, kv_tokens, seqs, q_heads, kv_heads;
  float scale_log2;                                // scale * log2(e)
  int causal;
};

// One warp per (token, head).
template <int D>
__global__ void __launch_bounds__(128) prompt_rows_kernel(const PromptArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / a.q_heads), h = static_cast<int>(w - static_cast<int64_t>(t) * a.q_heads);
  if (t >= a.tokens || t >= a.cu_q[a.seqs] || t < a.cu_q[0]) return;
  int lo = 0, hi = a.seqs;  // cu_q[lo] <= t < cu_q[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu_q[mid] <= t) lo = mid; else hi = mid;
  }
  const int q0 = a.cu_q[lo], lq = a.cu_q[lo + 1] - q0, k0 = a.cu_k[lo], lk = a.cu_k[lo + 1] - k0;
  if (q0 < 0 || lq > a.tokens - q0 || k0 < 0 || lk < 0 || lk > a.kv_tokens - k0) {
    if ((threadIdx.x & 31) == 0) report_error(ERR_BAD_ARGUMENT);
    return;
  }
  const int n = a.causal ? max(0, min(lk, t - q0 + 1 + lk - lq)) : lk;
  const int kh = h / (a.q_heads / a.kv_heads);
  attention_row<D>(a.q + t * a.q_stride + static_cast<int64_t>(h) * D,
                   a.k + k0 * a.k_stride + static_cast<int64_t>(kh) * D, a.k_stride,
                   a.v + k0 * a.v_stride + static_cast<int64_t>(kh) * D, a.v_stride, n, a.scale_log2,
                   a.o + t * a.o_stride + static_cast<int64_t>(h) * D);
}

}  // namespace convrot
