// Attention of one query row, by one warp, over exactly its visible keys:
//   o = sum_j softmax_j(scale q.k_j) v_j,  j = 0 .. n-1;  0 when n = 0.
// Keys are taken 32 at a time, one per lane; the running maximum m, the sum l
// of exp2(s - m) and the output (D / 32 elements per lane) are fp32.
//
// Nothing outside the visible keys enters the arithmetic, so an infinity or a
// NaN in a masked place cannot reach the result (a matrix product would
// multiply it by a probability of zero and give NaN).
#pragma once

#include "ptx.cuh"

namespace convrot {

constexpr float LOG2E = 1.4426950408889634f;

// Maximum that a NaN survives.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two bf16, lo in the low half, rounded to nearest even.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float bf16_at(const uint16_t* p, int i) {
  return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}

// q: D bf16 of the row; k, v: the first key's and value's row of the head, the
// next ones k_stride and v_stride elements on; o: D bf16.  The whole warp calls.
template <int D>
__device__ void attention_row(const uint16_t* q, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, int n, float scale_log2, uint16_t* o) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float qe[E], acc[E] = {};
#pragma unroll
  for (int e = 0; e < E; ++e) qe[e] = bf16_at(q, e * 32 + lane);
  float m = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    const uint16_t* kj = k + static_cast<int64_t>(min(j, n - 1)) * k_stride;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      for (int i = 0; i < 32; ++i)
        s = fmaf(__shfl_sync(0xFFFFFFFFu, qe[e], i), bf16_at(kj, e * 32 + i), s);
    s = j < n ? s * scale_log2 : -INFINITY;
    float top = s;
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    top = fmaxf(top, m);
    // no finite score yet (all -inf): exp2(s - 0) = 0 keeps the sums at zero
    const float base = top == -INFINITY ? 0.f : top;
    const float old = exp2f(m - base);
    const float p = j < n ? exp2f(s - base) : 0.f;
    m = top;
    l = l * old + p;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= old;
    for (int i = 0; i < min(32, n - j0); ++i) {
      const float pi = __shfl_sync(0xFFFFFFFFu, p, i);
      const uint16_t* vi = v + static_cast<int64_t>(j0 + i) * v_stride;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(pi, bf16_at(vi, e * 32 + lane), acc[e]);
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const __nv_bfloat16 r = __float2bfloat16(n > 0 ? acc[e] / l : 0.f);
    o[e * 32 + lane] = __bfloat16_as_ushort(r);
  }
}

}  // namespace convrot
