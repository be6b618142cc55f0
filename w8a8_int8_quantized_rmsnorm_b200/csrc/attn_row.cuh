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

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// q: D bf16 of the row; k, v: the first key's and value's row of the head, the
// next ones k_stride and v_stride elements on; o: D bf16.  The whole warp calls.
// A lane reads its key's row 16 bytes at a time (the query's too, all lanes the
// same piece) and holds D / 32 neighbouring elements of the result.  A row that
// is NaN throughout ends at the key that made it so.
template <int D>
__device__ void attention_row(const uint16_t* q, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, int n, float scale_log2, uint16_t* o) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float acc[E] = {};
  float m = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    const uint4* kj = reinterpret_cast<const uint4*>(k + static_cast<int64_t>(min(j, n - 1)) * k_stride);
    float s = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const uint4 x = kj[c], y = reinterpret_cast<const uint4*>(q)[c];
      s = fmaf(bf16_lo(x.x), bf16_lo(y.x), fmaf(bf16_hi(x.x), bf16_hi(y.x), s));
      s = fmaf(bf16_lo(x.y), bf16_lo(y.y), fmaf(bf16_hi(x.y), bf16_hi(y.y), s));
      s = fmaf(bf16_lo(x.z), bf16_lo(y.z), fmaf(bf16_hi(x.z), bf16_hi(y.z), s));
      s = fmaf(bf16_lo(x.w), bf16_lo(y.w), fmaf(bf16_hi(x.w), bf16_hi(y.w), s));
    }
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
#pragma unroll 4
    for (int i = 0; i < 32; ++i) {
      const float pi = __shfl_sync(0xFFFFFFFFu, p, i);
      if (j0 + i >= n) break;  // the same for the whole warp
      const uint32_t* vi = reinterpret_cast<const uint32_t*>(v + static_cast<int64_t>(j0 + i) * v_stride + lane * E);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t w = vi[e / 2];
        acc[e] = fmaf(pi, bf16_lo(w), acc[e]);
        acc[e + 1] = fmaf(pi, bf16_hi(w), acc[e + 1]);
      }
    }
    bool lost = true;
#pragma unroll
    for (int e = 0; e < E; ++e) lost &= acc[e] != acc[e];
    if (__any_sync(0xFFFFFFFFu, p != p) || __all_sync(0xFFFFFFFFu, lost)) {
      l = NAN;
      break;
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    reinterpret_cast<uint32_t*>(o + lane * E)[e / 2] = n > 0 ? bf16x2(acc[e] / l, acc[e + 1] / l) : 0u;
}

}  // namespace convrot
