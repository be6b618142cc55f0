// Position rotation of q and k and the append of k and v to a paged cache.
//
// Per head row x of D elements (q and k; v is only stored):
//   y = x                                       without a norm weight
//   y = x (1 + w) / sqrt(mean x^2 + eps)        with one
//   (y_i, y_{i+R/2}) <- (y_i c_i - y_{i+R/2} s_i,  y_{i+R/2} c_i + y_i s_i),  i < R/2
// with c and s from row positions[t] of an fp32 table [rows, R] (cosines, then
// sines).  The table is an input because an angle position * frequency needs
// more than fp32 at far positions; it is built once.
// int8 caches hold one fp32 scale per token and head, max|y| / 127, and codes
// rint(y / scale) (half to even), taken from the fp32 values: the row is
// rounded once, not first to bf16.
//
// Work split: D / 16 lanes hold one head row, each two 8-element chunks that
// rotate with one another (dimensions R and up pair off and pass through), so
// a rotation needs no exchange between lanes and every access is 16 bytes
// wide; a row's norm and absmax are xor-shuffles inside its lanes.  A warp
// keeps its token's cosines and sines in registers and walks over the token's
// head rows, APPEND_UNROLL row groups in flight at a time.
//
// Bound by memory: 8192 tokens x (32 + 8 + 8) x 128 in bf16, 223 MB read and
// written, take 36.6 us (6.08 TB/s, 0.93 of a copy's rate; graph replays); one
// token takes 1.9 us, 256 with norms into int8 caches 5.0.  Behind that stands
// the start of a warp (position and slot, then the table's row, then the head
// rows): 5035 tokens with both norms take 31 us (0.74), 1.7 waves of warps.
// Measured slower there: a token split over more
// warps (36, 40 and 51 us with 64, 128 and 256 warps per SM asked for), the norm
// weights kept in registers (44 us: 130 registers leave 12 warps per SM).
#pragma once

#include "attn_row.cuh"

namespace convrot {

struct AppendArgs {
  const uint16_t *q, *k, *v;            // bf16 [tokens, heads, D], row strides below
  int64_t q_stride, k_stride, v_stride; // elements
  const float* rope;                    // [rope_rows, rope_dim]
  const int32_t* positions;             // [tokens]
  const int64_t* slots;                 // [tokens], page * page_size + offset; negative: no write
  const float *q_norm, *k_norm;         // [D] or NULL
  uint16_t *q_out, *k_out;              // k_out may be NULL
  int64_t q_out_stride, k_out_stride;
  void *k_cache, *v_cache;              // [pages, kv_heads, page_size, D]
  float *k_scale, *v_scale;             // [pages, kv_heads, page_size] (int8 caches)
  int64_t slot_end;                     // pages * page_size
  int tokens, q_heads, kv_heads, rope_rows, rope_dim, page_size;
  int parts;                            // warps that share a token's head rows
  float eps;
};

constexpr int APPEND_WARPS = 4;
constexpr int APPEND_UNROLL = 4;

__device__ __forceinline__ void bf16x8_to_f32(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float* f) {
  return make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]),
                    bf16x2(f[6], f[7]));
}

// Eight codes rint(f * inv) in [-127, 127]; a NaN becomes 0 (its row's scale is NaN).
__device__ __forceinline__ uint2 f32_to_codes(const float* f, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = max(-127, min(127, __float2int_rn(f[4 * i + j] * inv)));
      w[i] |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * j);
    }
  }
  return make_uint2(w[0], w[1]);
}

template <int D, bool I8>
__global__ void __launch_bounds__(32 * APPEND_WARPS) append_kernel(const AppendArgs a) {
  constexpr int LANES = D / 16;        // lanes of one head row
  constexpr int ROWS = 32 / LANES;     // head rows of one warp step
  pdl_launch_dependents();
  const int warp = blockIdx.x * APPEND_WARPS + (threadIdx.x >> 5);
  const int t = warp / a.parts, part = warp - t * a.parts;
  if (t >= a.tokens) return;
  const int lane = threadIdx.x & 31, u = lane % LANES, sub = lane / LANES;
  const int half = a.rope_dim / 2;
  const bool turns = 8 * u < half;
  // first elements of this lane's two chunks
  const int e0 = turns ? 8 * u : 16 * u;
  const int e1 = turns ? e0 + half : e0 + 8;

  pdl_wait();
  const int pos = a.positions[t];
  const int64_t slot = a.slots[t];
  if (pos < 0 || pos >= a.rope_rows || slot >= a.slot_end) {
    if (lane == 0) report_error(ERR_BAD_ARGUMENT);
    return;
  }
  float c[8] = {}, s[8] = {};
  if (turns) {
    const float* r = a.rope + static_cast<int64_t>(pos) * a.rope_dim + 8 * u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<float4*>(c + 4 * i) = *reinterpret_cast<const float4*>(r + 4 * i);
      *reinterpret_cast<float4*>(s + 4 * i) = *reinterpret_cast<const float4*>(r + half + 4 * i);
    }
  }
  const int rows = a.q_heads + 2 * a.kv_heads;
  const int groups = (rows + ROWS - 1) / ROWS;
  const int g0 = static_cast<int>(static_cast<int64_t>(groups) * part / a.parts);
  const int g1 = static_cast<int>(static_cast<int64_t>(groups) * (part + 1) / a.parts);
  const int64_t page = slot >= 0 ? slot / a.page_size : 0;
  const int64_t in_page = slot >= 0 ? slot - page * a.page_size : 0;

  for (int g = g0; g < g1; g += APPEND_UNROLL) {
    uint4 in[APPEND_UNROLL][2];
#pragma unroll
    for (int j = 0; j < APPEND_UNROLL; ++j) {
      const int row = (g + j) * ROWS + sub;
      in[j][0] = in[j][1] = make_uint4(0, 0, 0, 0);
      if (g + j < g1 && row < rows) {
        const uint16_t* p;
        if (row < a.q_heads)
          p = a.q + t * a.q_stride + static_cast<int64_t>(row) * D;
        else if (row < a.q_heads + a.kv_heads)
          p = a.k + t * a.k_stride + static_cast<int64_t>(row - a.q_heads) * D;
        else
          p = a.v + t * a.v_stride + static_cast<int64_t>(row - a.q_heads - a.kv_heads) * D;
        in[j][0] = *reinterpret_cast<const uint4*>(p + e0);
        in[j][1] = *reinterpret_cast<const uint4*>(p + e1);
      }
    }
#pragma unroll
    for (int j = 0; j < APPEND_UNROLL; ++j) {
      if (g + j >= g1) break;  // the same for the whole warp
      const int row = (g + j) * ROWS + sub;
      const bool is_q = row < a.q_heads;
      const bool is_v = row >= a.q_heads + a.kv_heads;
      const bool live = row < rows;
      float x[8], y[8];
      bf16x8_to_f32(in[j][0], x);
      bf16x8_to_f32(in[j][1], y);
      const float* w = is_v ? nullptr : is_q ? a.q_norm : a.k_norm;
      if (a.q_norm || a.k_norm) {  // the same for the whole grid
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if (w) {
          const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = x[i] * r * (1.f + w[e0 + i]);
            y[i] = y[i] * r * (1.f + w[e1 + i]);
          }
        }
      }
      if (turns && !is_v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float lo = x[i], hi = y[i];
          x[i] = fmaf(lo, c[i], -hi * s[i]);
          y[i] = fmaf(hi, c[i], lo * s[i]);
        }
      }
      if (is_q) {
        uint16_t* o = a.q_out + t * a.q_out_stride + static_cast<int64_t>(row) * D;
        *reinterpret_cast<uint4*>(o + e0) = f32_to_bf16x8(x);
        *reinterpret_cast<uint4*>(o + e1) = f32_to_bf16x8(y);
      }
      const int h = row - a.q_heads - (is_v ? a.kv_heads : 0);
      if (live && !is_q && !is_v && a.k_out) {
        uint16_t* o = a.k_out + t * a.k_out_stride + static_cast<int64_t>(h) * D;
        *reinterpret_cast<uint4*>(o + e0) = f32_to_bf16x8(x);
        *reinterpret_cast<uint4*>(o + e1) = f32_to_bf16x8(y);
      }
      const bool store = live && !is_q && slot >= 0;
      const int64_t at = (page * a.kv_heads + h) * a.page_size + in_page;
      if (I8) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, max_nan(fabsf(x[i]), fabsf(y[i])));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        // 127 / m overflows for tiny rows: those are scaled up first (exactly)
        if (m < 1e-30f) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= 0x1p64f, y[i] *= 0x1p64f;
        }
        const float up = m < 1e-30f ? m * 0x1p64f : m;
        const float inv = up > 0.f ? 127.f / up : 0.f;
        if (store) {
          int8_t* o = static_cast<int8_t*>(is_v ? a.v_cache : a.k_cache) + at * D;
          *reinterpret_cast<uint2*>(o + e0) = f32_to_codes(x, inv);
          *reinterpret_cast<uint2*>(o + e1) = f32_to_codes(y, inv);
          if (u == 0) (is_v ? a.v_scale : a.k_scale)[at] = m / 127.f;
        }
      } else if (store) {
        uint16_t* o = static_cast<uint16_t*>(is_v ? a.v_cache : a.k_cache) + at * D;
        *reinterpret_cast<uint4*>(o + e0) = f32_to_bf16x8(x);
        *reinterpret_cast<uint4*>(o + e1) = f32_to_bf16x8(y);
      }
    }
  }
}

}  // namespace convrot
