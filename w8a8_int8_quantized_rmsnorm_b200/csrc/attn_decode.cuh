// Attention of one new token per sequence over a paged cache: a stream of
// every key and value, once, at memory speed.
//
// Work split.  The unit of work is a block of 64 keys of one (sequence,
// key/value head); the heads of its group (up to 8 or 16 at a time) share it.
// All blocks of the call are laid out in one line, sequence by sequence and
// head by head, and every CTA takes an equal stretch of the line, so sequences
// of any mix of lengths keep every SM streaming to the end.  A stretch covers
// the tail of one (sequence, head), any number of whole ones, and the front of
// another.  Whole ones are finished in place; a part leaves its (m, l, O) in
// the workspace, and the part that comes last, found by a counter, joins all
// of them in the order of the keys, so the result does not depend on timing.
//
// Inside a CTA one warp fetches (the block table's entries one block ahead,
// then one TMA box per page piece, into a ring of blocks) and four warps
// compute, each 16 keys of a block, on warp-level matrix instructions with the
// keys as rows and the heads as columns: S^T = K Q^T and O^T += V^T P^T, so a
// group of four or eight heads fills the 8-column operand and every score
// stays with the lane that made it.  16 keys x 8 heads are 2 * D / 16 products
// against 4 D (bf16) bytes a key: the tensor pipe idles, memory bounds.
//
// Each warp keeps a reference maximum per head, raised (with O and l) only
// when a score lies more than 2^8 above it, and fp32 sums; probabilities are
// rounded to bf16 for the product with V.  int8 codes become bf16 exactly in
// registers; a key's scale multiplies its score, a value's its probability.
//
// Rows past a sequence's end are never used: their scores are replaced, their
// values' registers cleared, pages behind the last one not fetched.
#pragma once

#include "attn_row.cuh"

namespace convrot {

struct DecodeArgs {
  const uint16_t* q;              // bf16 [seqs, q_heads, D]
  int64_t q_stride, o_stride;     // elements per sequence
  uint16_t* o;
  const float *k_scale, *v_scale; // [pages, kv_heads, page_size] (int8)
  const int32_t* table;           // [seqs, table_cols]
  int64_t table_stride;
  const int32_t* lens;            // [seqs]
  int seqs, q_heads, kv_heads, pages, page_size, table_cols;
  int chunk_heads;                // query heads of one unit (<= NQ)
  int chunks;                     // units side by side for one group
  int box_rows;                   // keys per TMA box: 16, 32 or 64
  int stages;
  float scale_log2;
  unsigned* counters;             // [grid], zero between calls
  float* parts;                   // [grid][2][decode_part_floats(chunk_heads, D)]
};

constexpr int DECODE_KEYS = 64;
constexpr int DECODE_THREADS = 160;
constexpr unsigned SITE_DECODE = 20;
constexpr int DECODE_MAX_STAGES = 8;

// A part: O [heads][D], then (m, l) [heads], to a multiple of 16 bytes.
__host__ __device__ constexpr int decode_part_floats(int heads, int D) { return heads * D + (2 * heads + 3) / 4 * 4; }

// What a ring slot holds besides keys and values.
struct DecodeBlock {
  int seq, unit;        // unit: (kv head, head chunk); seq < 0: no more blocks
  int left;             // keys of the sequence from the block's first one on
  unsigned slices;      // 16-key slices that are there
  int first, last;      // begins / ends this CTA's stretch of the (seq, unit)
  int owner, n_parts;   // CTA of the (seq, unit)'s first block; parts (1: whole)
};

template <int D, bool I8, int NQ>
struct DecodeSmem {
  static constexpr int ESZ = I8 ? 1 : 2;
  // CTAs per SM: two keep enough bf16 rows in flight (64 contexts of 1 .. 8192
  // keys: 0.98 of HBM); int8 rows need more warps, for the conversions
  static constexpr int CTAS = I8 && NQ == 8 ? 3 : 2;
  static constexpr int TILE = DECODE_KEYS * D * ESZ;
  static constexpr int SLOT = 2 * TILE;                            // K, V
  static constexpr int SIDE = NQ * D * 2 + 2 * DECODE_KEYS * 4;    // Q rows, scales
  static constexpr int PAD = D + 4;                                // floats per joined row
  static int join_bytes(int heads) { return 4 * heads * PAD * 4 + 2 * 4 * NQ * 8 + 2 * NQ * 8; }
  static int total(int stages, int heads) {
    return 1024 + stages * (SLOT + SIDE + 32) + join_bytes(heads) + 8 * (2 * stages + 1) + 32;
  }
};

__device__ __forceinline__ void ldsm_x4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t r) {
  uint32_t o;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o) : "r"(r));
  return o;
}
// d += a (16 x 16, rows) * b (16 x 8, columns), bf16 in, fp32 out
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two int8 codes, bytes 0 and 2 of x, as bf16, exactly:
// (128 + low 7 bits) - (128 or, with the sign bit, 256).
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t x) {
  const uint32_t v = (x & 0x007F007Fu) | 0x43004300u, w = (x & 0x00800080u) | 0x43004300u;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(w));
  return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Length of sequence b; a length outside [0, table_cols * page_size] counts as 0.
__device__ __forceinline__ int decode_length(const DecodeArgs& a, int b) {
  const int n = a.lens[b];
  if (n < 0 || n > static_cast<int64_t>(a.table_cols) * a.page_size) {
    report_error(ERR_BAD_ARGUMENT);
    return 0;
  }
  return n;
}
// A sequence without keys still has one (empty) block: its result is written.
__device__ __forceinline__ int decode_blocks(int len) { return max(1, (len + DECODE_KEYS - 1) / DECODE_KEYS); }

template <int D, bool I8, int NQ>
__global__ void __launch_bounds__(DECODE_THREADS, DecodeSmem<D, I8, NQ>::CTAS)
decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const DecodeArgs a) {
  using SM = DecodeSmem<D, I8, NQ>;
  constexpr int ROWB = D * SM::ESZ >= 128 ? 128 : 64;  // bytes of a swizzled line
  constexpr int HALVES = D * SM::ESZ / ROWB;
  constexpr int NT = NQ / 8;                           // 8-head column tiles
  constexpr int KS = D / 16;                           // 16-element steps
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  const int S = a.stages, heads = a.chunk_heads;
  uint8_t* side = smem + S * SM::SLOT;                  // per slot: Q rows, k scales, v scales
  DecodeBlock* meta = reinterpret_cast<DecodeBlock*>(side + S * SM::SIDE);
  float* join = reinterpret_cast<float*>(meta + S);     // [4][heads][PAD]
  float* stat = join + 4 * heads * SM::PAD;             // [2][4][NQ][2]: (m, l) by parity, warp, head
  float* stat_all = stat + 2 * 4 * NQ * 2;              // [2][NQ][2]: joined (m, l)
  uint64_t* full = reinterpret_cast<uint64_t*>(stat_all + 2 * NQ * 2);
  uint64_t *empty = full + S, *meet = empty + S;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(meet + 1);
  volatile int* is_last = abort_flag + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    mbar_init(meet, 4);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  pdl_wait();

  const int units = a.kv_heads * a.chunks;
  if (warp == 4) {
    // -------------------------------------------------------- fetch
    // this CTA's stretch [at, end) of the line of blocks
    int64_t total = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
      int n = b0 + lane < a.seqs ? decode_blocks(decode_length(a, b0 + lane)) : 0;
      total += __reduce_add_sync(0xFFFFFFFFu, n);
    }
    total *= units;
    const int64_t per = (total + gridDim.x - 1) / gridDim.x, begin = per * blockIdx.x;
    int64_t at = begin;
    const int64_t end = min(total, at + per);
    int seq = 0, len = 0, nb = 1, unit = 0, j = 0;
    int64_t start = 0;                       // line index of the sequence's first block
    if (at < end) {
      for (int b0 = 0;; b0 += 32) {
        const int ln = b0 + lane < a.seqs ? decode_length(a, b0 + lane) : 0;
        const int n = b0 + lane < a.seqs ? decode_blocks(ln) : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
          if (lane >= o) sum += up;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, start + static_cast<int64_t>(sum) * units > at);
        if (hit) {
          const int l = __ffs(hit) - 1;
          seq = b0 + l;
          len = __shfl_sync(0xFFFFFFFFu, ln, l);
          nb = decode_blocks(len);
          start += static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, sum, l) - nb) * units;
          break;
        }
        start += static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, sum, 31)) * units;
      }
      unit = static_cast<int>((at - start) / nb);
      j = static_cast<int>((at - start) - static_cast<int64_t>(unit) * nb);
    }
    const int boxes = DECODE_KEYS / a.box_rows;
    const unsigned page_size = a.page_size;
    // page of this lane's box of a block; -1: not there
    auto entry = [&](int b, int blk, int n) -> int {
      const unsigned key = static_cast<unsigned>(blk) * DECODE_KEYS + lane * a.box_rows;
      return lane < boxes && key < static_cast<unsigned>(n) ? a.table[b * a.table_stride + key / page_size] : -1;
    };
    bool ok = true;
    uint32_t it = 0, s = 0, phase = 1;  // slot and the parity its last emptying has
    int page = at < end ? entry(seq, j, len) : -1;
    const int group = a.q_heads / a.kv_heads;
    int kvh = unit / a.chunks, chunk = unit - kvh * a.chunks;
    int next_len = seq + 1 < a.seqs ? decode_length(a, seq + 1) : 0;
    while (at < end && ok) {
      // where the line goes on, and that block's pages
      int seq2 = seq, len2 = len, nb2 = nb, unit2 = unit, j2 = j + 1;
      int64_t start2 = start;
      if (j2 == nb) {
        j2 = 0;
        if (++unit2 == units) {
          unit2 = 0;
          ++seq2;
          start2 += static_cast<int64_t>(nb) * units;
          len2 = next_len;
          nb2 = decode_blocks(len2);
        }
      }
      const bool more = at + 1 < end;
      const int page2 = more ? entry(seq2, j2, len2) : -1;
      if (seq2 != seq) next_len = seq2 + 1 < a.seqs ? decode_length(a, seq2 + 1) : 0;

      ok = mbar_wait_spin(&empty[s], phase, abort_flag, SITE_DECODE);
      if (!ok) break;
      const int qh = min(heads, group - chunk * heads);
      const unsigned key = static_cast<unsigned>(j) * DECODE_KEYS + lane * a.box_rows;  // of this lane's box
      const bool wanted = lane < boxes && key < static_cast<unsigned>(len);
      const bool there = wanted && page >= 0 && page < a.pages;
      if (wanted && !there) report_error(ERR_BAD_ARGUMENT);
      const unsigned mask = __ballot_sync(0xFFFFFFFFu, there);
      const bool first = at == begin || j == 0;
      const bool last = j + 1 == nb || !more;
      if (lane == 0) {
        DecodeBlock m;
        m.seq = seq;
        m.unit = unit;
        m.left = len - j * DECODE_KEYS;
        m.slices = 0;
        for (int x = 0; x < 4; ++x) m.slices |= ((mask >> (16 * x / a.box_rows)) & 1u) << x;
        m.first = first;
        m.last = last;
        m.owner = blockIdx.x;
        m.n_parts = 1;
        const int64_t item = start + static_cast<int64_t>(unit) * nb;
        if (last && (item < begin || item + nb > end)) {  // twice per CTA at most: its two ends
          m.owner = static_cast<int>(item / per);
          m.n_parts = static_cast<int>((item + nb - 1) / per) - m.owner + 1;
        }
        meta[s] = m;
        const uint32_t bytes = __popc(mask) * a.box_rows * (2 * D * SM::ESZ + (I8 ? 8 : 0)) + (first ? qh * D * 2 : 0);
        mbar_arrive_expect_tx(&full[s], bytes);
        if (first)
          bulk_load_1d(side + s * SM::SIDE,
                       a.q + seq * a.q_stride + (static_cast<int64_t>(kvh) * group + chunk * heads) * D, qh * D * 2,
                       &full[s]);
      }
      __syncwarp();
      if (there) {
        const int64_t row = (static_cast<int64_t>(page) * a.kv_heads + kvh) * page_size + key % page_size;
        uint8_t* dst = smem + s * SM::SLOT + lane * a.box_rows * D * SM::ESZ;
        tma_load_3d(dst, &tm_k, &full[s], 0, static_cast<int>(row), 0);
        tma_load_3d(dst + SM::TILE, &tm_v, &full[s], 0, static_cast<int>(row), 0);
        if (I8) {
          float* sc = reinterpret_cast<float*>(side + s * SM::SIDE + NQ * D * 2) + lane * a.box_rows;
          bulk_load_1d(sc, a.k_scale + row, a.box_rows * 4, &full[s]);
          bulk_load_1d(sc + DECODE_KEYS, a.v_scale + row, a.box_rows * 4, &full[s]);
        }
      }
      ++it;
      if (++s == static_cast<uint32_t>(S)) s = 0, phase ^= 1u;
      ++at;
      if (unit2 != unit) kvh = unit2 / a.chunks, chunk = unit2 - kvh * a.chunks;
      seq = seq2;
      len = len2;
      nb = nb2;
      unit = unit2;
      j = j2;
      start = start2;
      page = page2;
    }
    ok = ok && mbar_wait_spin(&empty[s], phase, abort_flag, SITE_DECODE);
    if (ok && lane == 0) {
      meta[s].seq = -1;
      mbar_arrive(&full[s]);
    }
    // No copy may still be landing in shared memory when the CTA exits.  The
    // slot of the end mark has been taken back already: its copies are in.
    int never = 0;
    const uint32_t back = ok ? S - 1 : S;
    for (uint32_t x = it > back ? it - back : 0u; x < it; ++x)
      mbar_wait(&full[x % S], (x / S) & 1u, &never, SITE_DRAIN);
  } else {
    // -------------------------------------------------------- compute
    const int g = lane >> 2, t = lane & 3;
    uint32_t qf[NT][KS][2];
    float acc[NT][KS][4];
    float m[NT][2], l[NT][2];
    uint32_t met = 0, parity = 0;
    // bounded rendezvous of the four compute warps
    auto rendezvous = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      return mbar_wait_spin(meet, met++ & 1u, abort_flag, SITE_DECODE + 1);
    };
    // this lane's ldmatrix rows inside a 16-key slice
    const int box = 16 * warp / a.box_rows, row0 = 16 * warp - box * a.box_rows;
    const uint32_t slice = box * a.box_rows * D * SM::ESZ + row0 * ROWB;
    const uint32_t half_step = a.box_rows * ROWB;
    auto line = [&](uint32_t base, int row, int c16) -> uint32_t {  // 16-byte piece c16 of a key's row
      const int h = c16 * 16 / ROWB, c = c16 % (ROWB / 16);
      const int sw = ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
      return base + h * half_step + row * ROWB + ((c ^ sw) << 4);
    };
    uint32_t next = 0, phase = 0;
    for (;;) {
      const uint32_t s = next;
      if (!mbar_wait_spin(&full[s], phase, abort_flag, SITE_DECODE + 2)) break;
      if (++next == static_cast<uint32_t>(S)) next = 0, phase ^= 1u;
      const DecodeBlock b = meta[s];
      if (b.seq < 0) break;
      if (b.first) {
        const uint8_t* qs = side + s * SM::SIDE;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint8_t* p = qs + ((n * 8 + g) * D + k * 16) * 2;
            if (I8) {  // elements 4t .. 4t+3 of the step: see the keys' bytes below
              const uint2 v = *reinterpret_cast<const uint2*>(p + 8 * t);
              qf[n][k][0] = __byte_perm(v.x, v.y, 0x5410);
              qf[n][k][1] = __byte_perm(v.x, v.y, 0x7632);
            } else {
              qf[n][k][0] = *reinterpret_cast<const uint32_t*>(p + 4 * t);
              qf[n][k][1] = *reinterpret_cast<const uint32_t*>(p + 16 + 4 * t);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][k][e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) m[n][e] = -INFINITY, l[n][e] = 0.f;
        }
      }
      const int left = b.left - 16 * warp;  // keys of this slice that exist
      if (left > 0 && ((b.slices >> warp) & 1u)) {
        const uint32_t kb = smem_addr(smem + s * SM::SLOT) + slice, vb = kb + SM::TILE;
        float sc[NT][4], sd[NT][4];  // two chains of products
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] = sd[n][e] = 0.f;
        if (I8) {
          // one ldmatrix covers 32 elements: a lane gets elements 4t .. 4t+3 of
          // row g (and g + 8) of each 16; the even ones stand as the step's
          // columns 2t, 2t+1, the odd ones as 2t+8, 2t+9, in K and Q alike
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t r[4];
            ldsm_x4(line(kb, lane & 15, k + (lane >> 4)), r);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a0 = codes_to_bf16(r[2 * h]), a2 = codes_to_bf16(r[2 * h] >> 8);
              const uint32_t a1 = codes_to_bf16(r[2 * h + 1]), a3 = codes_to_bf16(r[2 * h + 1] >> 8);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_16x8x16(h ? sd[n] : sc[n], a0, a1, a2, a3, qf[n][k + h][0], qf[n][k + h][1]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t r[4];
            ldsm_x4(line(kb, lane & 15, 2 * k + (lane >> 4)), r);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16x8x16(k & 1 ? sd[n] : sc[n], r[0], r[1], r[2], r[3], qf[n][k][0], qf[n][k][1]);
          }
        }
        // rows g and g + 8: keys; columns 2t and 2t + 1: heads
        float ks[2] = {a.scale_log2, a.scale_log2}, vs[2] = {1.f, 1.f};
        if (I8) {
          const float* scales = reinterpret_cast<const float*>(side + s * SM::SIDE + NQ * D * 2) + 16 * warp + g;
          ks[0] *= scales[0];
          ks[1] *= scales[8];
          vs[0] = scales[DECODE_KEYS];
          vs[1] = scales[DECODE_KEYS + 8];
        }
        bool high = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[n][e] = (sc[n][e] + sd[n][e]) * ks[e >> 1];
            if (g + 8 * (e >> 1) >= left) sc[n][e] = -INFINITY;
            high |= sc[n][e] > m[n][e & 1] + 8.f;
          }
        if (__any_sync(0xFFFFFFFFu, high)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(m[n][e], fmaxf(sc[n][e], sc[n][e + 2]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
              const float f = top > m[n][e] ? ex2_approx(m[n][e] - top) : 1.f;
              m[n][e] = top;
              l[n][e] *= f;
#pragma unroll
              for (int k = 0; k < KS; ++k) acc[n][k][e] *= f, acc[n][k][e + 2] *= f;
            }
        }
        uint32_t pb[NT][2];
        if (I8 && left < 16) {
          if (g >= left) vs[0] = 0.f;
          if (g + 8 >= left) vs[1] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float base = m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1];
            p[e] = ex2_approx(sc[n][e] - base);
            l[n][e & 1] += p[e];
            if (I8) p[e] *= vs[e >> 1];
          }
          // [key][head] to [head][key]: the second operand of the next product
          pb[n][0] = transpose8x8(bf16x2_of(p[0], p[1]));
          pb[n][1] = transpose8x8(bf16x2_of(p[2], p[3]));
        }
        if (I8) {
          // a lane gets, for keys 2t and 2t + 1, elements 2g and 2g + 1: the
          // even ones stand as rows g, the odd ones as rows g + 8
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t r[4];
            ldsm_x4_t(line(vb, lane & 15, k + (lane >> 4)), r);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a0 = codes_to_bf16(r[2 * h]), a1 = codes_to_bf16(r[2 * h] >> 8);
              const uint32_t a2 = codes_to_bf16(r[2 * h + 1]), a3 = codes_to_bf16(r[2 * h + 1] >> 8);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_16x8x16(acc[n][k + h], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            }
          }
        } else {
          // rows past the end hold anything: 0 * NaN would be NaN
          uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;
          if (left < 16) {
            keep0 = (2 * t < left ? 0xFFFFu : 0u) | (2 * t + 1 < left ? 0xFFFF0000u : 0u);
            keep1 = (2 * t + 8 < left ? 0xFFFFu : 0u) | (2 * t + 9 < left ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t r[4];
            ldsm_x4_t(line(vb, (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), r);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_16x8x16(acc[n][k], r[0] & keep0, r[1] & keep0, r[2] & keep1, r[3] & keep1, pb[n][0], pb[n][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (!b.last) continue;

      // ---- join the four warps
      float* st = stat + parity * 4 * NQ * 2;
      float* all = stat_all + parity * NQ * 2;
      parity ^= 1u;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], o);
          if (g == 0) {
            st[(warp * NQ + n * 8 + 2 * t + e) * 2] = m[n][e];
            st[(warp * NQ + n * 8 + 2 * t + e) * 2 + 1] = l[n][e];
          }
        }
      if (!rendezvous()) break;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = n * 8 + 2 * t + e;
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) top = fmaxf(top, st[(x * NQ + h) * 2]);
          const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
          for (int x = 0; x < 4; ++x) sum += st[(x * NQ + h) * 2 + 1] * ex2_approx(st[(x * NQ + h) * 2] - base);
          if (warp == 0 && g == 0) all[h * 2] = top, all[h * 2 + 1] = sum;
          const float f = ex2_approx(m[n][e] - base);
          if (h < heads) {
            float* o = join + (warp * heads + h) * SM::PAD;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[16 * k + (I8 ? 2 * g : g)] = acc[n][k][e] * f;
              o[16 * k + (I8 ? 2 * g + 1 : g + 8)] = acc[n][k][e + 2] * f;
            }
          }
        }
      if (!rendezvous()) break;
      const int kvh = b.unit / a.chunks, chunk = b.unit - kvh * a.chunks, group = a.q_heads / a.kv_heads;
      const int qh = min(heads, group - chunk * heads);
      uint16_t* out = a.o + b.seq * a.o_stride + (static_cast<int64_t>(kvh) * group + chunk * heads) * D;
      const int part_floats = decode_part_floats(heads, D);
      auto joined = [&](int h, int d) -> float4 {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float4 y = *reinterpret_cast<const float4*>(join + (x * heads + h) * SM::PAD + d);
          v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
        }
        return v;
      };
      auto store = [&](int h, int d, float4 v, float sum) {
        const float inv = b.left > 0 || sum > 0.f ? 1.f / sum : 0.f;  // a sequence without keys: 0
        *reinterpret_cast<uint2*>(out + h * D + d) = make_uint2(bf16x2_of(v.x * inv, v.y * inv), bf16x2_of(v.z * inv, v.w * inv));
      };
      if (b.n_parts == 1) {
        for (int x = threadIdx.x; x < qh * (D / 4); x += 128) {
          const int h = x / (D / 4), d = (x % (D / 4)) * 4;
          store(h, d, joined(h, d), all[h * 2 + 1]);
        }
        continue;
      }
      // a part: the owner's in slot 1, every other CTA's in slot 0
      float* mine = a.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (b.owner == blockIdx.x ? 1 : 0)) * part_floats;
      for (int x = threadIdx.x; x < qh * (D / 4); x += 128) {
        const int h = x / (D / 4), d = (x % (D / 4)) * 4;
        *reinterpret_cast<float4*>(mine + h * D + d) = joined(h, d);
      }
      for (int h = threadIdx.x; h < qh; h += 128) {
        mine[heads * D + 2 * h] = all[2 * h];
        mine[heads * D + 2 * h + 1] = all[2 * h + 1];
      }
      if (!rendezvous()) break;
      if (threadIdx.x == 0) {
        __threadfence();
        const unsigned before = atomic_add_acq_rel_gpu(&a.counters[b.owner], 1u);
        *is_last = before + 1 == static_cast<unsigned>(b.n_parts);
        if (before + 1 == static_cast<unsigned>(b.n_parts)) a.counters[b.owner] = 0;
      }
      if (!rendezvous()) break;
      if (!*is_last) continue;
      for (int x = threadIdx.x; x < qh * (D / 4); x += 128) {
        const int h = x / (D / 4), d = (x % (D / 4)) * 4;
        float top = -INFINITY, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < b.n_parts; ++p) {
          float* part = a.parts + (static_cast<int64_t>(b.owner + p) * 2 + (p == 0 ? 1 : 0)) * part_floats;
          const float pm = __ldcg(part + heads * D + 2 * h), pl = __ldcg(part + heads * D + 2 * h + 1);
          const float4 y = __ldcg(reinterpret_cast<const float4*>(part + h * D + d));
          *reinterpret_cast<float4*>(part + h * D + d) = make_float4(0.f, 0.f, 0.f, 0.f);  // as it was found
          const float up = fmaxf(top, pm), base = up == -INFINITY ? 0.f : up;
          const float f = ex2_approx(top - base), fp = ex2_approx(pm - base);
          top = up;
          sum = sum * f + pl * fp;
          v.x = v.x * f + y.x * fp;
          v.y = v.y * f + y.y * fp;
          v.z = v.z * f + y.z * fp;
          v.w = v.w * f + y.w * fp;
        }
        store(h, d, v, sum);
      }
      if (!rendezvous()) break;
      for (int x = threadIdx.x; x < b.n_parts * 2 * qh; x += 128) {
        const int p = x / (2 * qh);
        a.parts[(static_cast<int64_t>(b.owner + p) * 2 + (p == 0 ? 1 : 0)) * part_floats + heads * D + x - p * 2 * qh] = 0.f;
      }
    }
  }
}

}  // namespace convrot
