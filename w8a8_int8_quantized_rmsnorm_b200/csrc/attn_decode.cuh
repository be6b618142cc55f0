// Attention of one new token per sequence over a paged cache: a stream of
// every key and value, once, at memory speed.
//
// Work split.  The unit of work is a block of 64 keys (128 of int8) of one (sequence,
// key/value head); the heads of its group (up to 8 or 16 at a time) share it.
// All blocks of the call are laid out in one line, sequence by sequence and
// head by head, and every CTA takes an equal stretch of the line, so sequences
// of any mix of lengths keep every SM streaming to the end.  A stretch covers
// the tail of one (sequence, head), any number of whole ones, and the front of
// another.  Whole ones are finished in place; a part leaves its (m, l, O) in
// the workspace, and the part that comes last, found by a counter, joins all
// of them in the order of the keys, so the result does not depend on timing.
//
// Inside a CTA one warp fetches (the block table's entries a batch of blocks
// ahead, then one TMA box per page piece, into a ring of blocks) and four warps
// compute, each 16 keys of a block (32 of int8), on warp-level matrix instructions with the
// keys as rows and the heads as columns: S^T = K Q^T and O^T += V^T P^T, so a
// group of four or eight heads fills the 8-column operand and every score
// stays with the lane that made it.
//
// Each warp keeps a reference maximum per head, raised (with O and l) only
// when a score lies more than 2^8 above it, and fp32 sums; probabilities are
// rounded to bf16 for the product with V.
//
// int8 caches.  Turning codes into bf16 costs 7 instructions per 4 codes, more
// than the stream leaves time for (both sides converted: 288 us for 128 contexts
// of 1 .. 8192 keys; the values alone: 215 us).  So both products are integer
// ones on the codes as they are.  A head's query becomes 16-bit fixed point,
// q = s (256 hi + lo) with s = max|q| / 32512, and hi and lo are two columns of
// one s8 x s8 -> s32 product; probabilities times value scales become the same,
// of the largest among a warp's 32 keys, and their sum joins the fp32 result.
// The integer sums are exact.  The query is off by at most half a step, 1/65024
// of its largest element, which moves a score by scale max|q| sum|k| / 65024 at
// most; a probability times its scale by 1/65024 of the largest beside it, where
// bf16 would be off by up to 2^-8 of itself.  Scales are taken to be 0 or more.
//
// Measured (32 query heads on 8, D = 128; graph replays): 64 contexts of 1 .. 8192
// keys, 1.2 GB of bf16, 183 us (6.56 TB/s, a copy's rate); 128 such contexts in
// int8, 1.14 GB, 176 us (6.48 TB/s, 0.99); one context of 131071, 93 us (0.88:
// about 8 us go into finding the stretch, the first fetch and the join of 37
// parts per head); one of 777, 10.7 us, those alone.  The batches of pages
// matter: with the block table read one block ahead the int8 stream took 231 us,
// each block waiting for a table entry that the stream itself had driven out of L2.
//
// Groups above 8 heads are slower: the second tile of columns spills (100 to 230
// bytes a thread) and leaves two ring slots.  64 such contexts with groups of 16
// on 8: bf16 238 us (5.07 TB/s), int8 205 us (3.05 TB/s).  Above 16 heads a unit
// takes 16 at a time and the cache is streamed once for each: 128 such contexts
// with 32 heads on one, 0.28 GB once, 111 us; 128 on one, 364 us.
//
// Rows past a sequence's end are never used: their scores are replaced, their
// values' registers cleared, pages behind the last one not fetched.  Neither is
// a page whose number is outside the cache; a sequence without a key that could
// be read is 0, told from one whose scores are all -inf (NaN) by its maximum.
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

constexpr int DECODE_THREADS = 160;
constexpr unsigned SITE_DECODE = 20;
constexpr int DECODE_MAX_STAGES = 8;

// A part: O [heads][D], then (m, l) [heads], to a multiple of 16 bytes.
__host__ __device__ constexpr int decode_part_floats(int heads, int D) { return heads * D + (2 * heads + 3) / 4 * 4; }

// What a ring slot holds besides keys and values.
struct DecodeBlock {
  int left;             // keys of the sequence from the block's first one on
  unsigned flags;       // bits 0-7: the 16-key slices that are there; then:
  int seq, unit;        // unit: (kv head, head chunk)
  int owner, n_parts;   // CTA of the (seq, unit)'s first block; parts (1: whole)
  int heads;            // query heads of the unit that there are
  int pad;
};
// The maximum of keys that all score -inf; -inf itself: there were no keys.
constexpr float LOWEST = -3.402823466e38f;
// begins / ends this CTA's stretch of the (seq, unit); no more blocks
constexpr unsigned BLOCK_FIRST = 256, BLOCK_LAST = 512, BLOCK_END = 1024;

template <int D, bool I8, int NQ>
struct DecodeSmem {
  static constexpr int ESZ = I8 ? 1 : 2;
  static constexpr int CTAS = 2;               // per SM; a ring holds two blocks (bf16 at D = 128: 64 KB) to six
  static constexpr int KEYS = I8 ? 128 : 64;  // of a block: the same bytes, a multiple of 4 warps x 32 or 16 keys
  static constexpr int TILE = KEYS * D * ESZ;
  static constexpr int SLOT = 2 * TILE;                            // K, V
  static constexpr int SIDE = NQ * D * 2 + 2 * KEYS * 4;    // Q rows, scales
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
// d += a (16 x 32, rows) * b (32 x 8, columns), int8 in, int32 out
__device__ __forceinline__ void mma_16x8x32(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a * b, the same shapes
__device__ __forceinline__ void mma_16x8x32_zero(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
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
template <int KEYS>
__device__ __forceinline__ int decode_blocks(int len) {
  return max(1, static_cast<int>((static_cast<unsigned>(len) + KEYS - 1) / KEYS));
}

template <int D, bool I8, int NQ>
__global__ void __launch_bounds__(DECODE_THREADS, DecodeSmem<D, I8, NQ>::CTAS)
decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const DecodeArgs a) {
  using SM = DecodeSmem<D, I8, NQ>;
  constexpr int ROWB = D * SM::ESZ >= 128 ? 128 : 64;  // bytes of a swizzled line
  constexpr int HALVES = D * SM::ESZ / ROWB;
  constexpr int HL = NQ / 4;                           // heads of a lane
  constexpr int NT = (HL + 1) / 2;                     // 8-column tiles of P and O
  constexpr int KS = D / 16;                           // 16-element steps
  constexpr int KEYS = SM::KEYS, SLICE = KEYS / 4;     // keys of a block, of a warp's share of it
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

  const unsigned units = a.kv_heads * a.chunks;
  if (warp == 4) {
    // -------------------------------------------------------- fetch
    // this CTA's stretch [begin, end) of the line of blocks
    unsigned total = 0;  // the host has seen that line indices fit in 31 bits
    for (int b0 = lane; b0 < a.seqs; b0 += 128) {
      int n = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x)  // four loads in flight
        if (b0 + 32 * x < a.seqs) n += decode_blocks<KEYS>(decode_length(a, b0 + 32 * x));
      total += n;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    total *= units;
    const unsigned per = (total + gridDim.x - 1) / gridDim.x, begin = min(total, per * blockIdx.x), end = min(total, begin + per);

    // A batch: consecutive blocks of one (sequence, unit), as many as a warp's
    // lanes can hold the pages of, so that the block table's latency is paid
    // once per batch and behind the one before.
    const int boxes = KEYS / a.box_rows, most = 32 / boxes;
    const unsigned page_size = a.page_size;
    struct Batch {
      unsigned at, start;  // line index of the batch, and of the sequence's first block
      int seq, unit, len, nb, j, n;
    } cur = {begin, 0, 0, 0, 0, 1, 0, 0}, next;
    if (begin < end) {
      for (int b0 = 0;; b0 += 32) {
        const int ln = b0 + lane < a.seqs ? decode_length(a, b0 + lane) : 0;
        const int n = b0 + lane < a.seqs ? decode_blocks<KEYS>(ln) : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
          if (lane >= o) sum += up;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, cur.start + static_cast<unsigned>(sum) * units > begin);
        if (hit) {
          const int l = __ffs(hit) - 1;
          cur.seq = b0 + l;
          cur.len = __shfl_sync(0xFFFFFFFFu, ln, l);
          cur.nb = decode_blocks<KEYS>(cur.len);
          cur.start += static_cast<unsigned>(__shfl_sync(0xFFFFFFFFu, sum, l) - cur.nb) * units;
          break;
        }
        cur.start += static_cast<unsigned>(__shfl_sync(0xFFFFFFFFu, sum, 31)) * units;
      }
      cur.unit = static_cast<int>((begin - cur.start) / static_cast<unsigned>(cur.nb));
      cur.j = static_cast<int>(begin - cur.start) - cur.unit * cur.nb;
    }
    auto size = [&](const Batch& b) {
      return min(min(most, b.nb - b.j), static_cast<int>(end - b.at));
    };
    // page of this lane's box of the batch; -1: not there
    auto pages_of = [&](const Batch& b) -> int {
      const unsigned key = static_cast<unsigned>(b.j) * KEYS + lane * a.box_rows;
      if (lane >= b.n * boxes || key >= static_cast<unsigned>(b.len)) return -1;
      return a.table[b.seq * a.table_stride + key / page_size];
    };
    bool ok = true;
    uint32_t it = 0, s = 0, phase = 1;  // slot and the parity its last emptying has
    cur.n = size(cur);
    int page = begin < end ? pages_of(cur) : -1;
    const int group = a.q_heads / a.kv_heads;
    int next_len = cur.seq + 1 < a.seqs ? decode_length(a, cur.seq + 1) : 0;
    while (cur.at < end && ok) {
      // where the line goes on, and that batch's pages
      next = cur;
      next.at += cur.n;
      next.j += cur.n;
      if (next.j == cur.nb) {
        next.j = 0;
        if (++next.unit == static_cast<int>(units)) {
          next.unit = 0;
          ++next.seq;
          next.start += static_cast<unsigned>(cur.nb) * units;
          next.len = next_len;
          next.nb = decode_blocks<KEYS>(next_len);
        }
      }
      int page2 = -1;
      if (next.at < end) {
        next.n = size(next);
        const bool same = next.seq == cur.seq && next.j == cur.j && next.n <= cur.n;  // another head, the same pages
        page2 = same ? page : pages_of(next);
        if (next.seq != cur.seq) next_len = next.seq + 1 < a.seqs ? decode_length(a, next.seq + 1) : 0;
      }
      const int kvh = cur.unit / a.chunks, chunk = cur.unit - kvh * a.chunks;
      const int qh = min(heads, group - chunk * heads);
      const unsigned item = cur.start + static_cast<unsigned>(cur.unit) * cur.nb;
      for (int i = 0; i < cur.n; ++i) {
        ok = mbar_wait_spin(&empty[s], phase, abort_flag, SITE_DECODE);
        if (!ok) break;
        const int j = cur.j + i;
        const int mine = __shfl_sync(0xFFFFFFFFu, page, (i * boxes + lane) & 31);
        const unsigned key = static_cast<unsigned>(j) * KEYS + lane * a.box_rows;  // of this lane's box
        const bool wanted = lane < boxes && key < static_cast<unsigned>(cur.len);
        const bool there = wanted && mine >= 0 && mine < a.pages;
        if (wanted && !there) report_error(ERR_BAD_ARGUMENT);
        const unsigned mask = __ballot_sync(0xFFFFFFFFu, there);
        const bool first = cur.at + i == begin || j == 0;
        const bool last = cur.at + i + 1 == end || j + 1 == cur.nb;
        if (lane == 0) {
          DecodeBlock m;
          m.seq = cur.seq;
          m.unit = cur.unit;
          m.left = cur.len - j * KEYS;
          m.flags = (first ? BLOCK_FIRST : 0) | (last ? BLOCK_LAST : 0);
          for (int x = 0; x < KEYS / 16; ++x) m.flags |= ((mask >> (16 * x / a.box_rows)) & 1u) << x;
          m.heads = qh;
          m.pad = 0;
          m.owner = blockIdx.x;
          m.n_parts = 1;
          if (last && (item < begin || item + cur.nb > end)) {  // twice per CTA at most: its two ends
            m.owner = static_cast<int>(item / per);
            m.n_parts = static_cast<int>((item + cur.nb - 1) / per) - m.owner + 1;
          }
          meta[s] = m;
          const uint32_t bytes = __popc(mask) * a.box_rows * (2 * D * SM::ESZ + (I8 ? 8 : 0)) + (first ? qh * D * 2 : 0);
          mbar_arrive_expect_tx(&full[s], bytes);
          if (first)
            bulk_load_1d(side + s * SM::SIDE,
                         a.q + cur.seq * a.q_stride + (static_cast<int64_t>(kvh) * group + chunk * heads) * D, qh * D * 2,
                         &full[s]);
        }
        __syncwarp();
        if (there) {
          const int64_t row = (static_cast<int64_t>(mine) * a.kv_heads + kvh) * page_size + key % page_size;
          uint8_t* dst = smem + s * SM::SLOT + lane * a.box_rows * D * SM::ESZ;
          tma_load_3d(dst, &tm_k, &full[s], 0, static_cast<int>(row), 0);
          tma_load_3d(dst + SM::TILE, &tm_v, &full[s], 0, static_cast<int>(row), 0);
          if (I8) {
            float* sc = reinterpret_cast<float*>(side + s * SM::SIDE + NQ * D * 2) + lane * a.box_rows;
            bulk_load_1d(sc, a.k_scale + row, a.box_rows * 4, &full[s]);
            bulk_load_1d(sc + KEYS, a.v_scale + row, a.box_rows * 4, &full[s]);
          }
        }
        ++it;
        if (++s == static_cast<uint32_t>(S)) s = 0, phase ^= 1u;
      }
      cur = next;
      page = page2;
    }
    ok = ok && mbar_wait_spin(&empty[s], phase, abort_flag, SITE_DECODE);
    if (ok && lane == 0) {
      meta[s].flags = BLOCK_END;
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
    // A lane's scores: keys g and g + 8, heads head(0 .. HL-1); head(x) is
    // column 2 t + (x & 1) of tile x / 2 in P and O.
    auto head = [&](int x) { return I8 ? 4 * x + t : (x / 2) * 8 + 2 * t + (x & 1); };
    uint32_t qf[I8 ? HL : NT][KS][I8 ? 1 : 2];  // queries as the second operand
    float qs[HL];                               // int8: scale of the head's query
    float acc[I8 ? HL : NT][KS][I8 ? 2 : 4];    // element rows g, g + 8 (int8: 2g, 2g + 1) of each step
    float m[HL], l[HL];
    auto out_at = [&](int x, int k, int r) -> float& { return acc[I8 ? x : x / 2][k][I8 ? r : (x & 1) + 2 * r]; };
    uint32_t met = 0, parity = 0;
    bool seen = false;  // this warp has met a key of the stretch
    // bounded rendezvous of the four compute warps
    auto rendezvous = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      return mbar_wait_spin(meet, met++ & 1u, abort_flag, SITE_DECODE + 1);
    };
    // where the 16 keys from `key` on begin inside a tile
    auto slice_at = [&](int key) -> uint32_t {
      const int box = key / a.box_rows;
      return box * a.box_rows * D * SM::ESZ + (key - box * a.box_rows) * ROWB;
    };
    const uint32_t slice[2] = {slice_at(SLICE * warp), slice_at(SLICE * warp + (I8 ? 16 : 0))};
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
      const unsigned flags = meta[s].flags;
      const int block_left = meta[s].left;
      if (flags & BLOCK_END) break;
      if (flags & BLOCK_FIRST) {
        const uint8_t* rows = side + s * SM::SIDE;
        const int live = meta[s].heads;  // the rows past them hold anything: zero
        if (I8) {
          // columns 2h and 2h + 1 of a tile: hi and lo of head h; this lane's is column g
#pragma unroll
          for (int x = 0; x < HL; ++x) {
            const uint8_t* p = rows + (4 * x + (g >> 1)) * D * 2 + 8 * t;
            float v[KS][4], top = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint2 w = make_uint2(0, 0);
              if (4 * x + (g >> 1) < live) w = *reinterpret_cast<const uint2*>(p + 32 * k);  // elements 16k + 4t ..
              v[k][0] = __uint_as_float(w.x << 16), v[k][1] = __uint_as_float(w.x & 0xFFFF0000u);
              v[k][2] = __uint_as_float(w.y << 16), v[k][3] = __uint_as_float(w.y & 0xFFFF0000u);
#pragma unroll
              for (int e = 0; e < 4; ++e) top = max_nan(top, fabsf(v[k][e]));
            }
            top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            // scaled up first where 1 / top would overflow
            const float up = top < 1e-30f ? 0x1p64f : 1.f;
            const float inv = top > 0.f ? 32512.f / (top * up) : 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              qf[x][k][0] = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int q = max(-32512, min(32512, __float2int_rn(v[k][e] * up * inv)));
                const int hi = (q + 128) >> 8, lo = q - hi * 256;
                qf[x][k][0] |= (static_cast<uint32_t>(g & 1 ? lo : hi) & 0xFFu) << (8 * e);
              }
            }
            // the scores' scale belongs to head 4x + t, held by lanes g = 2t, 2t + 1
            qs[x] = __shfl_sync(0xFFFFFFFFu, top, 8 * t) * (1.f / 32512.f);
          }
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              const uint8_t* p = rows + ((n * 8 + g) * D + k * 16) * 2;
              const bool mine = n * 8 + g < live;
              qf[n][k][0] = mine ? *reinterpret_cast<const uint32_t*>(p + 4 * t) : 0u;
              qf[n][k][I8 ? 0 : 1] = mine ? *reinterpret_cast<const uint32_t*>(p + 16 + 4 * t) : 0u;
            }
        }
#pragma unroll
        for (int n = 0; n < (I8 ? HL : NT); ++n)
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < (I8 ? 2 : 4); ++e) acc[n][k][e] = 0.f;
#pragma unroll
        for (int x = 0; x < HL; ++x) m[x] = -INFINITY, l[x] = 0.f;
        seen = false;
      }
      const int left = block_left - SLICE * warp;  // keys of this warp's share that exist
      const unsigned there = (flags >> (SLICE / 16 * warp)) & (I8 ? 3u : 1u);
      if (left > 0 && there) {
        seen = true;
        const uint32_t kb = smem_addr(smem + s * SM::SLOT), vb = kb + SM::TILE;
        constexpr int NR = SLICE / 8;  // keys g + 8 r, r < NR, are this lane's
        float sc[HL][NR];              // their scores, times log2(e)
        float vs[NR];
        if constexpr (I8) {
          const float* scales = reinterpret_cast<const float*>(side + s * SM::SIDE + NQ * D * 2) + SLICE * warp + g;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            int c[HL][4] = {};
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
              uint32_t r[4];
              ldsm_x4(line(kb + slice[u], lane & 15, k + (lane >> 4)), r);
#pragma unroll
              for (int x = 0; x < HL; ++x) mma_16x8x32(c[x], r, qf[x][k][0], qf[x][k + 1][0]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float ks = scales[16 * u + 8 * r] * a.scale_log2;
              vs[2 * u + r] = scales[KEYS + 16 * u + 8 * r];
#pragma unroll
              for (int x = 0; x < HL; ++x)  // |256 hi + lo| < 2^30
                sc[x][2 * u + r] = static_cast<float>(c[x][2 * r] * 256 + c[x][2 * r + 1]) * qs[x] * ks;
            }
          }
        } else {
          float c[NT][4] = {}, d[NT][4] = {};  // two chains of products
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t r[4];
            ldsm_x4(line(kb + slice[0], lane & 15, 2 * k + (lane >> 4)), r);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16x8x16(k & 1 ? d[n] : c[n], r[0], r[1], r[2], r[3], qf[n][k][0], qf[n][k][1]);
          }
#pragma unroll
          for (int x = 0; x < HL; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r) sc[x][r] = (c[x / 2][2 * r + (x & 1)] + d[x / 2][2 * r + (x & 1)]) * a.scale_log2;
        }
        if (left < SLICE || (I8 && there != 3u)) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (g + 8 * r >= left || !((there >> (r / 2)) & 1u)) {
              vs[r] = 0.f;
#pragma unroll
              for (int x = 0; x < HL; ++x) sc[x][r] = -INFINITY;
            }
        }
        bool high = false;
#pragma unroll
        for (int x = 0; x < HL; ++x)
#pragma unroll
          for (int r = 0; r < NR; ++r) high |= sc[x][r] > m[x] + 8.f;
        if (__any_sync(0xFFFFFFFFu, high)) {
#pragma unroll
          for (int x = 0; x < HL; ++x) {
            float top = m[x];
#pragma unroll
            for (int r = 0; r < NR; ++r) top = fmaxf(top, sc[x][r]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            // each head by its own scores: its result depends on nothing else
            const bool up = top > m[x] + 8.f;
            const float f = up ? ex2(m[x] - top) : 1.f;
            if (up) m[x] = top;
            l[x] *= f;
#pragma unroll
            for (int k = 0; k < KS; ++k) out_at(x, k, 0) *= f, out_at(x, k, 1) *= f;
          }
        }
        float p[I8 ? HL : 2 * NT][NR] = {};
#pragma unroll
        for (int x = 0; x < HL; ++x) {
          const float base = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            p[x][r] = ex2(sc[x][r] - base);
            l[x] += p[x][r];
            if (I8) p[x][r] *= vs[r];
          }
        }
        if constexpr (I8) {
          // probabilities times scales in 16-bit fixed point, of the largest
          // among these 32 keys: hi and lo in the columns of the head
          float ps[HL];
          uint32_t pb[HL][2];
#pragma unroll
          for (int x = 0; x < HL; ++x) {
            float top = max_nan(max_nan(p[x][0], p[x][1]), max_nan(p[x][2], p[x][3]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            // (scaled towards 1 first, by a power of two: 1 / top may overflow, and
            // the fast division is 0 for divisors above 2^126)
            const float up = top < 1.f ? 0x1p64f : 0x1p-64f, inv = top > 0.f ? __fdividef(32512.f, top * up) : 0.f;
            ps[x] = top * (1.f / 32512.f);
            uint32_t mv[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int q = min(32512, __float2int_rn(p[x][r] * up * inv));
              // hi = (q + 128) >> 8 in byte 0, lo in byte 2: [key][column] to [column][key]
              mv[r] = transpose8x8(__byte_perm(q + 128, q, 0x4411));
            }
            pb[x][0] = __byte_perm(mv[0], mv[1], 0x6420);
            pb[x][1] = __byte_perm(mv[2], mv[3], 0x6420);
          }
          // A lane gets, for keys 2t and 2t + 1 of each eight, elements 2g and
          // 2g + 1: the even ones stand as rows g, the odd ones as rows g + 8,
          // and the keys in the order of the probabilities' bytes.
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t r[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) ldsm_x4_t(line(vb + slice[u], lane & 15, k + (lane >> 4)), r[u]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a0 = __byte_perm(r[0][2 * h], r[0][2 * h + 1], 0x6420);
              const uint32_t a1 = __byte_perm(r[0][2 * h], r[0][2 * h + 1], 0x7531);
              const uint32_t a2 = __byte_perm(r[1][2 * h], r[1][2 * h + 1], 0x6420);
              const uint32_t a3 = __byte_perm(r[1][2 * h], r[1][2 * h + 1], 0x7531);
#pragma unroll
              for (int x = 0; x < HL; ++x) {
                int c[4];
                mma_16x8x32_zero(c, a0, a1, a2, a3, pb[x][0], pb[x][1]);
                acc[x][k + h][0] = fmaf(static_cast<float>(c[0] * 256 + c[1]), ps[x], acc[x][k + h][0]);
                acc[x][k + h][1] = fmaf(static_cast<float>(c[2] * 256 + c[3]), ps[x], acc[x][k + h][1]);
              }
            }
          }
        } else {
          uint32_t pb[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n)  // [key][head] to [head][key]: the second operand of the next product
#pragma unroll
            for (int r = 0; r < 2; ++r) pb[n][r] = transpose8x8(bf16x2(p[2 * n][r], p[2 * n + 1][r]));
          // rows past the end hold anything: 0 * NaN would be NaN
          uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;
          if (left < 16) {
            keep0 = (2 * t < left ? 0xFFFFu : 0u) | (2 * t + 1 < left ? 0xFFFF0000u : 0u);
            keep1 = (2 * t + 8 < left ? 0xFFFFu : 0u) | (2 * t + 9 < left ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t r[4];
            ldsm_x4_t(line(vb + slice[0], (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), r);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_16x8x16(acc[n][k], r[0] & keep0, r[1] & keep0, r[2] & keep1, r[3] & keep1, pb[n][0], pb[n][1]);
          }
        }
      }
      DecodeBlock b;
      if (flags & BLOCK_LAST) b = meta[s];
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (!(flags & BLOCK_LAST)) continue;

      // ---- join the four warps
      float* st = stat + parity * 4 * NQ * 2;
      float* all = stat_all + parity * NQ * 2;
      parity ^= 1u;
#pragma unroll
      for (int x = 0; x < HL; ++x) {
        if (seen) m[x] = fmaxf(m[x], LOWEST);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], o);
        if (g == 0) {
          st[(warp * NQ + head(x)) * 2] = m[x];
          st[(warp * NQ + head(x)) * 2 + 1] = l[x];
        }
      }
      if (!rendezvous()) break;
#pragma unroll
      for (int x = 0; x < HL; ++x) {
        const int h = head(x);
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int y = 0; y < 4; ++y) top = fmaxf(top, st[(y * NQ + h) * 2]);
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int y = 0; y < 4; ++y) sum += st[(y * NQ + h) * 2 + 1] * ex2(st[(y * NQ + h) * 2] - base);
        if (warp == 0 && g == 0) all[h * 2] = top, all[h * 2 + 1] = sum;
        const float f = ex2(m[x] - base);
        if (h < heads) {
          float* o = join + (warp * heads + h) * SM::PAD;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            o[16 * k + (I8 ? 2 * g : g)] = out_at(x, k, 0) * f;
            o[16 * k + (I8 ? 2 * g + 1 : g + 8)] = out_at(x, k, 1) * f;
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
      auto store = [&](int h, int d, float4 v, float top, float sum) {
        const float inv = top == -INFINITY ? 0.f : 1.f / sum;  // a sequence without keys: 0
        *reinterpret_cast<uint2*>(out + h * D + d) = make_uint2(bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
      };
      if (b.n_parts == 1) {
        for (int x = threadIdx.x; x < qh * (D / 4); x += 128) {
          const int h = x / (D / 4), d = (x % (D / 4)) * 4;
          store(h, d, joined(h, d), all[h * 2], all[h * 2 + 1]);
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
        const unsigned before = atomic_add_acq_rel_gpu(&a.counters[b.owner], 1u);
        *is_last = before + 1 == static_cast<unsigned>(b.n_parts);
        if (before + 1 == static_cast<unsigned>(b.n_parts)) a.counters[b.owner] = 0;
      }
      if (!rendezvous()) break;
      if (!*is_last) continue;
      // the last part to come joins them all, in the keys' order, eight in flight
      auto part = [&](int p) {
        return a.parts + (static_cast<int64_t>(b.owner + p) * 2 + (p == 0 ? 1 : 0)) * part_floats;
      };
      for (int x = threadIdx.x; x < qh * (D / 4); x += 128) {
        const int h = x / (D / 4), d = (x % (D / 4)) * 4;
        float top = -INFINITY, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = 0; p0 < b.n_parts; p0 += 8) {
          float2 ml[8];
          float4 y[8];
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            ml[p] = make_float2(-INFINITY, 0.f);
            y[p] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p0 + p < b.n_parts) {
              const float* from = part(p0 + p);
              ml[p] = __ldcg(reinterpret_cast<const float2*>(from + heads * D) + h);
              y[p] = __ldcg(reinterpret_cast<const float4*>(from + h * D + d));
            }
          }
          float up = top;
#pragma unroll
          for (int p = 0; p < 8; ++p) up = fmaxf(up, ml[p].x);
          const float base = up == -INFINITY ? 0.f : up, f = ex2(top - base);
          top = up;
          sum *= f;
          v.x *= f, v.y *= f, v.z *= f, v.w *= f;
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const float fp = ex2(ml[p].x - base);
            sum = fmaf(ml[p].y, fp, sum);
            v.x = fmaf(y[p].x, fp, v.x);
            v.y = fmaf(y[p].y, fp, v.y);
            v.z = fmaf(y[p].z, fp, v.z);
            v.w = fmaf(y[p].w, fp, v.w);
          }
        }
        store(h, d, v, top, sum);
      }
      if (!rendezvous()) break;
      for (int x = threadIdx.x; x < b.n_parts * (part_floats / 4); x += 128)  // as it was found
        reinterpret_cast<float4*>(part(x / (part_floats / 4)))[x % (part_floats / 4)] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

}  // namespace convrot
