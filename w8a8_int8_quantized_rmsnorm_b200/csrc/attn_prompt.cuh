// Attention over whole prompts, packed one after another, on the 5th-generation
// tensor cores.
//
//   O_i = sum_j softmax_j(scale q_i . k_j) v_j  over the keys row i sees
//
// One pass over the keys with a running reference m and sum l per row:
//   P = exp2(c S - c m), S = Q K^T, c = scale log2(e);  l += sum P;  O += P V
// m is a score that was the row's maximum at some point, not at every point:
// it is raised (and O and l multiplied by exp2(c (m_old - m_new))) only when a
// tile's maximum is more than 2^8 above it, so P stays below 256, O and l in
// fp32 lose nothing, and the accumulator is almost never re-read.  P is rounded
// to bf16 for its product with V (half a step, 2^-8 of a probability, as the
// result itself is); l is summed from the unrounded values.
//
// Work split.  A unit is 2 x 128 query rows of one key/value head: a row is
// (token, query head of the group), so a group's heads share every key and
// value tile and a short prompt still fills the matrix unit.  The grid has one
// CTA per unit, from the pack's end to its front, so that of a sequence the
// units with the most keys come first; one runs per SM, and when a unit's last
// copies are under way it takes over the next unit that has not started
// (clusterlaunchcontrol.try_cancel) instead of ending: a pack of very different
// lengths spreads evenly, and a unit's results are stored while the next one
// runs.  The next unit is asked for behind this one's last copy, so what a change
// of units costs shows where units are of one or two key tiles.
// Warps 0-3 and 4-7 each own one 128-row tile (a thread owns a row; no
// exchange between threads), warp 8 fetches by TMA and announces units, warp 9
// issues the matrix products.  While one tile's softmax runs, the tensor core
// works on the other's S or O.
//
// Tensor memory: S0, S1 (128 columns each; P overwrites its own S), O0, O1.
// Shared memory: the two Q tiles and a ring of K and V tiles (128 keys).
//
// Measured (32 query heads on 8, D = 128, causal; graph replays): 8192 tokens 417
// us at 1965 MHz (1.32 PFLOP/s, 0.81 of cuBLAS's burst rate), 487 us one after
// another under the power cap at 1580 MHz (0.82 of its sustained rate); 2048
// tokens 35 us on inputs that L2 still holds, 37 us on others, 39 us under the
// cap; 34 prompts of 16 .. 300 tokens 42 us, 2.8 TB/s.  With D = 64, groups of 8 and
// 12 prompts of 1 .. 1333: 76 us.
//
// A key tile of both row tiles takes 3600 cycles (8192 tokens: 225 of them per
// SM).  Its products need 2050 at the tensor core's rate, its exponentials as
// many (2 x 128 x 128, 16 a cycle); in 2048 tokens the tensor core is busy for 48 %
// of the cycles and the exponential unit for 48 %, in the D = 64 pack for 27 % and
// 53 %.  So no unit is full: what passes is a row tile's chain, from clock stamps
// scores 590 (both operands come from shared memory, 8 KB per 64 cycles, its whole
// bandwidth), fetching them 190, maximum 430, 128 exponentials a row 1500, the
// rest of the product with V 256, and four hand-overs between the issuing warp,
// which serves the two row tiles in a fixed order, and the softmax.  How much of
// it the hand-overs and that order are is not settled: without exponentials,
// maxima and conversions 4096 tokens still took 110 us of 115.
// Tensor memory has no room for a third row tile.  Measured no faster: steps of
// 64 keys with two S buffers (142 us for 4096 tokens: 128 x 64 products are bound
// by the reads of Q), P apart from S at D = 64 (104 us instead of 99: without
// turns both tiles reach their exponentials together), a quarter of the
// exponentials as a cubic on the multiply-add pipe (the same at D = 128, 0.5 % less
// at D = 64), three ring slots instead of four and room for whole result tiles
// (525 us for 8192 tokens under the cap).  Handing units out by cluster launch
// control instead of a fixed order took the ragged pack from 103 to 81 us.
//
// A probability of zero times an infinite or NaN value is NaN in the matrix
// unit.  Such a value may sit in a masked place (a later token, the next
// sequence of the pack, memory behind the last one), so a row whose result
// holds a NaN is computed again by attention_row over its visible keys alone.
// That is one warp's work at scalar speed: where every row sees a value with one
// NaN element, 2048 tokens take 18 ms and 8192 take 246 ms.
#pragma once

#include "attn_row.cuh"

namespace convrot {

struct PromptArgs {
  const uint16_t *q, *k, *v;                       // bf16 [tokens, heads, D]
  int64_t q_stride, k_stride, v_stride, o_stride;  // elements per token
  uint16_t* o;
  const int32_t *cu_q, *cu_k;                      // [seqs + 1]
  int tokens, kv_tokens, seqs, q_heads, kv_heads;
  int tile_heads;                                  // query heads of one tile (<= 128)
  int tile_tokens;                                 // tokens of one tile: 128 / tile_heads
  int head_chunks;                                 // tiles side by side for one group
  float scale_log2;                                // scale * log2(e)
  int causal;
  int boxed;                                       // a warp's 32 rows are whole tokens: tile_heads divides 32
};

constexpr int PROMPT_KEYS = 128;     // keys per tile
constexpr int PROMPT_HALF = 64;      // a last tile of no more keys than this is half a tile
constexpr int PROMPT_THREADS = 384;  // 2 softmax warpgroups, 1 of fetch + issue
constexpr unsigned SITE_ATTN = 9;    // wait sites SITE_ATTN .. SITE_ATTN + 5

template <int D>
struct PromptSmem {
  static constexpr int TILE = 128 * D * 2;                // bytes of a Q, K or V tile
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int RING = 2 * TILE;
  static constexpr int OUT = RING + STAGES * TILE;        // a softmax warp's 32 result rows, 64 elements after 64
  static constexpr int BARS = OUT + 8 * 4096;
  static constexpr int N_BARS = 2 * STAGES + 18;
  static constexpr int INFO = BARS + 8 * N_BARS;
  static constexpr int MISC = INFO + 2 * 48;
  static constexpr int TAKE = (MISC + 16 + 15) / 16 * 16; // two 16-byte answers to try_cancel
  static constexpr int TOTAL = TAKE + 32 + 1024;          // + alignment of the first tile
};

// One unit of work as the fetching warp announces it.
struct PromptUnit {
  int tok0, ntok;  // first query row of the unit (token) and its tokens
  int k0, lk;      // the sequence's keys
  int lim0;        // keys the first token sees (causal; may be negative)
  int head0;       // first query head
  int nheads;      // query heads of the unit
  int kvh;
  int n[2];        // half key tiles of the two row tiles; n[0] = -1: no more units
  int pad[2];
};
static_assert(sizeof(PromptUnit) == 48, "unit layout");

// ---------------------------------------------------------------- tcgen05 pieces
// Shared-memory descriptors are kept as their low words (address, and for an
// operand whose N elements are contiguous the distance of the next 64 of them)
// beside one constant high word (8-row groups 1024 bytes apart, version 1,
// 128-byte swizzle): the issuing thread has few registers, and a spilled
// descriptor costs more than the product it feeds.
constexpr uint32_t DESC_HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t kmajor_desc(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t mnmajor_desc(uint32_t saddr, uint32_t next64) {
  return ((saddr & 0x3FFFFu) >> 4) | ((next64 >> 4) << 16);
}

// Products are issued by a warp's elected lane, four to a statement.
//
// D[tmem] (+)= A[smem] * B[smem]^T over 64 elements (128 bytes) of a K-major
// line: 128 x N x 64 bf16.
__device__ __forceinline__ void mma_ss_x4(uint32_t d_tmem, uint32_t adesc, uint32_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 a, b, a1, b1, a2, b2, a3, b3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "add.s64 a1, a, 2;\n\tadd.s64 b1, b, 2;\n\t"
      "add.s64 a2, a, 4;\n\tadd.s64 b2, b, 4;\n\t"
      "add.s64 a3, a, 6;\n\tadd.s64 b3, b, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(adesc), "r"(bdesc), "r"(idesc), "r"(accumulate), "r"(DESC_HIGH)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T over 64 keys (lines of 128 bytes, 16 to a
// product): 128 x N x 64 bf16.
__device__ __forceinline__ void mma_ts_x4(uint32_t d_tmem, uint32_t a_tmem, uint32_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 b, b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "add.s64 b1, b, 128;\n\tadd.s64 b2, b, 256;\n\tadd.s64 b3, b, 384;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(bdesc), "r"(idesc), "r"(accumulate), "r"(DESC_HIGH)
      : "memory");
}
// r[0..15] to columns col .. col+15 of this warp's lanes.
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
constexpr uint32_t IDESC_B_MN_MAJOR = 1u << 16;

// 3-D tiled store shared -> global (bulk-group completion).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// Asks for the next CTA of the grid that has not started; the 16-byte answer
// completes on `bar`.
__device__ __forceinline__ void take_next(uint32_t answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
               "r"(smem_addr(bar))
               : "memory");
}
// The index of the CTA taken over, or -1 if every one has started.
__device__ __forceinline__ int taken_index(uint32_t answer) {
  uint32_t x, got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %1, 1, 0, p;\n\tmov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "=r"(x), "=r"(got)
      : "r"(answer)
      : "memory");
  return got ? static_cast<int>(x) : -1;
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Bounded wait that starts its limit anew while a softmax warp of this CTA is
// recomputing rows (*busy != 0): that work is finite, but may be long.
__device__ __forceinline__ bool prompt_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                            volatile int* busy, unsigned site) {
  if (mbar_try_wait(bar, parity)) return true;
  long long start = clock64();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (*busy) {
        start = clock64();
      } else if (clock64() - start > WAIT_LIMIT_CYCLES) {
        report_error(ERR_WAIT_TIMEOUT | ((site & 0xFFu) << 8));
        *abort = 1;
        return false;
      }
    }
  }
}

// ---------------------------------------------------------------- units
// Up to 32 sequences of the pack, one per lane of the fetching warp.
struct PromptChunk {
  int first;              // index of lane 0's sequence
  int before;             // blocks of the sequences before it
  int q0, lq, k0, lk;     // this lane's sequence
  int sum;                // blocks of the chunk's sequences up to this lane's
  int blocks;             // of this lane's: of 2 * tile_tokens tokens
};

// Reads the chunk's offsets; a sequence whose offsets leave the tensors has no
// blocks (and is reported).
__device__ __forceinline__ void prompt_load(const PromptArgs& a, PromptChunk& c) {
  const int lane = threadIdx.x & 31, i = c.first + lane;
  c.q0 = c.lq = c.k0 = c.lk = c.blocks = 0;
  if (i < a.seqs) {
    const int q0 = a.cu_q[i], q1 = a.cu_q[i + 1], k0 = a.cu_k[i], k1 = a.cu_k[i + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.tokens || k0 < 0 || k1 < k0 || k1 > a.kv_tokens) {
      report_error(ERR_BAD_ARGUMENT);
    } else {
      c.q0 = q0, c.lq = q1 - q0, c.k0 = k0, c.lk = k1 - k0;
      c.blocks = (c.lq + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
    }
  }
  c.sum = c.blocks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, c.sum, o);
    if (lane >= o) c.sum += up;
  }
}

// Keys that token `i` of the unit sees.
__device__ __forceinline__ int prompt_limit(const PromptUnit& u, int causal, int i) {
  return causal ? max(0, min(u.lk, u.lim0 + i)) : u.lk;
}

// ---------------------------------------------------------------- the kernel
template <int D>
__global__ void __launch_bounds__(PROMPT_THREADS, 1)
prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const PromptArgs a) {
  using SM = PromptSmem<D>;
  constexpr int S = SM::STAGES;
  constexpr int HALVES = D / 64;         // 128-byte lines per row
  constexpr uint32_t TM_S = 0, TM_O = 256;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::BARS);
  uint64_t *kv_full = bars, *kv_empty = bars + S, *q_full = bars + 2 * S, *q_empty = q_full + 2,
           *s_full = q_full + 4, *p_full = q_full + 6, *o_done = q_full + 8, *info_full = q_full + 10,
           *info_empty = q_full + 12, *drain = q_full + 14, *p_rest = q_full + 15, *taken = q_full + 17;
  PromptUnit* info = reinterpret_cast<PromptUnit*>(smem + SM::INFO);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* busy = reinterpret_cast<volatile int*>(tmem_slot + 2);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);  // a tile's probabilities come in two halves
      mbar_init(&p_rest[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&info_full[i], 1);
      mbar_init(&info_empty[i], 9);  // the issuing warp and the eight softmax warps
    }
    mbar_init(drain, 1);
    mbar_init(taken, 1);
    *abort_flag = 0;
    *busy = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_o);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(D == 128 ? 72 : 64));
    if (warp == 8) {
      // ------------------------------------------------------ fetch
      // All offsets are read once to count the blocks; the chunk read last, the
      // one whose blocks come first, stays, and others follow as they come up.
      PromptChunk c;
      c.before = 0;
      int64_t counted = 0;
      for (c.first = 0;; c.first += 32) {
        prompt_load(a, c);
        const int n = __shfl_sync(0xFFFFFFFFu, c.sum, 31);
        counted += n;
        if (c.first + 32 >= a.seqs) break;
        c.before += n;
      }
      // sequences that do not overlap have no more blocks than the grid has room for
      const bool fits = counted * a.kv_heads * a.head_chunks <= gridDim.x;
      if (!fits && lane == 0) report_error(ERR_BAD_ARGUMENT);
      const int total = fits ? static_cast<int>(counted) : 0;
      const int heads = a.kv_heads * a.head_chunks;
      const int64_t units = static_cast<int64_t>(total) * heads;
      const int group = a.q_heads / a.kv_heads;
      uint32_t it = 0, q_use[2] = {0, 0}, n_info = 0;
      bool ok = true;
      const uint32_t answer = smem_addr(smem + SM::TAKE);
      uint32_t asked = 0;
      for (int64_t at = blockIdx.x; ok && at >= 0;) {
        if (at < units) {
        // the blocks with the most keys first, a block's heads side by side
        const int block = total - 1 - static_cast<int>(at / heads);
        const int head = static_cast<int>(at % heads);
        while (block < c.before) {
          c.first -= 32;
          prompt_load(a, c);
          c.before -= __shfl_sync(0xFFFFFFFFu, c.sum, 31);
        }
        for (int n = __shfl_sync(0xFFFFFFFFu, c.sum, 31); block >= c.before + n;) {
          c.before += n;
          c.first += 32;
          prompt_load(a, c);
          n = __shfl_sync(0xFFFFFFFFu, c.sum, 31);
        }
        const int l = __ffs(__ballot_sync(0xFFFFFFFFu, c.before + c.sum > block)) - 1;
        const int first = (block - c.before - __shfl_sync(0xFFFFFFFFu, c.sum - c.blocks, l)) * 2 * a.tile_tokens;
        const int lq = __shfl_sync(0xFFFFFFFFu, c.lq, l);
        PromptUnit u;
        u.kvh = head / a.head_chunks;
        const int chunk = head % a.head_chunks;
        u.head0 = u.kvh * group + chunk * a.tile_heads;
        u.nheads = min(a.tile_heads, group - chunk * a.tile_heads);
        u.tok0 = __shfl_sync(0xFFFFFFFFu, c.q0, l) + first;
        u.ntok = min(2 * a.tile_tokens, lq - first);
        u.k0 = __shfl_sync(0xFFFFFFFFu, c.k0, l);
        u.lk = __shfl_sync(0xFFFFFFFFu, c.lk, l);
        u.lim0 = first + 1 + u.lk - lq;
        u.n[0] = (prompt_limit(u, a.causal, min(u.ntok, a.tile_tokens) - 1) + PROMPT_HALF - 1) / PROMPT_HALF;
        u.n[1] = u.ntok > a.tile_tokens ? (prompt_limit(u, a.causal, u.ntok - 1) + PROMPT_HALF - 1) / PROMPT_HALF : 0;
        u.pad[0] = u.pad[1] = 0;
        if (lane == 0) {
          const uint32_t slot = n_info & 1u;
          ok = prompt_wait(&info_empty[slot], ((n_info >> 1) & 1u) ^ 1u, abort_flag, busy, SITE_ATTN);
          if (ok) {
            info[slot] = u;
            mbar_arrive(&info_full[slot]);
          }
          auto load_q = [&](int w) {
            if (!ok || u.n[w] == 0) return;
            ok = prompt_wait(&q_empty[w], (q_use[w] & 1u) ^ 1u, abort_flag, busy, SITE_ATTN);
            if (!ok) return;
            mbar_arrive_expect_tx(&q_full[w], a.tile_heads * a.tile_tokens * D * 2);
            for (int h = 0; h < HALVES; ++h)
              tma_load_3d(smem + w * SM::TILE + h * 16384, &tm_q, &q_full[w], h * 64, u.head0,
                          u.tok0 + w * a.tile_tokens);
            ++q_use[w];
          };
          auto load_kv = [&](const CUtensorMap* map, int j) {
            if (!ok) return;
            const uint32_t s = it % S;
            ok = prompt_wait(&kv_empty[s], ((it / S) & 1u) ^ 1u, abort_flag, busy, SITE_ATTN + 1);
            if (!ok) return;
            mbar_arrive_expect_tx(&kv_full[s], SM::TILE);
            for (int h = 0; h < HALVES; ++h)
              tma_load_3d(smem + SM::RING + s * SM::TILE + h * 16384, map, &kv_full[s], h * 64, u.kvh,
                          u.k0 + j * PROMPT_KEYS);
            ++it;
          };
          const int n = (max(u.n[0], u.n[1]) + 1) / 2;
          load_q(0);
          if (n > 0) load_kv(&tm_k, 0);
          load_q(1);
          for (int j = 0; j < n && ok; ++j) {
            load_kv(&tm_v, j);
            if (j + 1 < n) load_kv(&tm_k, j + 1);
          }
        }
        ++n_info;
        }
        // (asked only now: whoever asks early keeps others from a fair share)
        if (lane == 0 && ok) {
          mbar_arrive_expect_tx(taken, 16);
          take_next(answer + 16 * (asked & 1u), taken);
          ok = prompt_wait(taken, asked & 1u, abort_flag, busy, SITE_ATTN);
          if (!ok) {  // its answer may not land after the CTA has gone
            int never = 0;
            mbar_wait(taken, asked & 1u, &never, SITE_DRAIN);
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, static_cast<int>(ok), 0) != 0;
        at = ok ? taken_index(answer + 16 * (asked & 1u)) : -1;
        fence_proxy_async_smem();  // this answer is read before a later one is written
        __syncwarp();
        ++asked;
      }
      if (lane == 0) {
        if (ok && prompt_wait(&info_empty[n_info & 1u], ((n_info >> 1) & 1u) ^ 1u, abort_flag, busy, SITE_ATTN)) {
          info[n_info & 1u].n[0] = -1;
          mbar_arrive(&info_full[n_info & 1u]);
        }
        // no copy may still be landing in shared memory when the CTA exits
        int never = 0;
        for (uint32_t j = it > S ? it - S : 0u; j < it; ++j) mbar_wait(&kv_full[j % S], (j / S) & 1u, &never, SITE_DRAIN);
        for (int w = 0; w < 2; ++w)
          if (q_use[w]) mbar_wait(&q_full[w], (q_use[w] - 1) & 1u, &never, SITE_DRAIN);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------ matrix products
      // The whole warp walks through this together and one elected lane issues:
      // operands then come from uniform registers.  From inside a branch of one
      // lane the same eight products took 600 to 900 cycles to issue, longer
      // than they take to run.
      const uint32_t idesc_s = idesc_bf16_f32(128, 128);
      const uint32_t idesc_o = idesc_bf16_f32(128, D) | IDESC_B_MN_MAJOR;
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t qd = __shfl_sync(0xFFFFFFFFu, kmajor_desc(smem_addr(smem)), 0);
      const uint32_t kd = __shfl_sync(0xFFFFFFFFu, kmajor_desc(smem_addr(smem + SM::RING)), 0);
      const uint32_t vd = __shfl_sync(0xFFFFFFFFu, mnmajor_desc(smem_addr(smem + SM::RING), 16384), 0);
      // (all three inside an elected lane's branch)
      auto scores = [&](int w, uint32_t stage, bool last) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h)  // the second half of the rows is 16 KB on
          mma_ss_x4(tm + TM_S + w * 128, qd + w * (SM::TILE >> 4) + h * (16384 >> 4),
                    kd + stage * (SM::TILE >> 4) + h * (16384 >> 4), idesc_s, h > 0);
        mma_commit(&s_full[w]);
        if (last) mma_commit(&q_empty[w]);
      };
      auto values = [&](int w, uint32_t stage, int half, bool accumulate) {  // 64 keys
        mma_ts_x4(tm + TM_O + w * 128, tm + TM_S + w * 128 + half * 32, vd + stage * (SM::TILE >> 4) + half * (8192 >> 4),
                  idesc_o, accumulate);
      };
      auto release = [&](uint32_t stage) { mma_commit(&kv_empty[stage]); };
      // A wait that gives up has raised the abort flag, which the warp looks at
      // together, once in eight tiles: until then it issues on without harm, since a
      // product touches this CTA's own memory only.
      auto wait = [&](uint64_t* bar, uint32_t parity, unsigned site) { prompt_wait(bar, parity, abort_flag, busy, site); };
      auto going = [&]() -> bool { return __all_sync(0xFFFFFFFFu, *abort_flag == 0); };
      uint32_t stage = 0, phase = 0, q_use[2] = {0, 0}, p_use[2] = {0, 0}, rest_use[2] = {0, 0};
      auto advance = [&](uint32_t& st, uint32_t& ph) {
        if (++st == S) st = 0, ph ^= 1u;
      };
      for (uint32_t n_info = 0;; ++n_info) {
        wait(&info_full[n_info & 1u], (n_info >> 1) & 1u, SITE_ATTN + 2);
        if (!going()) break;
        const int n0 = __shfl_sync(0xFFFFFFFFu, info[n_info & 1u].n[0], 0);
        const int n1 = __shfl_sync(0xFFFFFFFFu, info[n_info & 1u].n[1], 0);
        if (n0 < 0) break;
        if (lane == 0) mbar_arrive(&info_empty[n_info & 1u]);
        __syncwarp();
        const int nh[2] = {n0, n1}, nw[2] = {(n0 + 1) / 2, (n1 + 1) / 2}, n = max(nw[0], nw[1]);
        if (n == 0) continue;
        wait(&kv_full[stage], phase, SITE_ATTN + 2);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (nw[w] == 0) continue;
          wait(&q_full[w], q_use[w] & 1u, SITE_ATTN + 2);
          ++q_use[w];
          tc_fence_after();
          if (elect_one()) scores(w, stage, nw[w] == 1);
        }
        if (elect_one()) release(stage);
        advance(stage, phase);
        int j = 0;
        bool here = false;  // this tile's copies have been seen to be in
        for (; j < n && ((j & 7) || going()); ++j) {
          uint32_t sk = stage, phase_k = phase;  // values at `stage`, the next keys behind them
          advance(sk, phase_k);
          if (!here) {
            wait(&kv_full[stage], phase, SITE_ATTN + 2);
            if (j + 1 < n) wait(&kv_full[sk], phase_k, SITE_ATTN + 2);
          }
          here = false;
          uint32_t sv = j + 1 < n ? sk : stage, phase_v = j + 1 < n ? phase_k : phase;  // the next tile's values
          advance(sv, phase_v);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (j < nw[w]) {
              wait(&p_full[w], p_use[w] & 1u, SITE_ATTN + 3);
              ++p_use[w];
              tc_fence_after();
              if (elect_one()) values(w, stage, 0, j > 0);
              if (2 * j + 2 > nh[w]) {  // a last tile's first half is all there is
                if (elect_one()) mma_commit(&o_done[w]);
              } else {
                wait(&p_rest[w], rest_use[w] & 1u, SITE_ATTN + 3);
                ++rest_use[w];
                tc_fence_after();
                if (elect_one()) {
                  values(w, stage, 1, true);
                  if (j + 1 < nw[w])
                    scores(w, sk, j + 2 == nw[w]);
                  else
                    mma_commit(&o_done[w]);
                }
              }
            }
            // a look at the next tile's copies while the other row tile is at work
            if (w == 0 && j + 1 < n) {
              here = mbar_try_wait(&kv_full[sv], phase_v);
              if (j + 2 < n) {
                uint32_t s2 = sv, phase_2 = phase_v;
                advance(s2, phase_2);
                here = mbar_try_wait(&kv_full[s2], phase_2) && here;
              }
            }
          }
          if (elect_one()) {
            release(stage);
            if (j + 1 < n) release(sk);
          }
          stage = sv, phase = phase_v;
        }
        if (j < n) break;
      }
      // every product issued must be complete before tensor memory is released
      if (elect_one()) {
        mma_commit(drain);
        int never = 0;
        mbar_wait(drain, 0u, &never, SITE_DRAIN);
      }
    }
  } else {
    // -------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(216));  // 2 x 216 + 72 <= 3 x 168
    const int w = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int tok = row / a.tile_heads, hd = row - tok * a.tile_heads;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + TM_S + w * 128, t_o = tmem + lanes + TM_O + w * 128;
    const float c = a.scale_log2, raise = 8.f / c;
    uint32_t s_use = 0, o_use = 0;  // score tiles and results taken so far
    for (uint32_t n_info = 0;; ++n_info) {
      if (!prompt_wait(&info_full[n_info & 1u], (n_info >> 1) & 1u, abort_flag, busy, SITE_ATTN + 4)) break;
      const PromptUnit& u = info[n_info & 1u];  // read where it is needed: registers are short
      if (u.n[0] < 0) break;
      const int n_halves = u.n[w], n_tiles = (n_halves + 1) / 2;
      const int i = w * a.tile_tokens + tok;  // token of the unit
      const bool valid = tok < a.tile_tokens && i < u.ntok && hd < u.nheads;
      // rows that are not stored mask nothing
      const int lim = valid ? prompt_limit(u, a.causal, i) : 1 << 30;
      const int warp_lim = __reduce_min_sync(0xFFFFFFFFu, lim);
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < n_tiles; ++j, ++s_use) {
        ok = prompt_wait(&s_full[w], s_use & 1u, abort_flag, busy, SITE_ATTN + 4);
        if (!ok) break;
        tc_fence_after();
        const bool whole = 2 * j + 2 <= n_halves;  // else half a tile; the same for the whole warpgroup
        uint32_t s[4][32];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld_32x32b_x32(t_s + 32 * x, s[x]);
        tmem_ld_wait();
        if ((j + 1) * PROMPT_KEYS > warp_lim) {
          const int rel = lim - j * PROMPT_KEYS, warp_rel = warp_lim - j * PROMPT_KEYS;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (32 * (x + 1) > warp_rel && (x < 2 || whole)) {
              // one bit per key that is seen
              const int seen = min(32, max(0, rel - 32 * x));
              const uint32_t bits = seen < 32 ? (1u << seen) - 1u : 0xFFFFFFFFu;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(bits & (1u << e))) s[x][e] = 0xFF800000u;  // -inf
            }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; e += 4)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            top[x] = max3(top[x], __uint_as_float(s[x / 2][e + 2 * (x % 2)]), __uint_as_float(s[x / 2][e + 2 * (x % 2) + 1]));
        if (whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              top[x] = max3(top[x], __uint_as_float(s[2 + x / 2][e + 2 * (x % 2)]), __uint_as_float(s[2 + x / 2][e + 2 * (x % 2) + 1]));
        }
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if (j == 0) {
          m = high;
        } else if (__any_sync(0xFFFFFFFFu, high > m + raise)) {
          const float m_new = high > m + raise ? high : m;
          const float f = m_new == m ? 1.f : ex2((m - m_new) * c);
          m = m_new;
          l *= f;
          // (the product before these scores is complete: they were issued after it)
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {  // (sixteen at a time: the scores stay in registers)
            uint32_t o[16];
            tmem_ld_x16(t_o + 16 * x, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st_x16(t_o + 16 * x, o);
          }
        }
        const float shift = m == -INFINITY ? 0.f : -m * c;
        const uint64_t c2 = pack2(c, c), shift2 = pack2(shift, shift);
        uint64_t sum2[2] = {0, 0};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (x >= 2 && !whole) break;
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint32_t* in = &s[x][2 * e];
            float lo, hi;
            unpack2(fma2(pack2(__uint_as_float(in[0]), __uint_as_float(in[1])), c2, shift2), lo, hi);
            lo = ex2(lo);
            hi = ex2(hi);
            sum2[e & 1] = add2(sum2[e & 1], pack2(lo, hi));
            p[e] = bf16x2(lo, hi);
          }
          tmem_st_x16(t_s + 16 * x, p);
          if (x & 1) {  // half of the keys: the product with their values may begin
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(x == 1 ? &p_full[w] : &p_rest[w]);
          }
        }
        float s0, s1;
        unpack2(add2(sum2[0], sum2[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      // ---- result
      // A thread holds a row; stored as they are, 32 rows at a time, the pieces
      // of a warp's store would lie in 32 lines, and the softmax would wait for
      // the stores.  So the warp lays its rows out in shared memory and one TMA
      // store takes them while the next unit runs.  A box cannot end between
      // tokens of two sequences: the last rows of a sequence, and groups that
      // do not divide 32, are stored from there in whole 128-byte lines.
      const unsigned stored = __ballot_sync(0xFFFFFFFFu, valid);
      const bool boxed = a.boxed && stored == 0xFFFFFFFFu;
      uint64_t nan2 = 0;
      if (n_tiles > 0) {
        if (!prompt_wait(&o_done[w], o_use++ & 1u, abort_flag, busy, SITE_ATTN + 5)) break;
        tc_fence_after();
      }
      const float inv = lim > 0 ? 1.f / l : 0.f;
      const uint64_t inv2 = pack2(inv, inv);
      uint8_t* lines = smem + SM::OUT + warp * 4096;
      const uint32_t mine = smem_addr(lines);
      const uint32_t out_off = static_cast<uint32_t>(i) * static_cast<uint32_t>(a.o_stride / 8) + hd * (D / 8);  // 16-byte pieces
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {  // 64 elements of every row
        if (lane == 0) bulk_wait_group_read<0>();  // the store before this one has left shared memory
        __syncwarp();
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t o[32];
          if (n_tiles > 0) {
            tmem_ld_32x32b_x32(t_o + 64 * x + 32 * y, o);
            tmem_ld_wait();
          }
          if (lim == 0) {  // sees nothing: zero, whatever the accumulator holds
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          uint32_t r[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float lo, hi;
            const uint64_t f = mul2(pack2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), inv2);
            nan2 = add2(nan2, f);
            unpack2(f, lo, hi);
            r[e] = bf16x2(lo, hi);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sts128(mine + lane * 128 + (((4 * y + e) ^ (lane & 7)) << 4), r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
        }
        if (boxed) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tm_o, lines, 64 * x, u.head0, u.tok0 + i);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          uint16_t* out = a.o + static_cast<int64_t>(u.tok0) * a.o_stride + static_cast<int64_t>(u.head0) * D;
#pragma unroll
          for (int y = 0; y < 8; ++y) {  // four rows at a time, eight lanes a row
            const int r = 4 * y + (lane >> 3);
            const uint4 v = lds128(mine + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            const uint32_t off = __shfl_sync(0xFFFFFFFFu, out_off, r);
            if ((stored >> r) & 1u) *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(off) + 8 * x + (lane & 7)) * 8) = v;
          }
        }
      }
      if (n_tiles > 0) tc_fence_before();
      // a sum of results is a NaN if one of them is (or if two are opposite
      // infinities: that row is then computed twice, to the same end)
      float n0, n1;
      unpack2(nan2, n0, n1);
      const bool bad = lim > 0 && n0 + n1 != n0 + n1;
      unsigned again = __ballot_sync(0xFFFFFFFFu, bad && valid);
      if (again) {
        if (lane == 0) {
          atomicAdd(const_cast<int*>(busy), 1);
          bulk_wait_group<0>();  // the rows are stored before they are stored again
        }
        __syncwarp();
        while (again) {
          const int r = __ffs(again) - 1;
          again &= again - 1;
          const int ri = __shfl_sync(0xFFFFFFFFu, i, r), rh = __shfl_sync(0xFFFFFFFFu, hd, r);
          const int64_t t = u.tok0 + ri;
          const int64_t h = static_cast<int64_t>(u.head0 + rh) * D, kh = static_cast<int64_t>(u.kvh) * D;
          attention_row<D>(a.q + t * a.q_stride + h, a.k + u.k0 * a.k_stride + kh, a.k_stride,
                           a.v + u.k0 * a.v_stride + kh, a.v_stride, prompt_limit(u, a.causal, ri), c,
                           a.o + t * a.o_stride + h);
        }
        __syncwarp();
        if (lane == 0) atomicSub(const_cast<int*>(busy), 1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&info_empty[n_info & 1u]);
    }
    if (lane == 0) bulk_wait_group<0>();
  }
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

}  // namespace convrot
