// Host side of the attention entry points: validation and launches.
// Included by convrot_abi.cu, whose helpers it uses.
#pragma once

#include "append.cuh"
#include "attn_decode.cuh"
#include "attn_prompt.cuh"

namespace {

constexpr int kMaxHeads = 1024;
constexpr int kMaxPage = 4096;

// Heads, head size and a row stride (elements) of a [rows, heads, D] tensor.
bool heads_ok(int q_heads, int kv_heads) {
  return q_heads > 0 && kv_heads > 0 && q_heads <= kMaxHeads && q_heads % kv_heads == 0;
}
constexpr int64_t kMaxStride = 1 << 26;  // offsets inside a tile's rows stay below 2^32
bool stride_ok(int64_t stride, int heads, int D, int rows) {
  return stride % 8 == 0 && stride <= kMaxStride && (rows <= 1 || stride >= static_cast<int64_t>(heads) * D);
}

// A tensor's memory: rows of `width` bytes, `stride` bytes apart.
struct Rows {
  uintptr_t at;
  int64_t stride, width, rows;
  uintptr_t end() const { return at + static_cast<uintptr_t>((rows - 1) * stride + width); }
};
Rows head_rows(const void* p, int64_t stride, int heads, int D, int rows) {
  const int64_t width = static_cast<int64_t>(heads) * D * 2;
  return {reinterpret_cast<uintptr_t>(p), rows > 1 ? stride * 2 : width, width, p ? rows : 0};
}
Rows piece(const void* p, int64_t bytes) { return {reinterpret_cast<uintptr_t>(p), bytes, bytes, p && bytes > 0 ? 1 : 0}; }

// Whether two tensors share a byte.  Column views of one buffer lie between one
// another's rows and share none.
bool overlap(const Rows& a, const Rows& b) {
  if (a.rows == 0 || b.rows == 0 || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  const int64_t apart = static_cast<int64_t>(b.at - a.at);
  if (a.rows == 1 || b.rows == 1 || a.stride == b.stride) {
    // rows i and j meet where -b.width < apart + (j - i) stride < a.width
    const int64_t stride = a.rows > 1 ? a.stride : b.stride, low = -b.width - apart;
    int64_t k = low / stride - (low % stride < 0 ? 1 : 0) + 1;  // the first k with low < k stride
    k = std::max(k, -(a.rows - 1));
    return k <= b.rows - 1 && apart + k * stride < a.width;
  }
  for (int64_t i = 0, j = 0; i < a.rows && j < b.rows;) {
    const int64_t x = i * a.stride, y = apart + j * b.stride;
    if (x + a.width <= y)
      ++i;
    else if (y + b.width <= x)
      ++j;
    else
      return true;
  }
  return false;
}
// The one way in which a result may lie on an input: in its place.
bool in_place(const Rows& a, const Rows& b) { return a.at == b.at && a.stride == b.stride && a.width == b.width; }

convrot_status run_append(const AppendArgs& args, int D, bool int8, cudaStream_t st) {
  const DeviceInfo d = current_device();
  if (d.device < 0 || d.sms <= 0) return CONVROT_ERR_CUDA;
  AppendArgs a = args;
  const int lanes = D / 16, groups = ((a.q_heads + 2 * a.kv_heads) * lanes + 31) / 32;
  // warps per token: one where the tokens alone fill the GPU (splitting them
  // further there measured 12 % slower), else up to one per row group (a single
  // token's rows then load side by side)
  const int64_t want = static_cast<int64_t>(d.sms) * 32;
  a.parts = static_cast<int>(std::min<int64_t>(groups, std::max<int64_t>(1, want / a.tokens)));
  const int64_t warps = static_cast<int64_t>(a.tokens) * a.parts;
  const unsigned blocks = static_cast<unsigned>((warps + APPEND_WARPS - 1) / APPEND_WARPS);
  auto k = D == 128 ? (int8 ? append_kernel<128, true> : append_kernel<128, false>)
                    : (int8 ? append_kernel<64, true> : append_kernel<64, false>);
  return launch_pdl(k, dim3(blocks), dim3(32 * APPEND_WARPS), 0, st, 1, a);
}

// bf16 head rows as a 3-D map (element, head, row) with boxes of 64 elements,
// `box_heads` heads and `box_rows` rows, 128-byte swizzle.
bool make_heads_map(CUtensorMap* map, const void* base, int rows, int heads, int D, int64_t stride, int box_heads,
                    int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
convrot_status run_prompt(const PromptArgs& args, cudaStream_t st) {
  PromptArgs a = args;
  const DeviceInfo d = current_device();
  if (d.device < 0 || d.sms <= 0) return CONVROT_ERR_CUDA;
  const int group = a.q_heads / a.kv_heads;
  a.head_chunks = (group + 127) / 128;
  a.tile_heads = (group + a.head_chunks - 1) / a.head_chunks;
  a.tile_tokens = 128 / a.tile_heads;
  a.boxed = 32 % a.tile_heads == 0;
  CUtensorMap mq, mk, mv, mo;
  if (!make_heads_map(&mq, a.q, a.tokens, a.q_heads, D, a.q_stride, a.tile_heads, a.tile_tokens))
    return CONVROT_ERR_CUDA;
  mk = mv = mo = mq;  // without keys nothing is fetched through them
  if (a.boxed && !make_heads_map(&mo, a.o, a.tokens, a.q_heads, D, a.o_stride, a.tile_heads, 32 / a.tile_heads))
    return CONVROT_ERR_CUDA;
  if (a.kv_tokens > 0 && (!make_heads_map(&mk, a.k, a.kv_tokens, a.kv_heads, D, a.k_stride, 1, PROMPT_KEYS) ||
                          !make_heads_map(&mv, a.v, a.kv_tokens, a.kv_heads, D, a.v_stride, 1, PROMPT_KEYS)))
    return CONVROT_ERR_CUDA;
  auto k = prompt_kernel<D>;
  constexpr int smem = PromptSmem<D>::TOTAL;
  static std::atomic<bool> configured[64];
  if (!configured[d.device].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return CONVROT_ERR_CUDA;
    configured[d.device].store(true, std::memory_order_release);
  }
  // the lengths are on the device: at most this many units
  const int64_t units = (static_cast<int64_t>(a.tokens) / (2 * a.tile_tokens) + std::min(a.seqs, a.tokens)) *
                        a.kv_heads * a.head_chunks;
  if (units > 0x7FFFFFFF) return CONVROT_ERR_SHAPE;
  const unsigned grid = static_cast<unsigned>(units);
  return launch_pdl(k, dim3(grid), dim3(PROMPT_THREADS), smem, st, 1, mq, mk, mv, mo, a);
}

// Heads of a decode unit: a group of up to sixteen together, else sixteen at a time.
int decode_unit_heads(int q_heads, int kv_heads) { return std::min(q_heads / kv_heads, 16); }

constexpr int kDecodeCtas = 2;  // most CTAs per SM of any decode kernel

int decode_grid(const DeviceInfo& d) { return std::min(kDecodeCtas * d.sms, 1024); }

constexpr size_t kDecodeCounterBytes = 4096;  // a fixed region of counters at offset 0, one per CTA

size_t decode_ws_bytes(int grid, int heads, int D) {
  return kDecodeCounterBytes + static_cast<size_t>(grid) * 2 * decode_part_floats(heads, D) * sizeof(float);
}

// A paged cache as a 3-D map (bytes or elements of a line, row, line of the
// row): lines of 128 bytes (64 where a row is no longer), rows of all pages
// and heads one after another.
bool make_cache_map(CUtensorMap* map, const void* base, int64_t rows, int D, bool int8, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int esz = int8 ? 1 : 2, line = D * esz >= 128 ? 128 : 64, halves = D * esz / line;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(line / esz), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(halves)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * esz, static_cast<cuuint64_t>(line)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(line / esz), static_cast<cuuint32_t>(box_rows),
                             static_cast<cuuint32_t>(halves)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, int8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool I8, int NQ>
convrot_status run_decode(const DecodeArgs& args, const void* k_cache, const void* v_cache, int64_t blocks,
                          cudaStream_t st) {
  using SM = DecodeSmem<D, I8, NQ>;
  static_assert(SM::CTAS <= kDecodeCtas, "the workspace is sized for kDecodeCtas");
  constexpr int budget = 228 * 1024 / SM::CTAS - 1024;
  DecodeArgs a = args;
  const DeviceInfo d = current_device();
  const int64_t rows = std::max<int64_t>(1, static_cast<int64_t>(a.pages) * a.kv_heads * a.page_size);
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, k_cache, rows, D, I8, a.box_rows) || !make_cache_map(&mv, v_cache, rows, D, I8, a.box_rows))
    return CONVROT_ERR_CUDA;
  a.stages = DECODE_MAX_STAGES;
  while (a.stages > 2 && SM::total(a.stages, a.chunk_heads) > budget) --a.stages;
  const int smem = SM::total(a.stages, a.chunk_heads);
  auto k = decode_kernel<D, I8, NQ>;
  static std::atomic<bool> configured[64];
  if (!configured[d.device].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, budget) != cudaSuccess)
      return CONVROT_ERR_CUDA;
    configured[d.device].store(true, std::memory_order_release);
  }
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(std::min(SM::CTAS * d.sms, 1024), blocks));
  return launch_pdl(k, dim3(grid), dim3(DECODE_THREADS), smem, st, 1, mk, mv, a);
}

}  // namespace

extern "C" {

convrot_status convrot_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                   const void* v, int64_t v_stride, int tokens, int q_heads,
                                   int kv_heads, int head_dim, const float* rope, int rope_rows,
                                   int rope_dim, const int32_t* positions, const int64_t* slots,
                                   const float* q_norm, const float* k_norm, float eps, void* q_out,
                                   int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                   void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                   int pages, int page_size, convrot_stream_t stream) {
  if (tokens < 0 || !heads_ok(q_heads, kv_heads)) return CONVROT_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return CONVROT_ERR_UNSUPPORTED;
  if (tokens > (1 << 24) || pages < 0 || page_size < 1 || page_size > kMaxPage || page_size % 16)
    return CONVROT_ERR_SHAPE;
  if (rope_rows < 1 || rope_dim < 16 || rope_dim > head_dim || rope_dim % 16) return CONVROT_ERR_SHAPE;
  if ((q_norm || k_norm) && !(eps >= 0.f)) return CONVROT_ERR_SHAPE;
  if (!stride_ok(q_stride, q_heads, head_dim, tokens) || !stride_ok(k_stride, kv_heads, head_dim, tokens) ||
      !stride_ok(v_stride, kv_heads, head_dim, tokens) ||
      !stride_ok(q_out_stride, q_heads, head_dim, tokens) ||
      (k_out && !stride_ok(k_out_stride, kv_heads, head_dim, tokens)))
    return CONVROT_ERR_SHAPE;
  if (tokens == 0) return CONVROT_OK;
  if (!q || !k || !v || !rope || !positions || !slots || !q_out || !k_cache || !v_cache || !k_scale != !v_scale)
    return CONVROT_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(rope, 16) || !aligned(positions, 4) ||
      !aligned(slots, 8) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16) || !aligned(q_norm, 16) ||
      !aligned(k_norm, 16))
    return CONVROT_ERR_ALIGN;
  const Rows rq = head_rows(q, q_stride, q_heads, head_dim, tokens), rk = head_rows(k, k_stride, kv_heads, head_dim, tokens),
             rv = head_rows(v, v_stride, kv_heads, head_dim, tokens),
             rqo = head_rows(q_out, q_out_stride, q_heads, head_dim, tokens),
             rko = head_rows(k_out, k_out_stride, kv_heads, head_dim, tokens);
  if ((overlap(rqo, rq) && !in_place(rqo, rq)) || overlap(rqo, rk) || overlap(rqo, rv) || overlap(rqo, rko) ||
      (overlap(rko, rk) && !in_place(rko, rk)) || overlap(rko, rq) || overlap(rko, rv))
    return CONVROT_ERR_UNSUPPORTED;  // another warp may have yet to read what lies there
  const int64_t lines = static_cast<int64_t>(pages) * kv_heads * page_size;
  const int64_t bytes = lines * head_dim * (k_scale ? 1 : 2);
  if (overlap(piece(k_cache, bytes), piece(v_cache, bytes)) ||
      overlap(piece(k_scale, lines * 4), piece(v_scale, lines * 4)))
    return CONVROT_ERR_UNSUPPORTED;
  AppendArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.rope = rope;
  a.positions = positions;
  a.slots = slots;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.slot_end = static_cast<int64_t>(pages) * page_size;
  a.tokens = tokens;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.rope_rows = rope_rows;
  a.rope_dim = rope_dim;
  a.page_size = page_size;
  a.eps = eps;
  return run_append(a, head_dim, k_scale != nullptr, as_cuda(stream));
}

convrot_status convrot_attention_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                        const void* v, int64_t v_stride, int tokens, int kv_tokens,
                                        int q_heads, int kv_heads, int head_dim, const int32_t* cu_q,
                                        const int32_t* cu_k, int seqs, float scale, int causal, void* out,
                                        int64_t out_stride, convrot_stream_t stream) {
  if (tokens < 0 || kv_tokens < 0 || seqs < 0 || !heads_ok(q_heads, kv_heads)) return CONVROT_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return CONVROT_ERR_UNSUPPORTED;
  if (tokens > (1 << 24) || kv_tokens > (1 << 24) || seqs > (1 << 24)) return CONVROT_ERR_SHAPE;
  if (!(scale > 0.f) || !(scale * LOG2E < INFINITY)) return CONVROT_ERR_SHAPE;  // the kernels' scores are powers of two
  if (!stride_ok(q_stride, q_heads, head_dim, tokens) || !stride_ok(k_stride, kv_heads, head_dim, kv_tokens) ||
      !stride_ok(v_stride, kv_heads, head_dim, kv_tokens) || !stride_ok(out_stride, q_heads, head_dim, tokens))
    return CONVROT_ERR_SHAPE;
  if (tokens == 0 || seqs == 0) return CONVROT_OK;
  if (out == q || out == k || out == v) return CONVROT_ERR_UNSUPPORTED;  // q, k and v are read while out is written
  if (!q || !out || !cu_q || !cu_k || (kv_tokens > 0 && (!k || !v))) return CONVROT_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_q, 4) ||
      !aligned(cu_k, 4))
    return CONVROT_ERR_ALIGN;
  const Rows ro = head_rows(out, out_stride, q_heads, head_dim, tokens);
  if (overlap(ro, head_rows(q, q_stride, q_heads, head_dim, tokens)) ||
      overlap(ro, head_rows(k, k_stride, kv_heads, head_dim, kv_tokens)) ||
      overlap(ro, head_rows(v, v_stride, kv_heads, head_dim, kv_tokens)))
    return CONVROT_ERR_UNSUPPORTED;
  PromptArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.o_stride = out_stride;
  a.o = static_cast<uint16_t*>(out);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.tokens = tokens;
  a.kv_tokens = kv_tokens;
  a.seqs = seqs;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.scale_log2 = scale * LOG2E;
  a.causal = causal != 0;
  return head_dim == 128 ? run_prompt<128>(a, as_cuda(stream)) : run_prompt<64>(a, as_cuda(stream));
}

size_t convrot_attention_decode_workspace_bytes(int seqs, int q_heads, int kv_heads, int head_dim) {
  if (seqs <= 0 || !heads_ok(q_heads, kv_heads) || (head_dim != 64 && head_dim != 128)) return 0;
  const DeviceInfo d = current_device();
  if (d.device < 0 || d.sms <= 0) return 0;
  return decode_ws_bytes(decode_grid(d), decode_unit_heads(q_heads, kv_heads), head_dim);
}

convrot_status convrot_attention_decode(const void* q, int64_t q_stride, int seqs, int q_heads, int kv_heads,
                                        int head_dim, const void* k_cache, const void* v_cache,
                                        const float* k_scale, const float* v_scale, int pages, int page_size,
                                        const int32_t* table, int64_t table_stride, int table_cols,
                                        const int32_t* lens, float scale, void* out, int64_t out_stride,
                                        void* workspace, size_t workspace_bytes, convrot_stream_t stream) {
  if (seqs < 0 || !heads_ok(q_heads, kv_heads)) return CONVROT_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return CONVROT_ERR_UNSUPPORTED;
  if (seqs > (1 << 24) || pages < 0 || page_size < 1 || page_size > kMaxPage || page_size % 16 || table_cols < 0)
    return CONVROT_ERR_SHAPE;
  if (seqs > 1 && table_stride < table_cols) return CONVROT_ERR_SHAPE;
  if (!(scale > 0.f) || !(scale * LOG2E < INFINITY)) return CONVROT_ERR_SHAPE;  // the kernels' scores are powers of two
  if (!stride_ok(q_stride, q_heads, head_dim, seqs) || !stride_ok(out_stride, q_heads, head_dim, seqs))
    return CONVROT_ERR_SHAPE;
  if (seqs == 0) return CONVROT_OK;
  if (!q || !out || !lens || !k_scale != !v_scale) return CONVROT_ERR_NULL;
  if (!k_cache || !v_cache || (table_cols > 0 && !table)) return CONVROT_ERR_NULL;
  if (static_cast<int64_t>(pages) * kv_heads * page_size > 0x7FFFFFFF) return CONVROT_ERR_UNSUPPORTED;  // rows of a TMA map
  if (!aligned(workspace, 256) || !aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_scale, 16) || !aligned(v_scale, 16) || !aligned(table, 4) || !aligned(lens, 4))
    return CONVROT_ERR_ALIGN;
  // (a row's query is read before its result is written, by whichever CTA)
  const Rows rq = head_rows(q, q_stride, q_heads, head_dim, seqs), ro = head_rows(out, out_stride, q_heads, head_dim, seqs);
  if (overlap(ro, rq) && !in_place(ro, rq)) return CONVROT_ERR_UNSUPPORTED;
  DecodeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.o_stride = out_stride;
  a.o = static_cast<uint16_t*>(out);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = table;
  a.table_stride = table_stride;
  a.lens = lens;
  a.seqs = seqs;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.pages = pages;
  a.page_size = page_size;
  a.table_cols = table_cols;
  a.scale_log2 = scale * LOG2E;
  const DeviceInfo d = current_device();
  if (d.device < 0 || d.sms <= 0) return CONVROT_ERR_CUDA;
  const int group = q_heads / kv_heads;
  a.chunk_heads = decode_unit_heads(q_heads, kv_heads);
  a.chunks = (group + a.chunk_heads - 1) / a.chunk_heads;
  a.box_rows = page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : 16;
  const int grid = decode_grid(d);
  if (!workspace || workspace_bytes < decode_ws_bytes(grid, a.chunk_heads, head_dim)) return CONVROT_ERR_WORKSPACE;
  a.counters = static_cast<unsigned*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kDecodeCounterBytes);
  // no more CTAs than blocks there can be
  const int keys = k_scale ? DecodeSmem<128, true, 8>::KEYS : DecodeSmem<128, false, 8>::KEYS;
  const int64_t most = std::max<int64_t>(1, (static_cast<int64_t>(table_cols) * page_size + keys - 1) / keys);
  if (most > 0x7FFFFFFF / (static_cast<int64_t>(seqs) * kv_heads * a.chunks)) return CONVROT_ERR_UNSUPPORTED;
  const int64_t blocks = most * seqs * kv_heads * a.chunks;
  const bool i8 = k_scale != nullptr;
  const int h = a.chunk_heads;
  cudaStream_t st = as_cuda(stream);
#define CONVROT_DECODE(D, I8, NQ) run_decode<D, I8, NQ>(a, k_cache, v_cache, blocks, st)
  // heads of a unit: one 8-column tile takes eight (bf16) or four (int8, in
  // two columns each); fewer tiles take fewer registers and instructions
  if (head_dim == 128) {
    if (i8) return h > 8 ? CONVROT_DECODE(128, true, 16) : h > 4 ? CONVROT_DECODE(128, true, 8) : CONVROT_DECODE(128, true, 4);
    return h > 8 ? CONVROT_DECODE(128, false, 16) : CONVROT_DECODE(128, false, 8);
  }
  if (i8) return h > 8 ? CONVROT_DECODE(64, true, 16) : h > 4 ? CONVROT_DECODE(64, true, 8) : CONVROT_DECODE(64, true, 4);
  return h > 8 ? CONVROT_DECODE(64, false, 16) : CONVROT_DECODE(64, false, 8);
#undef CONVROT_DECODE
}

}  // extern "C"
