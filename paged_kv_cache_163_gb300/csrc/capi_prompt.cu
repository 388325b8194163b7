// C ABI of the calls that fill, read back and attend the cache for many tokens
// of a sequence: argument validation and launch.  Kernels live in rope.cu,
// gather.cu and extend*.cu.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <string>

#include "capi_common.h"
#include "dtypes.h"
#include "extend.h"
#include "extend_few.h"
#include "gather.h"
#include "pkv.h"
#include "rope.h"
#include "status.h"
#include "trace.h"

namespace pkv {
namespace {

// What every call over a paged cache asks of its pool; `where` names the call.
pkv_status check_pool(const char *where, const void *k_cache, const void *v_cache, pkv_dtype cache_dtype,
                      const float *k_scale, const float *v_scale, int32_t num_kv_heads, int32_t head_dim,
                      int32_t num_blocks, int32_t block_size) {
  auto say = [&](pkv_status s, const char *why) { return fail(s, (std::string(where) + ": " + why).c_str()); };
  if (num_kv_heads <= 0 || num_blocks <= 0) return say(PKV_ERR_INVALID, "bad sizes");
  if (block_size != PKV_BLOCK_SIZE && block_size != PKV_BLOCK_SIZE_32)
    return say(PKV_ERR_UNSUPPORTED, "block_size must be 16 or 32");
  if (head_dim != 64 && head_dim != 128) return say(PKV_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (!is_cache_type(cache_dtype)) return say(PKV_ERR_INVALID, "bad cache dtype");
  if (static_cast<int64_t>(num_blocks) * num_kv_heads * block_size >= (int64_t(1) << 31))
    return say(PKV_ERR_UNSUPPORTED, "pool larger than 2^31 token rows");
  if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache))
    return say(PKV_ERR_INVALID, "NULL or misaligned cache");
  if (has_scales(cache_dtype) && (!k_scale || !aligned16(k_scale) || v_scale != k_scale + block_size))
    return say(PKV_ERR_INVALID, "a coded cache needs an aligned k_scale, and v_scale = k_scale + block_size");
  return PKV_OK;
}

bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(b_bytes) && y < x + static_cast<uintptr_t>(a_bytes);
}

// The kernels of a pair of types, for many query rows and for few.
struct ExtendPair {
  ExtendFn many;
  ExtendFewFn few;
};
ExtendPair pick_extend(pkv_dtype q_dtype, pkv_dtype cache_dtype, int32_t head_dim) {
  const bool wide = head_dim == 128;
#define PKV_PICK(SUF) return {wide ? extend_call_##SUF##_d128 : extend_call_##SUF##_d64, extend_few_##SUF}
  if (cache_dtype == PKV_F16 && q_dtype == PKV_F16) PKV_PICK(f16);
  if (cache_dtype == PKV_BF16 && q_dtype == PKV_BF16) PKV_PICK(bf16);
  if (cache_dtype == PKV_FP8_E4M3 && q_dtype == PKV_F16) PKV_PICK(e4m3_f16);
  if (cache_dtype == PKV_FP8_E4M3 && q_dtype == PKV_BF16) PKV_PICK(e4m3_bf16);
  if (cache_dtype == PKV_FP8_E5M2 && q_dtype == PKV_F16) PKV_PICK(e5m2_f16);
  if (cache_dtype == PKV_FP8_E5M2 && q_dtype == PKV_BF16) PKV_PICK(e5m2_bf16);
  if (cache_dtype == PKV_INT8 && q_dtype == PKV_F16) PKV_PICK(int8_f16);
  if (cache_dtype == PKV_INT8 && q_dtype == PKV_BF16) PKV_PICK(int8_bf16);
  if (cache_dtype == PKV_FP8_E4M3_INT4 && q_dtype == PKV_F16) PKV_PICK(e4m3i4_f16);
  if (cache_dtype == PKV_FP8_E4M3_INT4 && q_dtype == PKV_BF16) PKV_PICK(e4m3i4_bf16);
#undef PKV_PICK
  return {nullptr, nullptr};
}

// Workspace of paged_attention_extend: a counter per CTA, then two partials per CTA.
struct ExtendLayout {
  int64_t ml_off, o_off, total;
};
ExtendLayout extend_layout(int sms, int32_t head_dim) {
  ExtendLayout l;
  l.ml_off = (static_cast<int64_t>(sms) * 4 + 255) / 256 * 256;
  l.o_off = l.ml_off + static_cast<int64_t>(sms) * 2 * kExtRows * 2 * 4;
  l.total = l.o_off + static_cast<int64_t>(sms) * 2 * kExtRows * head_dim * 4;
  return l;
}

// Map of 16-bit elements with 64-element boxes and the 128-byte swizzle:
// rank 2 [rows][head_dim] with boxes of 16 rows, or rank 3 [queries][heads]
// [head_dim] with boxes of `heads` x `tokens`.
pkv_status map_16bit(const void *base, int32_t head_dim, int64_t rows, int32_t box_heads, int64_t tokens,
                     int32_t box_tokens, CUtensorMap *out) {
  auto enc = tensor_map_encoder();
  if (!enc) return fail(PKV_ERR_CUDA, "paged_attention_extend: cuTensorMapEncodeTiled is unavailable");
  const bool three = box_tokens > 0;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2, static_cast<cuuint64_t>(head_dim) * 2 * rows};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t elem[3] = {1, 1, 1};
  CUresult r = enc(out, CU_TENSOR_MAP_DATA_TYPE_UINT16, three ? 3 : 2, const_cast<void *>(base), dims, strides, box,
                   elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "paged_attention_extend: cuTensorMapEncodeTiled rejected a layout");
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_rope_table(float *cos_sin, int32_t max_positions, int32_t rot_dim, double base,
                          pkv_rope_scaling scaling, double factor, int32_t original_max, double slow_turns,
                          double fast_turns, double magnitude, pkv_stream_t stream) {
  pkv::TraceRange trace("pkv.rope_table");
  if (max_positions < 0 || rot_dim < 16 || rot_dim > 128 || rot_dim % 16 != 0)
    return fail(PKV_ERR_INVALID, "pkv_rope_table: rot_dim must be a multiple of 16 in [16, 128]");
  if (scaling != PKV_ROPE_NONE && scaling != PKV_ROPE_LINEAR && scaling != PKV_ROPE_NTK &&
      scaling != PKV_ROPE_BY_PARTS)
    return fail(PKV_ERR_INVALID, "pkv_rope_table: unknown scaling");
  if (!(base > 1.0) || !std::isfinite(base) || !(magnitude >= 0.0) || !std::isfinite(magnitude))
    return fail(PKV_ERR_INVALID, "pkv_rope_table: base must exceed 1, magnitude must not be negative");
  if (scaling != PKV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(PKV_ERR_INVALID, "pkv_rope_table: factor must be at least 1");
  if (scaling == PKV_ROPE_BY_PARTS &&
      (original_max <= 0 || !(slow_turns < fast_turns) || !std::isfinite(slow_turns) || !std::isfinite(fast_turns)))
    return fail(PKV_ERR_INVALID, "pkv_rope_table: by parts needs original_max > 0 and slow_turns < fast_turns");
  if (max_positions == 0) return PKV_OK;
  if (!cos_sin || !aligned16(cos_sin)) return fail(PKV_ERR_INVALID, "pkv_rope_table: NULL or misaligned pointer");
  RopeTable t{};
  t.scaling = scaling;
  t.base = scaling == PKV_ROPE_NTK ? base * std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2)) : base;
  t.factor = scaling == PKV_ROPE_NONE ? 1.0 : factor;
  t.original_max = original_max;
  t.slow_turns = slow_turns;
  t.fast_turns = fast_turns;
  t.magnitude = magnitude > 0.0 ? magnitude : (scaling == PKV_ROPE_BY_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0);
  cudaError_t e = run_rope_table(cos_sin, max_positions, rot_dim, t, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "pkv_rope_table");
  add_launches(1);
  return PKV_OK;
}

pkv_status paged_kv_append_rope(void *q_out, const void *q, const void *k, const void *v, pkv_dtype in_dtype,
                                int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t num_tokens,
                                int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                const int32_t *positions, const int32_t *slot_mapping, const float *cos_sin,
                                int32_t max_positions, int32_t rot_dim, int32_t interleaved, void *k_cache,
                                void *v_cache, pkv_dtype cache_dtype, float *k_scale, float *v_scale,
                                int32_t num_blocks, int32_t block_size, int32_t *d_error, pkv_stream_t stream) {
  pkv::TraceRange trace("pkv.append_rope");
  if (num_tokens < 0 || num_q_heads < 0 || max_positions < 0)
    return fail(PKV_ERR_INVALID, "paged_kv_append_rope: bad sizes");
  if (in_dtype != PKV_F16 && in_dtype != PKV_BF16)
    return fail(PKV_ERR_INVALID, "paged_kv_append_rope: input rows must be F16 or BF16");
  pkv_status s = check_pool("paged_kv_append_rope", k_cache, v_cache, cache_dtype, k_scale, v_scale, num_kv_heads,
                            head_dim, num_blocks, block_size);
  if (s != PKV_OK) return s;
  if (!has_scales(cache_dtype) && cache_dtype != in_dtype)
    return fail(PKV_ERR_UNSUPPORTED, "paged_kv_append_rope: a 16-bit cache must match the input dtype");
  if (rot_dim < 16 || rot_dim > head_dim || rot_dim % 16 != 0)
    return fail(PKV_ERR_UNSUPPORTED, "paged_kv_append_rope: rot_dim must be a multiple of 16, at most head_dim");
  if (num_q_heads > (1 << 20) || num_kv_heads > (1 << 20))
    return fail(PKV_ERR_UNSUPPORTED, "paged_kv_append_rope: too many heads");
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if ((num_q_heads && (q_stride < q_row || q_stride % 8)) || k_stride < kv_row || k_stride % 8 || v_stride < kv_row ||
      v_stride % 8)
    return fail(PKV_ERR_INVALID,
                "paged_kv_append_rope: a token stride must be a multiple of 8 and cover the token's rows");
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !positions || !slot_mapping || !cos_sin || (num_q_heads && (!q || !q_out)) || !aligned16(k) ||
      !aligned16(v) || !aligned16(cos_sin) || (num_q_heads && (!aligned16(q) || !aligned16(q_out))))
    return fail(PKV_ERR_INVALID, "paged_kv_append_rope: NULL or misaligned pointer");
  if (num_q_heads) {
    const int64_t last = num_tokens - 1;
    const int64_t out_bytes = num_tokens * q_row * 2;
    const bool in_place = q_out == q && q_stride == q_row;
    if ((!in_place && overlap(q_out, out_bytes, q, (last * q_stride + q_row) * 2)) ||
        overlap(q_out, out_bytes, k, (last * k_stride + kv_row) * 2) ||
        overlap(q_out, out_bytes, v, (last * v_stride + kv_row) * 2))
      return fail(PKV_ERR_INVALID, "paged_kv_append_rope: q_out overlaps an input (only q_out = q, dense, may)");
  }
  AppendRopeArgs a{};
  a.q_out = static_cast<uint8_t *>(q_out);
  a.q = static_cast<const uint8_t *>(q);
  a.k = static_cast<const uint8_t *>(k);
  a.v = static_cast<const uint8_t *>(v);
  a.in_dtype = in_dtype;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.num_tokens = num_tokens;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.cos_sin = cos_sin;
  a.max_positions = max_positions;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved ? 1 : 0;
  a.positions = positions;
  a.slot_mapping = slot_mapping;
  a.k_cache = static_cast<uint8_t *>(k_cache);
  a.v_cache = static_cast<uint8_t *>(v_cache);
  a.cache_dtype = cache_dtype;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.d_error = d_error;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = run_append_rope(a);
  if (e != cudaSuccess) return cuda_fail(e, "paged_kv_append_rope");
  add_launches(1);
  return PKV_OK;
}

pkv_status paged_kv_gather(void *k_out, void *v_out, pkv_dtype out_dtype, int32_t num_rows, const void *k_cache,
                           const void *v_cache, pkv_dtype cache_dtype, const float *k_scale, const float *v_scale,
                           const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *token_starts,
                           const int32_t *context_lens, const int32_t *out_starts, int32_t num_seqs,
                           int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, int32_t block_size,
                           int32_t *d_error, pkv_stream_t stream) {
  pkv::TraceRange trace("pkv.gather");
  if (num_rows < 0 || max_blocks_per_seq < 0) return fail(PKV_ERR_INVALID, "paged_kv_gather: bad sizes");
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS_PER_CALL)
    return fail(PKV_ERR_UNSUPPORTED, "paged_kv_gather: num_seqs must be in [0, 1024]");
  pkv_status s = check_pool("paged_kv_gather", k_cache, v_cache, cache_dtype, k_scale, v_scale, num_kv_heads,
                            head_dim, num_blocks, block_size);
  if (s != PKV_OK) return s;
  if (out_dtype != PKV_F32 && out_dtype != PKV_F16 && out_dtype != PKV_BF16)
    return fail(PKV_ERR_INVALID, "paged_kv_gather: out_dtype must be F32, F16 or BF16");
  if (!has_scales(cache_dtype) && out_dtype != PKV_F32 && out_dtype != cache_dtype)
    return fail(PKV_ERR_UNSUPPORTED, "paged_kv_gather: a 16-bit cache is read back as its own type or F32");
  if (num_kv_heads > (1 << 20)) return fail(PKV_ERR_UNSUPPORTED, "paged_kv_gather: too many heads");
  if (num_rows == 0 || num_seqs == 0) return PKV_OK;
  if (!k_out || !v_out || !block_tables || !context_lens || !out_starts || !aligned16(k_out) || !aligned16(v_out))
    return fail(PKV_ERR_INVALID, "paged_kv_gather: NULL or misaligned pointer");
  GatherArgs a{};
  a.k_out = static_cast<uint8_t *>(k_out);
  a.v_out = static_cast<uint8_t *>(v_out);
  a.out_dtype = out_dtype;
  a.num_rows = num_rows;
  a.k_cache = static_cast<const uint8_t *>(k_cache);
  a.v_cache = static_cast<const uint8_t *>(v_cache);
  a.cache_dtype = cache_dtype;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_tables = block_tables;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.token_starts = token_starts;
  a.context_lens = context_lens;
  a.out_starts = out_starts;
  a.num_seqs = num_seqs;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.d_error = d_error;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = run_gather(a);
  if (e != cudaSuccess) return cuda_fail(e, "paged_kv_gather");
  add_launches(1);
  return PKV_OK;
}

pkv_status paged_attention_extend_workspace_bytes(int32_t head_dim, size_t *bytes) {
  if (!bytes) return fail(PKV_ERR_INVALID, "paged_attention_extend_workspace_bytes: NULL pointer");
  if (head_dim != 64 && head_dim != 128)
    return fail(PKV_ERR_UNSUPPORTED, "paged_attention_extend_workspace_bytes: head_dim must be 64 or 128");
  const int sms = sm_count();
  if (sms <= 0) return fail(PKV_ERR_CUDA, "paged_attention_extend_workspace_bytes: cannot query the SM count");
  *bytes = static_cast<size_t>(extend_layout(sms, head_dim).total);
  return PKV_OK;
}

pkv_status paged_attention_extend(void *out, pkv_dtype out_dtype, const void *q, pkv_dtype q_dtype,
                                  int32_t num_queries, const void *k_cache, const void *v_cache,
                                  pkv_dtype cache_dtype, const float *k_scale, const float *v_scale,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  const int32_t *context_lens, const int32_t *query_starts, int32_t num_seqs,
                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t num_blocks, int32_t block_size, float scale, int32_t window,
                                  int32_t sinks, void *workspace, size_t workspace_bytes, int32_t *d_error,
                                  pkv_stream_t stream) {
  pkv::TraceRange trace("pkv.extend");
  if (num_queries < 0 || max_blocks_per_seq < 0) return fail(PKV_ERR_INVALID, "paged_attention_extend: bad sizes");
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS_PER_CALL)
    return fail(PKV_ERR_UNSUPPORTED, "paged_attention_extend: num_seqs must be in [0, 1024]");
  pkv_status s = check_pool("paged_attention_extend", k_cache, v_cache, cache_dtype, k_scale, v_scale, num_kv_heads,
                            head_dim, num_blocks, block_size);
  if (s != PKV_OK) return s;
  if (num_q_heads <= 0 || num_q_heads % num_kv_heads != 0)
    return fail(PKV_ERR_INVALID, "paged_attention_extend: num_q_heads must be a positive multiple of num_kv_heads");
  const int32_t group = num_q_heads / num_kv_heads;
  if (group > kExtMaxGroup || (group & (group - 1)) != 0)
    return fail(PKV_ERR_UNSUPPORTED, "paged_attention_extend: query heads per KV head must be 1, 2, 4, 8 or 16");
  const ExtendPair fn = pick_extend(q_dtype, cache_dtype, head_dim);
  if (!fn.many) return fail(PKV_ERR_UNSUPPORTED, "paged_attention_extend: unsupported q / cache dtype pair");
  if (out_dtype != PKV_F32 && out_dtype != q_dtype)
    return fail(PKV_ERR_UNSUPPORTED, "paged_attention_extend: out_dtype must be F32 or q_dtype");
  if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID, "paged_attention_extend: scale must be finite");
  if (window < 0 || sinks < 0)
    return fail(PKV_ERR_INVALID, "paged_attention_extend: window and sinks must not be negative");
  if (static_cast<int64_t>(num_queries) * group >= (int64_t(1) << 30) || num_q_heads > (1 << 20) ||
      static_cast<int64_t>(max_blocks_per_seq) * block_size >= (int64_t(1) << 31) - 64)
    return fail(PKV_ERR_UNSUPPORTED, "paged_attention_extend: too many queries, heads or table entries");
  if (num_seqs == 0 || num_queries == 0) return PKV_OK;
  if (!out || !q || !block_tables || !context_lens || !query_starts || !workspace || !aligned16(out) ||
      !aligned16(q) || !aligned16(workspace))
    return fail(PKV_ERR_INVALID, "paged_attention_extend: NULL or misaligned pointer");
  const int64_t q_elems = static_cast<int64_t>(num_queries) * num_q_heads * head_dim;
  if (overlap(out, q_elems * (out_dtype == PKV_F32 ? 4 : 2), q, q_elems * 2))
    return fail(PKV_ERR_INVALID, "paged_attention_extend: out overlaps q");
  const int sms = sm_count();
  if (sms <= 0) return fail(PKV_ERR_CUDA, "paged_attention_extend: cannot query the SM count");
  const ExtendLayout lay = extend_layout(sms, head_dim);
  if (workspace_bytes < static_cast<size_t>(lay.total))
    return fail(PKV_ERR_WORKSPACE, "paged_attention_extend: workspace smaller than required");

  uint8_t *ws = static_cast<uint8_t *>(workspace);
  ExtendParams p{};
  p.out = static_cast<uint8_t *>(out);
  p.out_f32 = out_dtype == PKV_F32 ? 1 : 0;
  p.q = static_cast<const uint8_t *>(q);
  p.k_cache = static_cast<const uint8_t *>(k_cache);
  p.v_cache = static_cast<const uint8_t *>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_starts = query_starts;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.num_queries = num_queries;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  while ((1 << p.group_shift) < group) ++p.group_shift;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.tiles_per_block = block_size / PKV_BLOCK_SIZE;
  p.window = window;
  p.sinks = sinks;
  // never 0, so that an invisible token's score of minus infinity stays that
  p.scale_log2 = std::min(std::max(std::fabs(scale) * 1.4426950408889634f, FLT_MIN), FLT_MAX);
  p.negate = scale < 0.f ? 1 : 0;
  p.ws_ctr = reinterpret_cast<uint32_t *>(ws);
  p.ws_ml = reinterpret_cast<float *>(ws + lay.ml_off);
  p.ws_o = reinterpret_cast<float *>(ws + lay.o_off);
  p.d_error = d_error;
  p.stream = reinterpret_cast<cudaStream_t>(stream);

  // Query rows of a KV head, on average over the sequences: the kernel for few
  // rows is right for any number, but reads an item's cache once for each 8 or
  // 32 of them, where the other's tiles are 128 rows.
  const int64_t rows = (static_cast<int64_t>(num_queries) * group + num_seqs - 1) / num_seqs;
  const bool short_tables = static_cast<int64_t>(max_blocks_per_seq) * block_size <= kFewReach;
  if (rows <= (has_scales(cache_dtype) ? kFewRowsCoded : short_tables ? kFewRowsShort : kFewRows)) {
    cudaError_t few = fn.few(p, head_dim, static_cast<int>(rows), sms);
    if (few != cudaSuccess) return cuda_fail(few, "paged_attention_extend");
    add_launches(1);
    return PKV_OK;
  }
  CUtensorMap tmq, tmk{}, tmv{};
  s = map_16bit(q, head_dim, num_q_heads, group, num_queries, 128 / group, &tmq);
  if (s == PKV_OK && !has_scales(cache_dtype)) {
    const int64_t rows = static_cast<int64_t>(num_blocks) * num_kv_heads * block_size;
    s = map_16bit(k_cache, head_dim, rows, PKV_BLOCK_SIZE, 1, 0, &tmk);
    if (s == PKV_OK) s = map_16bit(v_cache, head_dim, rows, PKV_BLOCK_SIZE, 1, 0, &tmv);
  }
  if (s != PKV_OK) return s;
  cudaError_t e = fn.many(p, tmq, tmk, tmv, sms);
  if (e != cudaSuccess) return cuda_fail(e, "paged_attention_extend");
  add_launches(1);
  return PKV_OK;
}

}  // extern "C"
