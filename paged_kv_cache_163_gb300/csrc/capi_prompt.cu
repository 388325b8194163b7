// C ABI of the calls that fill, read back and attend the cache for many tokens
// of a sequence: argument validation and launch.  Kernels live in rope.cu,
// gather.cu and extend*.cu.
#include <cmath>
#include <string>

#include "capi_common.h"
#include "dtypes.h"
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

}  // extern "C"
