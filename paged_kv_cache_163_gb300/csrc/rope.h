// Launch interfaces of the rotary table and the rotating append (validated arguments).
#pragma once

#include <cuda_runtime.h>

#include "pkv.h"

namespace pkv {

// From this many tokens on, one CTA turns all rows of a token.
constexpr int kRopeFullTokens = 600;

struct RopeTable {
  int32_t scaling;  // pkv_rope_scaling
  double base, factor;
  double original_max, slow_turns, fast_turns;  // PKV_ROPE_BY_PARTS
  double magnitude;
};

struct AppendRopeArgs {
  uint8_t *q_out;
  const uint8_t *q, *k, *v;
  pkv_dtype in_dtype;
  int64_t q_stride, k_stride, v_stride;  // elements from one token's rows to the next's
  int32_t num_tokens, num_q_heads, num_kv_heads, head_dim;
  const float *cos_sin;
  int32_t max_positions, rot_dim, interleaved;
  const int32_t *positions, *slot_mapping;
  uint8_t *k_cache, *v_cache;
  pkv_dtype cache_dtype;
  float *k_scale, *v_scale;
  int32_t num_blocks, block_size;
  int32_t *d_error;
  cudaStream_t stream;
};

cudaError_t run_rope_table(float *table, int64_t max_positions, int32_t rot_dim, const RopeTable &t,
                           cudaStream_t stream);
cudaError_t run_append_rope(const AppendRopeArgs &a);

}  // namespace pkv
