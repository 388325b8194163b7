// Launch interface of the cache read-back (validated arguments).
#pragma once

#include <cuda_runtime.h>

#include "pkv.h"

namespace pkv {

struct GatherArgs {
  uint8_t *k_out, *v_out;
  pkv_dtype out_dtype;
  int32_t num_rows;
  const uint8_t *k_cache, *v_cache;
  pkv_dtype cache_dtype;
  const float *k_scale, *v_scale;
  const int32_t *block_tables;
  int32_t max_blocks_per_seq;
  const int32_t *token_starts;  // NULL: 0 for every sequence
  const int32_t *context_lens, *out_starts;
  int32_t num_seqs, num_kv_heads, head_dim, num_blocks, block_size;
  int32_t *d_error;
  cudaStream_t stream;
};

cudaError_t run_gather(const GatherArgs &a);

}  // namespace pkv
