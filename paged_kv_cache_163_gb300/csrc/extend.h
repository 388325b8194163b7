// Launch interface of the multi-token attention kernels (validated arguments).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"

namespace pkv {

constexpr int kExtRows = 256;      // query rows (token, head of the group) of an item: two 128-row tiles
constexpr int kExtMaxGroup = 16;   // query heads per KV head

struct ExtendParams {
  uint8_t *out;
  int32_t out_f32;  // 1: out is float32, 0: out has the query's 16-bit type
  const uint8_t *q;
  const uint8_t *k_cache;
  const uint8_t *v_cache;
  const float *k_scale;
  const float *v_scale;
  const int32_t *block_tables;
  const int32_t *context_lens;
  const int32_t *query_starts;
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t num_queries;   // rows of q and out
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group_shift;   // log2 of query heads per KV head
  int32_t num_blocks;
  int32_t block_size;
  int32_t tiles_per_block;
  int32_t window;        // 0: none
  int32_t sinks;
  float scale_log2;      // |scale| * log2(e)
  int32_t negate;        // 1: scale is negative
  uint32_t *ws_ctr;      // [grid] pieces stored of the item that CTA leaves unfinished; zero between calls
  float *ws_ml;          // [2 * grid][kExtRows][2] partial (max, sum), base-2 domain
  float *ws_o;           // [2 * grid][head_dim / 4][kExtRows][4] partial unnormalised outputs
  int32_t *d_error;
  cudaStream_t stream;
};

// Launch on `grid` CTAs.  tmq maps q as [queries][q heads][head_dim]; tmk,
// tmv the pools as rows of head_dim elements (16-bit caches only).
using ExtendFn = cudaError_t (*)(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                                 const CUtensorMap &tmv, int grid);
#define PKV_EXTEND_DECL(SUF)                                                                                    \
  cudaError_t extend_call_##SUF##_d64(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,    \
                                      const CUtensorMap &tmv, int grid);                                        \
  cudaError_t extend_call_##SUF##_d128(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,   \
                                       const CUtensorMap &tmv, int grid);
PKV_EXTEND_DECL(f16)
PKV_EXTEND_DECL(bf16)
PKV_EXTEND_DECL(e4m3_f16)
PKV_EXTEND_DECL(e4m3_bf16)
PKV_EXTEND_DECL(e5m2_f16)
PKV_EXTEND_DECL(e5m2_bf16)
PKV_EXTEND_DECL(int8_f16)
PKV_EXTEND_DECL(int8_bf16)
PKV_EXTEND_DECL(e4m3i4_f16)
PKV_EXTEND_DECL(e4m3i4_bf16)
#undef PKV_EXTEND_DECL

}  // namespace pkv
