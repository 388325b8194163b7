// Launch interface of multi-token attention for few query rows (validated arguments).
#pragma once

#include "extend.h"

namespace pkv {

// Query rows of a KV head, on average over the sequences, up to which it is
// taken, over 16-bit and over coded caches.  Measured on 16 sequences of 1024
// and of 4096 tokens, 8 KV heads, head_dim 128, this kernel / the other, us:
//   8 rows   BF16 25 / 35 and 68 / 68       E4M3 19 / 56 and 42 / 115
//   32 rows  BF16 31 / 37 and 81 / 68       E4M3 31 / 62 and 70 / 133
//   64 rows  BF16 48 / 37 and 134 / 70      E4M3 50 / 62 and 130 / 138
// (16-bit caches, ragged lengths of 512 to 4096, 32 rows at most: 53 / 45; of
// 100 to 1000: 29 / 33; 64 tokens 15 / 21.)  So over 16-bit caches more than 8
// rows are taken only where the block tables reach no further than kFewReach tokens.
constexpr int kFewRows = 8, kFewRowsShort = 32, kFewRowsCoded = 64;
constexpr int kFewReach = 1024;

// rows: that average, rounded up.
using ExtendFewFn = cudaError_t (*)(const ExtendParams &p, int head_dim, int rows, int grid);
#define PKV_FEW_DECL(SUF) cudaError_t extend_few_##SUF(const ExtendParams &p, int head_dim, int rows, int grid);
PKV_FEW_DECL(f16)
PKV_FEW_DECL(bf16)
PKV_FEW_DECL(e4m3_f16)
PKV_FEW_DECL(e4m3_bf16)
PKV_FEW_DECL(e5m2_f16)
PKV_FEW_DECL(e5m2_bf16)
PKV_FEW_DECL(int8_f16)
PKV_FEW_DECL(int8_bf16)
PKV_FEW_DECL(e4m3i4_f16)
PKV_FEW_DECL(e4m3i4_bf16)
#undef PKV_FEW_DECL

}  // namespace pkv
