// Launch interface of multi-token attention for few query rows (validated arguments).
#pragma once

#include "extend.h"

namespace pkv {

// Query rows of a KV head, on average over the sequences, up to which it is taken.
constexpr int kFewRows = 8, kFewRowsCoded = 32;

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
