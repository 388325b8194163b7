// Attention of few new tokens, instances: cache FP8_E4M3_INT4, query BF16.
#include "extend_few.cuh"

namespace pkv {

cudaError_t extend_few_e4m3i4_bf16(const ExtendParams &p, int head_dim, int rows, int grid) {
  return extend_few_family<PKV_FP8_E4M3_INT4, PKV_BF16>(p, head_dim, rows, grid);
}

}  // namespace pkv
