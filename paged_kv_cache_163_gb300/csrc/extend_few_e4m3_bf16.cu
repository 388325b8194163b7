// Attention of few new tokens, instances: cache FP8_E4M3, query BF16.
#include "extend_few.cuh"

namespace pkv {

cudaError_t extend_few_e4m3_bf16(const ExtendParams &p, int head_dim, int rows, int grid) {
  return extend_few_family<PKV_FP8_E4M3, PKV_BF16>(p, head_dim, rows, grid);
}

}  // namespace pkv
