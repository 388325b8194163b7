// Attention of few new tokens, instances: cache FP8_E5M2, query F16.
#include "extend_few.cuh"

namespace pkv {

cudaError_t extend_few_e5m2_f16(const ExtendParams &p, int head_dim, int rows, int grid) {
  return extend_few_family<PKV_FP8_E5M2, PKV_F16>(p, head_dim, rows, grid);
}

}  // namespace pkv
