// Attention of few new tokens, instances: cache F16, query F16.
#include "extend_few.cuh"

namespace pkv {

cudaError_t extend_few_f16(const ExtendParams &p, int head_dim, int rows, int grid) {
  return extend_few_family<PKV_F16, PKV_F16>(p, head_dim, rows, grid);
}

}  // namespace pkv
