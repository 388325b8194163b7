// Multi-token attention instances: cache INT8, query F16.
#include "extend.cuh"

namespace pkv {

cudaError_t extend_call_int8_f16_d64(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                                  const CUtensorMap &tmv, int grid) {
  return launch_extend<64, PKV_INT8, PKV_F16>(p, tmq, tmk, tmv, grid);
}

cudaError_t extend_call_int8_f16_d128(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                                   const CUtensorMap &tmv, int grid) {
  return launch_extend<128, PKV_INT8, PKV_F16>(p, tmq, tmk, tmv, grid);
}

}  // namespace pkv
