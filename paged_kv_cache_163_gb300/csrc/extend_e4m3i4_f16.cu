// Multi-token attention instances: cache FP8_E4M3_INT4, query F16.
#include "extend.cuh"

namespace pkv {

cudaError_t extend_call_e4m3i4_f16_d64(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                                  const CUtensorMap &tmv, int grid) {
  return launch_extend<64, PKV_FP8_E4M3_INT4, PKV_F16>(p, tmq, tmk, tmv, grid);
}

cudaError_t extend_call_e4m3i4_f16_d128(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                                   const CUtensorMap &tmv, int grid) {
  return launch_extend<128, PKV_FP8_E4M3_INT4, PKV_F16>(p, tmq, tmk, tmv, grid);
}

}  // namespace pkv
