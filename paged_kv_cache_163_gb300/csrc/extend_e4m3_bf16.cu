// Multi-token attention instances: cache FP8_E4M3, query BF16.
#include "extend.cuh"

namespace pkv {

cudaError_t extend_call_e4m3_bf16_d64(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                                  const CUtensorMap &tmv, int grid) {
  return launch_extend<64, PKV_FP8_E4M3, PKV_BF16>(p, tmq, tmk, tmv, grid);
}

cudaError_t extend_call_e4m3_bf16_d128(const ExtendParams &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                                   const CUtensorMap &tmv, int grid) {
  return launch_extend<128, PKV_FP8_E4M3, PKV_BF16>(p, tmq, tmk, tmv, grid);
}

}  // namespace pkv
