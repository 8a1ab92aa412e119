// k_attend_256.cu -- paged attention kernels of head_dim 256 (see attend_dev.cuh).
#include "attend_dev.cuh"

namespace sv {

cudaError_t prepare_attend_256() {
  cudaError_t e = attend_prepare<256, SV_KV_BF16>();
  return e != cudaSuccess ? e : attend_prepare<256, SV_KV_E4M3>();
}

cudaError_t launch_attend_256(const AttendParams& p, int fmt, int num_sms, cudaStream_t s, bool pdl) {
  return fmt == SV_KV_BF16 ? attend_launch<256, SV_KV_BF16>(p, num_sms, s, pdl)
                           : attend_launch<256, SV_KV_E4M3>(p, num_sms, s, pdl);
}

}  // namespace sv
