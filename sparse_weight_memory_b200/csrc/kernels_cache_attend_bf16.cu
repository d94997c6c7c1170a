// kernels_cache_attend_bf16.cu -- the kernels of kernels_cache_attend.cuh for
// bf16 caches, by the head width rounded up to 64, 128 or 256.
#include "kernels_cache_attend.cuh"

namespace fwpkm {

cudaError_t launch_cache_attend_bf16(const AttendArgs &a, cudaStream_t st) {
  switch (attend_shape(FWPKM_BF16, a.p.dim).dp) {
    case 64: return attend::launch<attend::Bf16<64, 32>, __nv_bfloat16, 8, 3>(a, st);
    case 128: return attend::launch<attend::Bf16<128, 16>, __nv_bfloat16, 8, 3>(a, st);
    default: return attend::launch<attend::Bf16<256, 16>, __nv_bfloat16, 4, 3>(a, st);
  }
}

}  // namespace fwpkm
