// kernels_cache_attend_e4m3.cu -- the kernels of kernels_cache_attend.cuh for
// e4m3 caches, by the head width rounded up to 64, 128 or 256.
#include "kernels_cache_attend.cuh"

namespace fwpkm {

cudaError_t launch_cache_attend_e4m3(const AttendArgs &a, cudaStream_t st) {
  switch (attend_shape(FWPKM_E4M3, a.p.dim).dp) {
    case 64: return attend::launch<attend::E4m3<64, 32>, __nv_bfloat16, 8, 4>(a, st);
    case 128: return attend::launch<attend::E4m3<128, 32>, __nv_bfloat16, 8, 3>(a, st);
    default: return attend::launch<attend::E4m3<256, 16>, __nv_bfloat16, 8, 3>(a, st);
  }
}

}  // namespace fwpkm
