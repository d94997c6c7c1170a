// kernels_cache_attend_f32.cu -- the kernels of kernels_cache_attend.cuh for
// f32 caches, by the head width rounded up to 64, 128 or 256.
#include "kernels_cache_attend.cuh"

namespace fwpkm {

cudaError_t launch_cache_attend_f32(const AttendArgs &a, cudaStream_t st) {
  switch (attend_shape(FWPKM_F32, a.p.dim).dp) {
    case 64: return attend::launch<attend::F32<64, 8>, float, 8, 4>(a, st);
    case 128: return attend::launch<attend::F32<128, 8>, float, 4, 4>(a, st);
    default: return attend::launch<attend::F32<256, 8>, float, 4, 2>(a, st);
  }
}

}  // namespace fwpkm
