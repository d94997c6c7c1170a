// kernels_cache_attend_f32.cu -- the kernels of kernels_cache_attend.cuh for
// f32 caches, by the head width rounded up to 64, 128 or 256 and the query heads
// of a segment.
#include "kernels_cache_attend.cuh"

namespace fwpkm {

cudaError_t launch_cache_attend_f32(const AttendArgs &a, cudaStream_t st) {
  using namespace attend;
  const AttendShape s = attend_shape(FWPKM_F32, a.p.dim, a.group);
  if (a.p.dim <= 64)
    return s.heads == 4   ? launch<F32<64, 4>, 16, 6>(a, st)
           : s.heads == 8 ? launch<F32<64, 8>, 16, 6>(a, st)
                          : launch<F32<64, 16>, 8, 8>(a, st);
  if (a.p.dim <= 128)
    return s.heads == 4   ? launch<F32<128, 4>, 12, 4>(a, st)
           : s.heads == 8 ? launch<F32<128, 8>, 12, 4>(a, st)
                          : launch<F32<128, 16>, 8, 6>(a, st);
  return s.heads == 4 ? launch<F32<256, 4>, 8, 3>(a, st) : launch<F32<256, 8>, 8, 3>(a, st);
}

}  // namespace fwpkm
