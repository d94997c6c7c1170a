// kernels_cache_attend_e4m3.cu -- the kernels of kernels_cache_attend.cuh for
// e4m3 caches, by the head width rounded up to 64, 128 or 256 and the query heads
// of a segment.
#include "kernels_cache_attend.cuh"

namespace fwpkm {

cudaError_t launch_cache_attend_e4m3(const AttendArgs &a, cudaStream_t st) {
  using namespace attend;
  const AttendShape s = attend_shape(FWPKM_E4M3, a.p.dim, a.group);
  if (a.p.dim <= 64)
    return s.heads == 8    ? launch<E4m3<64, 32, 1>, 16, 5>(a, st)
           : s.heads == 16 ? launch<E4m3<64, 32, 2>, 12, 6>(a, st)
                           : launch<E4m3<64, 32, 4>, 8, 6>(a, st);
  if (a.p.dim <= 128)
    return s.heads == 8 ? launch<E4m3<128, 32, 1>, 8, 6>(a, st)
                        : launch<E4m3<128, 32, 2>, 8, 5>(a, st);
  return launch<E4m3<256, 16, 1>, 8, 6>(a, st);
}

}  // namespace fwpkm
