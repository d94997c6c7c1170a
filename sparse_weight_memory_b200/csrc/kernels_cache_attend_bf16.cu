// kernels_cache_attend_bf16.cu -- the kernels of kernels_cache_attend.cuh for
// bf16 caches, by the head width rounded up to 64, 128 or 256 and the query heads
// of a segment.
#include "kernels_cache_attend.cuh"

namespace fwpkm {

cudaError_t launch_cache_attend_bf16(const AttendArgs &a, cudaStream_t st) {
  using namespace attend;
  const AttendShape s = attend_shape(FWPKM_BF16, a.p.dim, a.group);
  if (a.p.dim <= 64)
    return s.heads == 8    ? launch<Bf16<64, 32, 1>, 16, 3>(a, st)
           : s.heads == 16 ? launch<Bf16<64, 32, 2>, 12, 3>(a, st)
                           : launch<Bf16<64, 32, 4>, 8, 4>(a, st);
  if (a.p.dim <= 128)
    return s.heads == 8    ? launch<Bf16<128, 16, 1>, 12, 4>(a, st)
           : s.heads == 16 ? launch<Bf16<128, 16, 2>, 8, 6>(a, st)
                           : launch<Bf16<128, 16, 4>, 8, 4>(a, st);
  return s.heads == 8 ? launch<Bf16<256, 16, 1>, 8, 3>(a, st)
                      : launch<Bf16<256, 16, 2>, 8, 2>(a, st);
}

}  // namespace fwpkm
