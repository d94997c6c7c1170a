// fwpkm_cache_internal.cuh -- shared by the kernels of the paged key-value
// cache (include/fwpkm_cache.h) and their host side (fwpkm_cache.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/fwpkm_cache.h"
#include "cache_schedule.cuh"
#include "fwpkm_internal.cuh"

namespace fwpkm {

// The pool and the batch as the kernels take them (strides in bytes).
struct CachePool {
  char *keys, *values;
  int64_t page_stride, head_stride, row_stride;
  const float *key_scale, *value_scale;
  int pages, page_size, kv_heads, dim;
};
struct CacheBatch {
  const int32_t *table, *lengths;
  int64_t table_stride;
  int B, table_width;
};

struct AppendArgs {
  CachePool p;
  CacheBatch s;
  const char *k, *v, *q;
  char *q_out;
  int64_t k_stride, v_stride, q_stride, q_out_stride;  // bytes
  const int32_t *starts;
  const float *freqs;
  unsigned *errors;
  int rows, heads;  // heads: query heads (0 without queries)
  int rotary, pairs;
};
cudaError_t launch_cache_append(const AppendArgs &a, int in_dtype, int cache_dtype,
                                cudaStream_t st);

// Pieces are sized for the B200's 148 multiprocessors (a launch geometry: any
// other count would only be slower).
constexpr int kAttendCtas = 148;

// The variant for a cache type, head width and number of query heads to a
// cached head: warps of a CTA, query heads of a segment, floats of a part.
// launch_cache_attend_* take the same ones.
struct AttendShape {
  int warps, heads, part;
};
AttendShape attend_shape(int cache_dtype, int dim, int group);

struct AttendArgs {
  CachePool p;
  CacheBatch s;
  const char *q;
  int64_t q_stride;  // bytes
  char *out;
  float *lse;
  float *parts;  // [2 * warps][part] sums o of the segments' parts
  float2 *ml;    // [2 * warps][heads] their (m, l)
  int4 *tails;   // [CTAs][warps] (sequence, head * blocks + block, last warp, pieces of a CTA) of
                 // the segment whose first part is the warp's tail slot; last warp -1: none
  int4 *middles; // [CTAs] (.., last warp, first warp) of the one its first warp is inside of
  unsigned *errors;
  float scale_log2;  // scale * log2(e)
  int heads, group, blocks;  // group: query heads of a cached head, in `blocks` segments
  int window;
  int64_t tokens;  // no sequence has more visible ones
  int aligned;     // segments are short: none is divided between CTAs
  PageDiv div;  // by the page size
};
cudaError_t launch_cache_attend_bf16(const AttendArgs &a, cudaStream_t st);
cudaError_t launch_cache_attend_e4m3(const AttendArgs &a, cudaStream_t st);
cudaError_t launch_cache_attend_f32(const AttendArgs &a, cudaStream_t st);

}  // namespace fwpkm
