// kernels_cache_append.cu -- new keys and values into the pages of a cache.
//
// Per row (token): x_j = position * freqs[j]; each pair (a, b) of a rotated
// head becomes (a cos x_j - b sin x_j, b cos x_j + a sin x_j); keys and values
// go to the row's place in the pool, queries to q_out.  Every element is read
// and written once, so HBM bytes bound it.
//
// A position of a million times a frequency near 1 needs 20 bits before the
// binary point, which leaves 32-bit floats no accuracy behind it: the angle is
// formed in 64 bits, in turns, and only its fraction of a turn goes to 32.
#include <cuda_fp8.h>

#include "cache_schedule.cuh"
#include "fwpkm_cache_internal.cuh"

namespace fwpkm {
namespace {

constexpr int kMaxRowsPerCta = 8;
constexpr int kMaxPairs = FWPKM_CACHE_MAX_DIM / 2;

struct Eight {
  float x[8];
};
__device__ __forceinline__ Eight load8(const float *p) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  const float4 b = *reinterpret_cast<const float4 *>(p + 4);
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ Eight load8(const __nv_bfloat16 *p) {
  const uint4 raw = *reinterpret_cast<const uint4 *>(p);
  const unsigned w[4] = {raw.x, raw.y, raw.z, raw.w};
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e.x[2 * i] = __uint_as_float(w[i] << 16);
    e.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return e;
}
__device__ __forceinline__ void store8(float *p, const Eight &e) {
  *reinterpret_cast<float4 *>(p) = make_float4(e.x[0], e.x[1], e.x[2], e.x[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(e.x[4], e.x[5], e.x[6], e.x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Eight &e) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(e.x[2 * i], e.x[2 * i + 1]);
  *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(h);
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3 *p, const Eight &e) {
  __nv_fp8x2_storage_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(e.x[2 * i], e.x[2 * i + 1]), __NV_SATFINITE,
                                    __NV_E4M3);
  *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(h);
}

// Where a row goes: its sequence's page and the row in it (byte offset of
// cached head 0), or -1; and its position, or -1 for a row of no sequence.
struct Place {
  int64_t off;
  int pos;
};

// Warp-level: the place of row r.
__device__ Place find_place(const AppendArgs &a, int r) {
  const int lane = threadIdx.x & 31;
  Place pl{-1, -1};
  int b = r, after = 1;  // after: rows from r to the sequence's end
  int before = 0;
  if (a.starts) {
    if (r >= __ldg(a.starts + a.s.B)) return pl;
    // the last b with starts[b] <= r: 32 probes a step
    int lo = 0, n = a.s.B;  // among starts[lo .. lo + n - 1]
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int i = lane * step;
      const bool le = i < n && __ldg(a.starts + lo + i) <= r;
      const unsigned hits = __ballot_sync(FULL, le);
      const int last = hits ? 31 - __clz(hits) : 0;
      lo += last * step;
      n = min(step, n - last * step);
    }
    b = lo;
    before = r - __ldg(a.starts + b);
    after = __ldg(a.starts + b + 1) - r;
  }
  const int len = __ldg(a.s.lengths + b);
  if (!a.starts && len == 0) return pl;  // an empty place of a padded batch
  bool bad_len;
  pl.pos = append_position(len, before, after, a.s.table_width, a.p.page_size, bad_len);
  unsigned bad = bad_len ? FWPKM_CACHE_BAD_LENGTH : 0u;
  if (!bad_len) {
    const int page = __ldg(a.s.table + b * a.s.table_stride + pl.pos / a.p.page_size);
    if ((unsigned)page >= (unsigned)a.p.pages) bad = FWPKM_CACHE_BAD_PAGE;
    else
      pl.off = page * a.p.page_stride + (int64_t)(pl.pos % a.p.page_size) * a.p.row_stride;
  }
  if (bad && a.errors && lane == 0) atomicOr(a.errors, bad);
  return pl;
}

__device__ __forceinline__ void divide(Eight &e, float by) {
#pragma unroll
  for (int i = 0; i < 8; ++i) e.x[i] = __fdiv_rn(e.x[i], by);
}

// A CTA takes `per_cta` consecutive rows.  Its threads share out the row's
// items: an item is 8 elements of a head, or, in a head rotated by halves, two
// groups of 8 that turn together.
template <typename TI, typename TC>
__global__ void __launch_bounds__(512) k_append(const __grid_constant__ AppendArgs a, int per_cta) {
  __shared__ Place place[kMaxRowsPerCta];
  __shared__ float2 turn[kMaxRowsPerCta * kMaxPairs];  // (cos, sin) of each row's angles
  griddep_wait();
  griddep_launch();
  const int r0 = blockIdx.x * per_cta;
  const int nrows = min(per_cta, a.rows - r0);
  for (int i = threadIdx.x >> 5; i < nrows; i += blockDim.x >> 5) {
    const Place pl = find_place(a, r0 + i);
    if ((threadIdx.x & 31) == 0) place[i] = pl;
  }
  __syncthreads();
  const int half = a.rotary / 2;
  for (int i = threadIdx.x; i < nrows * half; i += blockDim.x) {
    const int row = i / half, j = i - row * half;
    // in turns, reduced to [-1/2, 1/2]: 1 / (2 pi) in 64 bits
    const double t = (double)max(place[row].pos, 0) * (double)__ldg(a.freqs + j) *
                     0.15915494309189533577;
    float sn, cs;
    sincospif(2.f * (float)(t - rint(t)), &sn, &cs);
    turn[row * half + j] = make_float2(cs, sn);
  }
  __syncthreads();

  const int D8 = a.p.dim / 8, R8 = a.rotary / 8, H8 = R8 / 2;
  const int turned = a.pairs ? D8 : D8 - H8;  // items of a query or key head
  const int qk = a.heads + a.p.kv_heads;      // of them the first a.heads are queries
  const int per_row = qk * turned + a.p.kv_heads * D8;
  for (int i = threadIdx.x; i < nrows * per_row; i += blockDim.x) {
    const int row = i / per_row;
    int it = i - row * per_row;
    const int r = r0 + row;
    const Place pl = place[row];
    int head, c;
    const TI *src;
    bool is_v = it >= qk * turned, is_q = false;
    if (is_v) {
      it -= qk * turned;
      head = it / D8;
      c = it - head * D8;
      src = reinterpret_cast<const TI *>(a.v + r * a.v_stride) + head * a.p.dim;
    } else {
      head = it / turned;
      c = it - head * turned;
      is_q = head < a.heads;
      if (!is_q) head -= a.heads;
      src = reinterpret_cast<const TI *>(is_q ? a.q + r * a.q_stride : a.k + r * a.k_stride) +
            head * a.p.dim;
    }
    if (is_q ? pl.pos < 0 : pl.off < 0) continue;
    int c2 = -1;  // the partner group of 8, in a head rotated by halves
    if (!is_v && !a.pairs) {
      if (c < H8) c2 = c + H8;
      else c += H8;  // behind the rotated elements
    }
    Eight x = load8(src + c * 8), y;
    if (c2 >= 0) {
      y = load8(src + c2 * 8);
      const float2 *t = turn + row * half + c * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 w = t[e];
        const float u = x.x[e], z = y.x[e];
        x.x[e] = u * w.x - z * w.y;
        y.x[e] = z * w.x + u * w.y;
      }
    } else if (!is_v && a.pairs && c < R8) {
      const float2 *t = turn + row * half + c * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 w = t[e];
        const float u = x.x[2 * e], z = x.x[2 * e + 1];
        x.x[2 * e] = u * w.x - z * w.y;
        x.x[2 * e + 1] = z * w.x + u * w.y;
      }
    }
    if (is_q) {
      TI *dst = reinterpret_cast<TI *>(a.q_out + r * a.q_out_stride) + head * a.p.dim;
      store8(dst + c * 8, x);
      if (c2 >= 0) store8(dst + c2 * 8, y);
    } else {
      const float *scale = is_v ? a.p.value_scale : a.p.key_scale;
      if (scale) {
        const float by = __ldg(scale + head);
        divide(x, by);
        if (c2 >= 0) divide(y, by);
      }
      TC *dst = reinterpret_cast<TC *>((is_v ? a.p.values : a.p.keys) + pl.off +
                                       head * a.p.head_stride);
      store8(dst + c * 8, x);
      if (c2 >= 0) store8(dst + c2 * 8, y);
    }
  }
}

template <typename TI, typename TC>
cudaError_t launch(const AppendArgs &a, cudaStream_t st) {
  const int D8 = a.p.dim / 8, H8 = a.rotary / 16;
  const int per_row = (a.heads + a.p.kv_heads) * (a.pairs ? D8 : D8 - H8) + a.p.kv_heads * D8;
  int per_cta = 256 / per_row;
  per_cta = per_cta < 1 ? 1 : per_cta > kMaxRowsPerCta ? kMaxRowsPerCta : per_cta;
  // as many threads as even rounds over the items take
  const int items = per_cta * per_row, rounds = (items + 383) / 384;
  int threads = ((items + rounds - 1) / rounds + 31) / 32 * 32;
  if (threads < 64) threads = 64;
  const int grid = (a.rows + per_cta - 1) / per_cta;
  return launch_k(true, k_append<TI, TC>, dim3(grid), dim3(threads), 0, st, a, per_cta);
}

template <typename TI>
cudaError_t launch_in(const AppendArgs &a, int cache_dtype, cudaStream_t st) {
  switch (cache_dtype) {
    case FWPKM_F32: return launch<TI, float>(a, st);
    case FWPKM_BF16: return launch<TI, __nv_bfloat16>(a, st);
    default: return launch<TI, __nv_fp8_e4m3>(a, st);
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs &a, int in_dtype, int cache_dtype,
                                cudaStream_t st) {
  return in_dtype == FWPKM_F32 ? launch_in<float>(a, cache_dtype, st)
                               : launch_in<__nv_bfloat16>(a, cache_dtype, st);
}

}  // namespace fwpkm
