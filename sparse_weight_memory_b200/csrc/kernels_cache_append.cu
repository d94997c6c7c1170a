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

constexpr int kMaxThreads = 512;
constexpr int kMaxRows = 8;  // rows of a CTA of k_append_few
// Items of a head, over all rows, from which k_append_many is the faster one: 128
// rows of 48 bf16 heads of 128 (1024 items) take 5.3 us with k_append_few and 6.3
// with it, 512 rows 8.5 and 6.4, 256 rows the same; 20 heads of 256 alike.  In fp32
// 256 rows of 48 heads of 128 are still 6.4 and 8.4, 512 rows 10.5 and 8.5.
constexpr int kManyThreads = 2048;
template <typename TI>
constexpr int kBatch = sizeof(TI) == 2 ? 6 : 3;  // heads that a thread of it loads at once
constexpr int kMaxPairs = FWPKM_CACHE_MAX_DIM / 2;

struct Eight {
  float x[8];
};
// Eight elements as they lie in memory.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load8(const T *p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
  return r;
}
__device__ __forceinline__ Eight unpack(const Raw<float> &r) {
  Eight e;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    e.x[4 * i] = __uint_as_float(r.w[i].x);
    e.x[4 * i + 1] = __uint_as_float(r.w[i].y);
    e.x[4 * i + 2] = __uint_as_float(r.w[i].z);
    e.x[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
  return e;
}
__device__ __forceinline__ Eight unpack(const Raw<__nv_bfloat16> &r) {
  const unsigned w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
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

// The place of row r.
__device__ Place find_place(const AppendArgs &a, int r) {
  Place pl{-1, -1};
  int b = r, after = 1;  // after: rows from r to the sequence's end
  int before = 0;
  if (a.starts) {
    if (r >= __ldg(a.starts + a.s.B)) return pl;
    int lo = 0, n = a.s.B;  // the last b with starts[b] <= r is among lo .. lo + n - 1
    while (n > 1) {
      const int half = n >> 1;
      if (__ldg(a.starts + lo + half) <= r) {
        lo += half;
        n -= half;
      } else {
        n = half;
      }
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
  if (bad && a.errors) atomicOr(a.errors, bad);
  return pl;
}

__device__ __forceinline__ void divide(Eight &e, float by) {
#pragma unroll
  for (int i = 0; i < 8; ++i) e.x[i] = __fdiv_rn(e.x[i], by);
}

// cos and sin of position p times frequency f, in turns reduced to [-1/2, 1/2]:
// 1 / (2 pi) in 64 bits.  FINE (where 32-bit elements come out): what 32 bits lose
// of the angle, up to 2^-25 of half a turn and as much as such an element's own
// rounding, turns the pair a little further, so that cos and sin are as accurate as
// 32 bits hold them, small ones included.  Beside the rounding of 16- and 8-bit
// elements (2^-9, 2^-4) it is nothing, and 256 tokens take 6.4 us without it, 7.6 with.
template <bool FINE>
__device__ __forceinline__ float2 turn_of(int p, float f) {
  const double t = (double)p * (double)f * 0.15915494309189533577, d = t - rint(t);
  float c, s;
  if (!FINE) {
    sincospif(2.f * (float)d, &s, &c);
    return make_float2(c, s);
  }
  const float hi = (float)(2. * d), lo = (float)(2. * d - hi) * 3.14159265358979f;
  sincospif(hi, &s, &c);
  return make_float2(fmaf(-s, lo, c), fmaf(c, lo, s));
}
template <typename TI, typename TC>
constexpr bool kFine = sizeof(TI) == 4 || sizeof(TC) == 4;
__device__ __forceinline__ void rotate(float &u, float &z, const float2 &w) {
  const float u0 = u;
  u = fmaf(u0, w.x, -z * w.y);
  z = fmaf(z, w.x, u0 * w.y);
}

// What a thread does of a row's head: two groups of 8 elements (one where their
// number is odd), in a head rotated by halves two that turn together.  With one
// group a thread behind the rotated elements, half the bytes were under way: 64
// of 256 elements rotated took 112 us where all 256 took 63.
struct Item {
  int c, c2;  // groups of 8; c2 may be -1
};
FWPKM_HD int lanes_of(const AppendArgs &a) { return (a.p.dim + 8) / 16; }
__device__ __forceinline__ Item item_of(const AppendArgs &a, int i, bool value) {
  const int half = value || a.pairs ? 0 : a.rotary / 16;  // groups of half the rotated elements
  if (i < half) return {i, i + half};
  const int c = i + half, c2 = c + lanes_of(a) - half;  // behind them
  return {c, c2 < a.p.dim / 8 ? c2 : -1};
}
// Heads of a row in the order queries, keys, values.
template <typename TI>
__device__ __forceinline__ const TI *head_of(const AppendArgs &a, int64_t row, int h) {
  const char *base = a.q + row * a.q_stride;
  if (h >= a.heads) {
    h -= a.heads;
    base = a.k + row * a.k_stride;
    if (h >= a.p.kv_heads) {
      h -= a.p.kv_heads;
      base = a.v + row * a.v_stride;
    }
  }
  return reinterpret_cast<const TI *>(base) + h * a.p.dim;
}
// Stores a finished item of head h.
template <typename TI, typename TC>
__device__ __forceinline__ void put(const AppendArgs &a, int64_t row, const Place &pl, int h,
                                    const Item &m, Eight &u, Eight &z) {
  if (h < a.heads) {
    if (pl.pos < 0) return;
    TI *dst = reinterpret_cast<TI *>(a.q_out + row * a.q_out_stride) + h * a.p.dim;
    store8(dst + m.c * 8, u);
    if (m.c2 >= 0) store8(dst + m.c2 * 8, z);
    return;
  }
  if (pl.off < 0) return;
  h -= a.heads;
  const bool value = h >= a.p.kv_heads;
  if (value) h -= a.p.kv_heads;
  const float *scale = value ? a.p.value_scale : a.p.key_scale;
  if (scale) {
    const float by = __ldg(scale + h);
    divide(u, by);
    if (m.c2 >= 0) divide(z, by);
  }
  TC *dst = reinterpret_cast<TC *>((value ? a.p.values : a.p.keys) + pl.off + h * a.p.head_stride);
  store8(dst + m.c * 8, u);
  if (m.c2 >= 0) store8(dst + m.c2 * 8, z);
}

// Few rows: a CTA to a row (or several small ones), a thread to an item of a
// head, the angles shared through shared memory.  What counts is the latency:
// the elements are loaded before the row's place is looked up.
template <typename TI, typename TC>
__global__ void __launch_bounds__(kMaxThreads)
    k_append_few(const __grid_constant__ AppendArgs a, int per_cta, int per_row) {
  __shared__ Place place[kMaxRows];
  __shared__ float2 turn[kMaxRows * kMaxPairs];  // (cos, sin) of each row's angles
  griddep_wait();
  griddep_launch();
  const int r0 = blockIdx.x * per_cta, rows = min(per_cta, a.rows - r0);
  const int lanes = lanes_of(a), half = a.rotary / 2;
  const int rotated = a.heads + a.p.kv_heads;
  bool first = true;
  for (int n = threadIdx.x;; n += blockDim.x) {
    const bool live = n < rows * per_row;
    const int row = n / per_row, it = n - row * per_row, h = it / lanes, i = it - h * lanes;
    Item m{0, -1};
    Raw<TI> x, y;
    if (live) {
      m = item_of(a, i, h >= rotated);
      const TI *src = head_of<TI>(a, r0 + row, h);
      x = load8(src + m.c * 8);
      if (m.c2 >= 0) y = load8(src + m.c2 * 8);
    }
    if (first) {
      if (threadIdx.x < rows) place[threadIdx.x] = find_place(a, r0 + threadIdx.x);
      __syncthreads();
      for (int j = threadIdx.x; j < rows * half; j += blockDim.x)
        turn[j] = turn_of<kFine<TI, TC>>(max(place[j / half].pos, 0), __ldg(a.freqs + j % half));
      __syncthreads();
      first = false;
    }
    if (!live) break;
    Eight u = unpack(x), z;
    if (m.c2 >= 0) z = unpack(y);
    if (h < rotated) {
      if (a.pairs) {
        if (m.c < a.rotary / 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            rotate(u.x[2 * e], u.x[2 * e + 1], turn[row * half + m.c * 4 + e]);
        if (m.c2 >= 0 && m.c2 < a.rotary / 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            rotate(z.x[2 * e], z.x[2 * e + 1], turn[row * half + m.c2 * 4 + e]);
      } else if (i < a.rotary / 16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate(u.x[e], z.x[e], turn[row * half + i * 8 + e]);
      }
    }
    put<TI, TC>(a, r0 + row, place[row], h, m, u, z);
  }
}

// Many rows: `splits` threads to an item of a row, each for every splits-th head.
// The angles are the same for all heads: they stay in registers, and no thread
// waits for another.  The splits of a row are neighbours, so that neighbouring
// heads are read and written at about the same time: in CTAs of their own, the
// same shares took 64 us instead of 50 at heads of 80.  19235 rows of 36 bf16
// heads of 128 (354 MB) take 64 us, 85% of the measured copy rate; with the angles
// in shared memory, shared by a CTA's threads behind barriers, they took 96.
template <typename TI, typename TC, bool PAIRS>
__global__ void __launch_bounds__(256, 2)
    k_append_many(const __grid_constant__ AppendArgs a, int splits) {
  griddep_wait();
  griddep_launch();
  const int lanes = lanes_of(a);
  const int64_t n = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int threads = lanes * splits;  // of a row
  if (n >= (int64_t)a.rows * threads) return;
  const int row = (int)(n / threads), split = (int)(n - (int64_t)row * threads) / lanes;
  const int i = (int)(n - (int64_t)row * threads) - split * lanes;
  const int all = a.heads + 2 * a.p.kv_heads, rotated = a.heads + a.p.kv_heads;
  const Item turned = item_of(a, i, false), copied = item_of(a, i, true);
  Raw<TI> x[kBatch<TI>], y[kBatch<TI>];
  auto load = [&](int h0) {
#pragma unroll
    for (int j = 0; j < kBatch<TI>; ++j) {
      const int h = h0 + j * splits;
      if (h >= all) break;
      const Item m = h < rotated ? turned : copied;
      const TI *src = head_of<TI>(a, row, h);
      x[j] = load8(src + m.c * 8);
      if (m.c2 >= 0) y[j] = load8(src + m.c2 * 8);
    }
  };
  int h0 = split;
  load(h0);
  const Place pl = find_place(a, row);
  // by halves: angles 8 i .. of both groups; by pairs: 4 of each group's own
  const bool turns = PAIRS ? turned.c < a.rotary / 8 : i < a.rotary / 16;
  const bool turns2 = PAIRS && turned.c2 >= 0 && turned.c2 < a.rotary / 8;
  float2 w[8];
  if (turns)
#pragma unroll
    for (int e = 0; e < (PAIRS ? 4 : 8); ++e)
      w[e] = turn_of<kFine<TI, TC>>(max(pl.pos, 0), __ldg(a.freqs + i * (PAIRS ? 4 : 8) + e));
  if (turns2)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[4 + e] = turn_of<kFine<TI, TC>>(max(pl.pos, 0), __ldg(a.freqs + turned.c2 * 4 + e));
  while (true) {
#pragma unroll
    for (int j = 0; j < kBatch<TI>; ++j) {
      const int h = h0 + j * splits;
      if (h >= all) break;
      const Item m = h < rotated ? turned : copied;
      Eight u = unpack(x[j]), z;
      if (m.c2 >= 0) z = unpack(y[j]);
      if (h < rotated && turns) {
#pragma unroll
        for (int e = 0; e < (PAIRS ? 4 : 8); ++e) {
          if (PAIRS) rotate(u.x[2 * (e % 4)], u.x[2 * (e % 4) + 1], w[e]);
          else rotate(u.x[e], z.x[e], w[e]);
        }
      }
      if (PAIRS && h < rotated && turns2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) rotate(z.x[2 * e], z.x[2 * e + 1], w[4 + e]);
      }
      put<TI, TC>(a, row, pl, h, m, u, z);
    }
    h0 += kBatch<TI> * splits;
    if (h0 >= all) break;
    load(h0);
  }
}

template <typename TI, typename TC>
cudaError_t launch(const AppendArgs &a, cudaStream_t st) {
  const int lanes = lanes_of(a), all = a.heads + 2 * a.p.kv_heads;
  const int64_t threads = (int64_t)a.rows * lanes;
  if (threads >= kManyThreads) {
    // the splits of the heads that take the least time: rounds of two CTAs an
    // SM, times the heads of a split and what its angles cost beside them; two
    // at the least where each has a batch of heads (19235 rows of 36 heads of 80:
    // 60 us with one, 50 with two; of 3 heads of 128: 12.5 and 18.7)
    auto ctas = [&](int n) { return (threads * n + 255) / 256; };
    int splits = 1;
    int64_t best = INT64_MAX;
    for (int n = all >= 2 * kBatch<TI> ? 2 : 1; n <= all && n <= 64; ++n) {
      const int64_t time = (ctas(n) + 295) / 296 * ((all + n - 1) / n + 8);
      if (time < best) {
        best = time;
        splits = n;
      }
    }
    const dim3 grid((unsigned)ctas(splits));
    return a.pairs ? launch_k(true, k_append_many<TI, TC, true>, grid, dim3(256), 0, st, a, splits)
                   : launch_k(true, k_append_many<TI, TC, false>, grid, dim3(256), 0, st, a, splits);
  }
  const int per_row = all * lanes;
  int per_cta = 256 / per_row;  // rows of a CTA, where a row has few items
  per_cta = per_cta < 1 ? 1 : per_cta > kMaxRows ? kMaxRows : per_cta;
  // as many threads as even rounds over the items take
  const int items = per_cta * per_row, rounds = (items + kMaxThreads - 1) / kMaxThreads;
  int size = ((items + rounds - 1) / rounds + 31) / 32 * 32;
  if (size < 64) size = 64;
  return launch_k(true, k_append_few<TI, TC>, dim3((a.rows + per_cta - 1) / per_cta), dim3(size), 0,
                  st, a, per_cta, per_row);
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
