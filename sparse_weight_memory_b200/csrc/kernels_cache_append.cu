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
constexpr int kMaxBlock = 8;     // rows of a block
constexpr int kMaxChunk = 256;   // rows of a CTA
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

// What a thread does of a row: 8 elements of a head or, in a head rotated by
// halves, two groups of 8 that turn together.
struct Item {
  bool is_q, is_v;
  int head, c, c2;  // c: group of 8; c2: its partner, or -1
};
__device__ __forceinline__ Item item_of(const AppendArgs &a, int it) {
  const int D8 = a.p.dim / 8, H8 = a.rotary / 16;
  const int turned = a.pairs ? D8 : D8 - H8;  // items of a query or key head
  const int qk = (a.heads + a.p.kv_heads) * turned;
  Item m;
  m.is_v = it >= qk;
  m.is_q = false;
  m.c2 = -1;
  if (m.is_v) {
    m.head = (it - qk) / D8;
    m.c = (it - qk) - m.head * D8;
  } else {
    m.head = it / turned;
    m.c = it - m.head * turned;
    m.is_q = m.head < a.heads;  // queries first
    if (!m.is_q) m.head -= a.heads;
    if (!a.pairs) {
      if (m.c < H8) m.c2 = m.c + H8;
      else m.c += H8;  // behind the rotated elements
    }
  }
  return m;
}
int items_of_row(const AppendArgs &a) {
  const int D8 = a.p.dim / 8, H8 = a.rotary / 16;
  return (a.heads + a.p.kv_heads) * (a.pairs ? D8 : D8 - H8) + a.p.kv_heads * D8;
}

// A CTA takes `chunk` consecutive rows in blocks of groups x ROWS, a thread the
// same items of ROWS rows of a block.  Finding where a row goes takes dependent
// loads: a thread to a row, all of the CTA's rows at once.  In the loop a
// block's elements are loaded, all rows' at once, before the next block's angles
// are computed, so the memory is busy meanwhile.
template <typename TI, typename TC, int ROWS>
__global__ void __launch_bounds__(kMaxThreads, 2)
    k_append(const __grid_constant__ AppendArgs a, int chunk, int per_row, int groups,
             int per_group) {
  __shared__ Place place[kMaxChunk];
  __shared__ float2 turn[2][kMaxBlock * kMaxPairs];  // (cos, sin) of a block's angles
  griddep_wait();
  griddep_launch();
  const int r0 = blockIdx.x * chunk, rows = min(chunk, a.rows - r0);
  const int block = groups * ROWS, half = a.rotary / 2;
  const int group = threadIdx.x / per_group, it0 = threadIdx.x - group * per_group;
  for (int i = threadIdx.x; i < rows; i += blockDim.x) place[i] = find_place(a, r0 + i);
  __syncthreads();
  auto angles = [&](int b0) {
    const int n = min(block, rows - b0) * half;
    float2 *to = turn[b0 / block & 1];
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int row = i / half, j = i - row * half;
      // in turns, reduced to [-1/2, 1/2]: 1 / (2 pi) in 64 bits
      const double t = (double)max(place[b0 + row].pos, 0) * (double)__ldg(a.freqs + j) *
                       0.15915494309189533577;
      float sn, cs;
      sincospif(2.f * (float)(t - rint(t)), &sn, &cs);
      to[i] = make_float2(cs, sn);
    }
  };
  angles(0);
  for (int b0 = 0; b0 < rows; b0 += block) {
    const float2 *at = turn[b0 / block & 1];
    bool first = true;
    for (int it = it0;; it += per_group) {
      const bool live = group < groups && it < per_row;
      Item m{};
      Raw<TI> x[ROWS], y[ROWS];
      if (live) {
        m = item_of(a, it);
        const char *base = m.is_v ? a.v : m.is_q ? a.q : a.k;
        const int64_t stride = m.is_v ? a.v_stride : m.is_q ? a.q_stride : a.k_stride;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
          const int row = b0 + group + j * groups;
          if (row >= rows) continue;
          const TI *src =
              reinterpret_cast<const TI *>(base + (r0 + row) * stride) + m.head * a.p.dim;
          x[j] = load8(src + m.c * 8);
          if (m.c2 >= 0) y[j] = load8(src + m.c2 * 8);
        }
      }
      if (first) {
        __syncthreads();  // this block's angles are there, the last block's are used
        if (b0 + block < rows) angles(b0 + block);
        first = false;
      }
      if (!live) break;
      const float *scale = m.is_q ? nullptr : m.is_v ? a.p.value_scale : a.p.key_scale;
      const float by = scale ? __ldg(scale + m.head) : 1.f;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const int row = group + j * groups;
        if (b0 + row >= rows) continue;
        const Place pl = place[b0 + row];
        if (m.is_q ? pl.pos < 0 : pl.off < 0) continue;
        Eight u = unpack(x[j]), z;
        if (m.c2 >= 0) {
          z = unpack(y[j]);
          const float4 *t = reinterpret_cast<const float4 *>(at + row * half + m.c * 8);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float4 w = t[e / 2];
            const float u0 = u.x[e], z0 = z.x[e], u1 = u.x[e + 1], z1 = z.x[e + 1];
            u.x[e] = u0 * w.x - z0 * w.y;
            z.x[e] = z0 * w.x + u0 * w.y;
            u.x[e + 1] = u1 * w.z - z1 * w.w;
            z.x[e + 1] = z1 * w.z + u1 * w.w;
          }
        } else if (!m.is_v && a.pairs && m.c < a.rotary / 8) {
          const float2 *t = at + row * half + m.c * 4;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 w = t[e];
            const float u0 = u.x[2 * e], z0 = u.x[2 * e + 1];
            u.x[2 * e] = u0 * w.x - z0 * w.y;
            u.x[2 * e + 1] = z0 * w.x + u0 * w.y;
          }
        }
        if (m.is_q) {
          TI *dst = reinterpret_cast<TI *>(a.q_out + (r0 + b0 + row) * a.q_out_stride) +
                    m.head * a.p.dim;
          store8(dst + m.c * 8, u);
          if (m.c2 >= 0) store8(dst + m.c2 * 8, z);
        } else {
          if (scale) {
            divide(u, by);
            if (m.c2 >= 0) divide(z, by);
          }
          TC *dst = reinterpret_cast<TC *>((m.is_v ? a.p.values : a.p.keys) + pl.off +
                                           m.head * a.p.head_stride);
          store8(dst + m.c * 8, u);
          if (m.c2 >= 0) store8(dst + m.c2 * 8, z);
        }
      }
    }
  }
}

template <typename TI, typename TC, int ROWS>
cudaError_t launch_rows(const AppendArgs &a, cudaStream_t st) {
  const int per_row = items_of_row(a);
  int groups = 256 / per_row;  // rows side by side, where a row has few items
  groups = groups < 1 ? 1 : groups * ROWS > kMaxBlock ? kMaxBlock / ROWS : groups;
  // as many threads a row as even rounds over its items take
  const int rounds = (per_row + kMaxThreads - 1) / kMaxThreads;
  const int per_group = (per_row + rounds - 1) / rounds, block = groups * ROWS;
  int threads = (groups * per_group + 31) / 32 * 32;
  if (threads < 64) threads = 64;
  // one wave of CTAs, in whole blocks
  const int wave = 148 * (1024 / threads < 2 ? 2 : 1024 / threads);
  int chunk = (a.rows + wave - 1) / wave;
  chunk = (chunk + block - 1) / block * block;
  if (chunk > kMaxChunk) chunk = kMaxChunk / block * block;
  return launch_k(true, k_append<TI, TC, ROWS>, dim3((a.rows + chunk - 1) / chunk), dim3(threads),
                  0, st, a, chunk, per_row, groups, per_group);
}

// Several rows a thread keep the memory busy (as many as 32 registers of raw
// elements hold); with fewer rows than would fill the SMs so, one.
template <typename TI, typename TC>
cudaError_t launch(const AppendArgs &a, cudaStream_t st) {
  constexpr int kRows = sizeof(TI) == 2 ? 4 : 2;
  return a.rows >= kRows * 296 ? launch_rows<TI, TC, kRows>(a, st) : launch_rows<TI, TC, 1>(a, st);
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
