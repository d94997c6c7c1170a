// kernels_cache_attend.cuh -- attention of one token of each sequence over a
// paged cache.  Per query row, over the visible tokens t in tiles:
//   m' = max(m, s_t),  l' = l 2^(m-m') + sum 2^(s_t-m'),
//   o' = o 2^(m-m') + sum 2^(s_t-m') v_t,      s_t = scale log2(e) q.k_t,
// and at the end out = o / l, lse = ln 2 (m + log2 l): one pass over the cache.
//
// Every cached byte is read once and takes only heads/kv_heads products, so
// HBM bandwidth bounds it (8 query heads to a cached bf16 head: 8 flops a byte,
// 52 TFLOP/s at the measured 6.55 TB/s).  What counts is that all SMs read all
// the time, whatever the lengths are:
//   - The line of all tiles is cut evenly over the warps (cache_schedule.cuh).
//   - A warp streams its piece through a ring of its own in shared memory
//     (cp.async, one tile a stage), across the ends of segments, and waits for
//     no other warp: the loop has no CTA barrier.
//   - A tile's products run on mma.sync with the 16 rows of its A operand
//     taken by the query heads that share the cached head.  The tcgen05 path
//     would need 64 or 128 rows; 16 already hold the work well under the time
//     that the bytes take.
// Parts of segments that a cut falls into go to the workspace and are joined
// by k_join; where a CTA's whole piece lies in one segment its warps join in
// shared memory first.
#pragma once
#include <cuda_fp16.h>

#include "cache_schedule.cuh"
#include "fwpkm_cache_internal.cuh"

namespace fwpkm {
namespace attend {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -__builtin_huge_valf();
// Fewer tiles than this are not worth a warp of their own.
constexpr int kLeastTiles = 2;

__device__ __forceinline__ void cp_async16(uint32_t dst, const char *src, bool ok) {
  const int n = ok ? 16 : 0;  // 0: nothing is read, zeros are written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(unsigned (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(unsigned (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const unsigned (&a)[4], unsigned b0,
                                         unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const unsigned (&a)[4], unsigned b0,
                                        unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const unsigned (&a)[4], unsigned b0,
                                         unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const unsigned *>(&h);
}
__device__ __forceinline__ unsigned pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const unsigned *>(&h);
}
// Two 8-bit floats (the low 16 bits of v) as two 16-bit ones, exactly.
__device__ __forceinline__ unsigned e4m3_f16(unsigned v) {
  unsigned d;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(d)
      : "r"(v));
  return d;
}
// x as two TF32 parts: the rest beyond them is under 2^-22 of x.
__device__ __forceinline__ void split_tf32(unsigned x, unsigned &hi, unsigned &lo) {
  hi = (x + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}

// ---------------------------------------------------------------------------
// Element types.  Each says how a tile of TT tokens turns into scores and how
// weights and the tile turn into outputs:
//   s[TT/8][4]  scores; thread (g = lane/4, t = lane%4) holds rows g, g + 8 and
//               tokens 8n + 2t, + 1, the accumulator layout of mma.m16n8
//   o[DP/8][4]  outputs in the same layout; element (n, c) of row g is head
//               element col(n) + c
// ---------------------------------------------------------------------------

// bf16: weights go in as two bf16 parts, so that rounding them costs nothing
// of the result's accuracy (one part alone would add an error of the size of
// the final rounding).  The second product is hidden behind the loads.
template <int DP_, int TT_>
struct Bf16 {
  static constexpr int DP = DP_, TT = TT_, ESZ = 2, PITCH = DP * 2 + 16, QSMEM = 0;
  static constexpr float kShift = 0.f;
  unsigned q[DP / 16][4];

  __device__ __forceinline__ void load_q(const char *qp, int rows, int dim, uint32_t) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = g + (i & 1) * 8, c = k * 16 + t * 2 + (i >> 1) * 8;
        q[k][i] = row < rows && c < dim
                      ? __ldg(reinterpret_cast<const unsigned *>(qp + ((int64_t)row * dim + c) * 2))
                      : 0u;
      }
  }
  __device__ __forceinline__ void scores(float (&s)[TT / 8][4], uint32_t ks, uint32_t) {
    const int l = threadIdx.x & 31;
    const uint32_t a0 = ks + ((l & 7) + (l >> 4) * 8) * PITCH + ((l >> 3) & 1) * 16;
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
#pragma unroll
      for (int n = 0; n < TT / 16; ++n) {
        unsigned b[4];
        ldsm4(b, a0 + n * 16 * PITCH + k * 32);
        mma_bf16(s[2 * n], q[k], b[0], b[1]);
        mma_bf16(s[2 * n + 1], q[k], b[2], b[3]);
      }
  }
  __device__ __forceinline__ void outputs(float (&o)[DP / 8][4], const float (&p)[TT / 8][4],
                                          uint32_t vs) {
    const int l = threadIdx.x & 31;
    const uint32_t a0 = vs + (l & 15) * PITCH + (l >> 4) * 16;
#pragma unroll
    for (int k = 0; k < TT / 16; ++k) {
      unsigned hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = p[2 * k + (i >> 1)][(i & 1) * 2], y = p[2 * k + (i >> 1)][(i & 1) * 2 + 1];
        hi[i] = pack_bf16(x, y);
        lo[i] = pack_bf16(x - __uint_as_float(hi[i] << 16),
                          y - __uint_as_float(hi[i] & 0xffff0000u));
      }
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        unsigned b[4];
        ldsm4t(b, a0 + k * 16 * PITCH + n * 32);
        mma_bf16(o[2 * n], hi, b[0], b[1]);
        mma_bf16(o[2 * n + 1], hi, b[2], b[3]);
        mma_bf16(o[2 * n], lo, b[0], b[1]);
        mma_bf16(o[2 * n + 1], lo, b[2], b[3]);
      }
    }
  }
  // f(row half, first column, values of two neighbouring columns)
  template <typename F>
  __device__ __forceinline__ static void each(const float (&o)[DP / 8][4], F &&f) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      f(0, n * 8 + t * 2, o[n][0], o[n][1]);
      f(1, n * 8 + t * 2, o[n][2], o[n][3]);
    }
  }
};

// e4m3: an 8-bit element is exact in 16-bit floats, so the products run on
// those.  A row of queries is scaled by a power of two so that its largest
// element lies in [1, 2): what a bf16 element then loses to the 16-bit range is
// under 2^-25 of the largest, no more than the 32-bit sum.  Weights are held
// 2^12 too large (kShift), which keeps all down to 2^-26 of the largest above
// the 16-bit format's smallest normal number; at 11 bits their rounding is an
// eighth of the result's.
// ldmatrix moves pairs of 8-bit elements: a lane gets 4 neighbouring elements
// of a token, taken as elements 2t, 2t+1, 2t+8, 2t+9 of the product's 16; the
// queries are loaded in the same order, the outputs come out in it.
template <int DP_, int TT_>
struct E4m3 {
  static constexpr int DP = DP_, TT = TT_, ESZ = 1, PITCH = DP + 16, QSMEM = 0;
  static constexpr float kShift = 12.f;
  unsigned q[DP / 16][4];

  float f0, f1;  // the powers of two taken out of rows g and g + 8
  __device__ __forceinline__ void load_q(const char *qp, int rows, int dim, uint32_t) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    float top[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = g + r * 8, c = k * 16 + t * 4;
        uint2 v = make_uint2(0u, 0u);
        if (row < rows && c < dim)
          v = __ldg(reinterpret_cast<const uint2 *>(qp + ((int64_t)row * dim + c) * 2));
        q[k][r] = v.x;
        q[k][2 + r] = v.y;
        const float m0 = fmaxf(fabsf(__uint_as_float(v.x << 16)),
                               fabsf(__uint_as_float(v.x & 0xffff0000u)));
        const float m1 = fmaxf(fabsf(__uint_as_float(v.y << 16)),
                               fabsf(__uint_as_float(v.y & 0xffff0000u)));
        top[r] = fmaxf(top[r], fmaxf(m0, m1));
      }
    float down[2], up[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 2));
      // 2^-e and 2^e, e the exponent of the largest element kept where both
      // are normal numbers (a row of zeros, or one with infinities: 1)
      int e = (int)((__float_as_uint(top[r]) >> 23) & 255u);
      e = e == 0 || e == 255 ? 127 : e < 2 ? 2 : e > 252 ? 252 : e;
      down[r] = __uint_as_float((unsigned)(254 - e) << 23);
      up[r] = __uint_as_float((unsigned)e << 23);
    }
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        q[k][i] = pack_f16(__uint_as_float(q[k][i] << 16) * down[i & 1],
                           __uint_as_float(q[k][i] & 0xffff0000u) * down[i & 1]);
    f0 = up[0];
    f1 = up[1];
  }
  __device__ __forceinline__ void scores(float (&s)[TT / 8][4], uint32_t ks, uint32_t) {
    const int l = threadIdx.x & 31;
    const uint32_t a0 = ks + ((l & 7) + (l >> 4) * 8) * PITCH + ((l >> 3) & 1) * 16;
    // four matrices: 16 tokens x two groups of 16 elements
#pragma unroll
    for (int k = 0; k < DP / 32; ++k)
#pragma unroll
      for (int n = 0; n < TT / 16; ++n) {
        unsigned b[4];
        ldsm4(b, a0 + n * 16 * PITCH + k * 32);
        mma_f16(s[2 * n], q[2 * k], e4m3_f16(b[0]), e4m3_f16(b[0] >> 16));
        mma_f16(s[2 * n + 1], q[2 * k], e4m3_f16(b[2]), e4m3_f16(b[2] >> 16));
        mma_f16(s[2 * n], q[2 * k + 1], e4m3_f16(b[1]), e4m3_f16(b[1] >> 16));
        mma_f16(s[2 * n + 1], q[2 * k + 1], e4m3_f16(b[3]), e4m3_f16(b[3] >> 16));
      }
#pragma unroll
    for (int n = 0; n < TT / 8; ++n) {
      s[n][0] *= f0;
      s[n][1] *= f0;
      s[n][2] *= f1;
      s[n][3] *= f1;
    }
  }
  __device__ __forceinline__ void outputs(float (&o)[DP / 8][4], const float (&p)[TT / 8][4],
                                          uint32_t vs) {
    const int l = threadIdx.x & 31;
    const uint32_t a0 = vs + (l & 15) * PITCH + (l >> 4) * 16;
#pragma unroll
    for (int k = 0; k < TT / 16; ++k) {
      unsigned w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack_f16(p[2 * k + (i >> 1)][(i & 1) * 2], p[2 * k + (i >> 1)][(i & 1) * 2 + 1]);
#pragma unroll
      for (int n = 0; n < DP / 32; ++n) {
        unsigned b[4];
        // matrices: tokens 0-7 and 8-15 of element pairs 32n .. +15, then +16 .. +31
        ldsm4t(b, a0 + k * 16 * PITCH + n * 32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // bytes (t, 2g) (t, 2g+1) (t+1, 2g) (t+1, 2g+1): sort by element
          const unsigned x = __byte_perm(b[2 * h], 0, 0x3120);
          const unsigned y = __byte_perm(b[2 * h + 1], 0, 0x3120);
          mma_f16(o[4 * n + 2 * h], w, e4m3_f16(x), e4m3_f16(y));
          mma_f16(o[4 * n + 2 * h + 1], w, e4m3_f16(x >> 16), e4m3_f16(y >> 16));
        }
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ static void each(const float (&o)[DP / 8][4], F &&f) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < DP / 16; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        f(0, n * 16 + t * 4 + c * 2, o[2 * n][c], o[2 * n + 1][c]);
        f(1, n * 16 + t * 4 + c * 2, o[2 * n][2 + c], o[2 * n + 1][2 + c]);
      }
  }
};

// f32: every product in three TF32 ones (high x high, high x low, low x high),
// which leaves errors of 2^-22 of a term.  The queries lie in shared memory:
// their parts would not fit the registers.  The tokens of a product's 8 are
// taken in the order 0 2 4 6 1 3 5 7, so that a thread's scores are already
// its share of the second product.
template <int DP_, int TT_>
struct F32 {
  static constexpr int DP = DP_, TT = TT_, ESZ = 4, PITCH = DP * 4 + 16, QSMEM = 16 * PITCH;
  static constexpr float kShift = 0.f;
  static_assert(TT == 8, "one token tile of the product");

  __device__ __forceinline__ void load_q(const char *qp, int rows, int dim, uint32_t qs) {
    __syncwarp();
    for (int i = threadIdx.x & 31; i < 16 * (DP / 4); i += 32) {
      const int row = i / (DP / 4), c = (i % (DP / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < rows && c < dim)
        v = __ldg(reinterpret_cast<const float4 *>(qp + ((int64_t)row * dim + c) * 4));
      asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(qs + row * PITCH + c * 4),
                   "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                   : "memory");
    }
    __syncwarp();
  }
  __device__ __forceinline__ void scores(float (&s)[1][4], uint32_t ks, uint32_t qs) {
    const int l = threadIdx.x & 31;
    const uint32_t kb = ks + (l & 7) * PITCH + (l >> 3) * 16;
    const uint32_t qb = qs + ((l & 7) + ((l >> 3) & 1) * 8) * PITCH + (l >> 4) * 16;
    float x[4] = {0.f, 0.f, 0.f, 0.f};  // the cross terms
#pragma unroll 4
    for (int k = 0; k < DP / 16; ++k) {
      unsigned b[4];
      ldsm4(b, kb + k * 64);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unsigned a[4], ah[4], al[4], bh0, bl0, bh1, bl1;
        ldsm4(a, qb + k * 64 + h * 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) split_tf32(a[i], ah[i], al[i]);
        split_tf32(b[2 * h], bh0, bl0);
        split_tf32(b[2 * h + 1], bh1, bl1);
        mma_tf32(x, al, bh0, bh1);
        mma_tf32(x, ah, bl0, bl1);
        mma_tf32(s[0], ah, bh0, bh1);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[0][i] += x[i];
  }
  __device__ __forceinline__ void outputs(float (&o)[DP / 8][4], const float (&p)[1][4],
                                          uint32_t vs) {
    const int l = threadIdx.x & 31;
    const uint32_t a0 = vs + (l & 3) * 2 * PITCH + (l >> 2) * 4;
    unsigned wh[4], wl[4];
    split_tf32(__float_as_uint(p[0][0]), wh[0], wl[0]);
    split_tf32(__float_as_uint(p[0][2]), wh[1], wl[1]);
    split_tf32(__float_as_uint(p[0][1]), wh[2], wl[2]);
    split_tf32(__float_as_uint(p[0][3]), wh[3], wl[3]);
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      unsigned b0, b1, bh0, bl0, bh1, bl1;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b0) : "r"(a0 + n * 32) : "memory");
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b1) : "r"(a0 + PITCH + n * 32) : "memory");
      split_tf32(b0, bh0, bl0);
      split_tf32(b1, bh1, bl1);
      mma_tf32(o[n], wl, bh0, bh1);
      mma_tf32(o[n], wh, bl0, bl1);
      mma_tf32(o[n], wh, bh0, bh1);
    }
  }
  template <typename F>
  __device__ __forceinline__ static void each(const float (&o)[DP / 8][4], F &&f) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      f(0, n * 8 + t * 2, o[n][0], o[n][1]);
      f(1, n * 8 + t * 2, o[n][2], o[n][3]);
    }
  }
};

// ---------------------------------------------------------------------------

// Length of sequence b within what the table can hold.
__device__ __forceinline__ int length_of(const AttendArgs &a, int b, bool &bad) {
  return cache_length(__ldg(a.s.lengths + b), a.s.table_width, a.p.page_size, bad);
}

// A place on the line of tiles.
struct Cursor {
  int b, hr, tile;  // sequence, cached head * blocks + row block, tile of the segment
  Span s;
  __device__ __forceinline__ void enter(const AttendArgs &a, int tile_tokens) {
    bool bad;
    s = cache_span(length_of(a, b, bad), a.window, tile_tokens);
  }
  __device__ __forceinline__ void next(const AttendArgs &a, int tile_tokens) {
    if (++tile < s.count) return;
    tile = 0;
    if (++hr < a.p.kv_heads * a.blocks) return;
    hr = 0;
    if (++b < a.s.B) enter(a, tile_tokens);
  }
};

template <typename T>
__device__ __forceinline__ void store2(char *p, float x, float y);
template <>
__device__ __forceinline__ void store2<float>(char *p, float x, float y) {
  *reinterpret_cast<float2 *>(p) = make_float2(x, y);
}
template <>
__device__ __forceinline__ void store2<__nv_bfloat16>(char *p, float x, float y) {
  *reinterpret_cast<unsigned *>(p) = pack_bf16(x, y);
}

template <typename TY, int WARPS, int STAGES>
struct Layout {
  static constexpr int kTile = TY::TT * TY::PITCH;  // keys, then values
  static constexpr int kStage = 2 * kTile;
  static constexpr int kRing = STAGES * kStage;
  static constexpr int kWarp = kRing + TY::QSMEM;
  static constexpr int kJoinPitch = TY::DP + 8;  // floats: rows 8 banks apart
  static constexpr int kSmem = WARPS * kWarp;
  static_assert(kRing >= kAttendRows * kJoinPitch * 4, "a warp's sums fit its ring");
  static_assert(kSmem <= 222 * 1024, "shared memory of an SM, less the static part");
};

template <typename TY, typename TO, int WARPS, int STAGES>
__global__ void __launch_bounds__(WARPS * 32, 1) k_attend(const __grid_constant__ AttendArgs a) {
  using L = Layout<TY, WARPS, STAGES>;
  constexpr int DP = TY::DP, TT = TY::TT, ESZ = TY::ESZ;
  extern __shared__ __align__(128) char smem[];
  __shared__ long long before[WARPS * 32 + 1];  // tiles before each thread's sequences
  __shared__ long long wsum[WARPS];
  __shared__ unsigned bits[WARPS][STAGES];       // visible tokens of a stage's tile
  __shared__ float2 jml[WARPS][kAttendRows];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2;
  char *ring = smem + warp * L::kWarp;
  const uint32_t ring_u = smem_u32(ring), qs = ring_u + L::kRing;

  if (a.p.dim < DP) {  // elements behind the head's own: zeros, which no copy touches
    for (int i = lane; i < L::kRing / 16; i += 32)
      reinterpret_cast<uint4 *>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncwarp();
  }
  griddep_wait();
  griddep_launch();

  // ---- the line of tiles, and this warp's piece of it ---------------------
  const int chunk = (a.s.B + WARPS * 32 - 1) / (WARPS * 32);
  const int hrs = a.p.kv_heads * a.blocks;
  {
    long long mine = 0;
    for (int i = 0; i < chunk; ++i) {
      const int b = threadIdx.x * chunk + i;
      if (b >= a.s.B) break;
      bool bad;
      const int len = length_of(a, b, bad);
      if (bad && blockIdx.x == 0 && a.errors) atomicOr(a.errors, (unsigned)FWPKM_CACHE_BAD_LENGTH);
      mine += cache_span(len, a.window, TT).count;
    }
    mine *= hrs;
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(FULL, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) wsum[warp] = sum;
    __syncthreads();
    long long base = 0;
    for (int w = 0; w < warp; ++w) base += wsum[w];
    before[threadIdx.x] = base + sum - mine;
    if (threadIdx.x == WARPS * 32 - 1) before[WARPS * 32] = base + sum;
    __syncthreads();
  }
  const long long total = before[WARPS * 32];
  const int warps = cache_warps(total, gridDim.x * WARPS, kLeastTiles);
  const int w = blockIdx.x * WARPS + warp;
  const int wa = min(blockIdx.x * WARPS, warps), wb = min(wa + WARPS, warps);
  const long long cta0 = cache_cut(total, warps, wa), cta1 = cache_cut(total, warps, wb);
  const long long t0 = w < warps ? cache_cut(total, warps, w) : total;
  const long long t1 = w < warps ? cache_cut(total, warps, w + 1) : total;

  Cursor at{};        // the tile that is computed
  long long seg = 0;  // first tile of its segment
  if (t0 < t1) {
    int i = 0;  // the thread whose sequences t0 falls into
    for (int j = lane; j < WARPS * 32; j += 32) i += before[j + 1] <= t0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) i += __shfl_xor_sync(FULL, i, o);
    long long p = before[i];
    at.b = i * chunk;
    at.enter(a, TT);
    while (p + (long long)at.s.count * hrs <= t0) {
      p += (long long)at.s.count * hrs;
      ++at.b;
      at.enter(a, TT);
    }
    at.hr = (int)((t0 - p) / at.s.count);
    at.tile = (int)((t0 - p) - (long long)at.hr * at.s.count);
    seg = t0 - at.tile;
  }
  // the whole piece of the CTA lies in one segment (all its warps agree)
  const bool joined = cta0 < cta1 && (t0 >= t1 || (seg <= cta0 && seg + at.s.count >= cta1));
  // a warp without tiles cannot tell, and has no part in either case

  // ---- loads ---------------------------------------------------------------
  constexpr int CPR = DP * ESZ / 16;  // 16-byte pieces of a padded row
  const int cpr = a.p.dim * ESZ / 16;
  Cursor ld = at;
  int token = 0, page = -1;  // of this lane's row of the next tile to load
  bool seen = false;
  auto look = [&] {
    token = (ld.s.first + ld.tile) * TT + (lane % TT);
    seen = token >= ld.s.lo && token < ld.s.len;
    page = seen ? __ldg(a.s.table + ld.b * a.s.table_stride + token / a.p.page_size) : -1;
  };
  auto load = [&](int stage) {
    const bool ok = seen && (unsigned)page < (unsigned)a.p.pages;
    if (seen && !ok && a.errors && lane < TT) atomicOr(a.errors, (unsigned)FWPKM_CACHE_BAD_PAGE);
    const unsigned vis = __ballot_sync(FULL, ok);
    if (lane == 0) bits[warp][stage] = vis;
    const int64_t off = ok ? page * a.p.page_stride +
                                 (int64_t)(ld.hr / a.blocks) * a.p.head_stride +
                                 (int64_t)(token % a.p.page_size) * a.p.row_stride
                           : 0;
    const uint32_t dst = ring_u + stage * L::kStage;
#pragma unroll
    for (int i = 0; i < TT * CPR / 32; ++i) {
      const int flat = i * 32 + lane, row = flat / CPR, c = flat % CPR;
      const int64_t ro = __shfl_sync(FULL, off, row) + c * 16;
      const bool rok = (vis >> row) & 1u;
      if (c < cpr) {
        cp_async16(dst + row * TY::PITCH + c * 16, rok ? a.p.keys + ro : a.p.keys, rok);
        cp_async16(dst + L::kTile + row * TY::PITCH + c * 16, rok ? a.p.values + ro : a.p.values,
                   rok);
      }
    }
  };
  long long next = t0;  // next tile to load
  if (t0 < t1) look();
  auto advance = [&](int stage) {
    if (next < t1) {
      load(stage);
      if (++next < t1) {
        ld.next(a, TT);
        look();
      }
    }
    cp_commit();
  };
  for (int i = 0; i < STAGES - 1; ++i) advance(i);

  // ---- the pass --------------------------------------------------------------
  TY ty;
  float o[DP / 8][4];
  float m[2], l[2], c = 0.f;  // of rows g and g + 8; c: scale of the scores
  int rows = 0;
  bool fresh = true, whole = at.tile == 0;
  auto reset = [&] {
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    m[0] = m[1] = kNegInf;
    l[0] = l[1] = 0.f;
  };
  reset();
  auto sum_l = [&] {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(FULL, l[r], 1);
      l[r] += __shfl_xor_sync(FULL, l[r], 2);
    }
  };
  // Row r of the segment's result, finished.
  auto row_of = [&](const Cursor &k, int r) {
    return (int64_t)k.b * a.heads + (k.hr / a.blocks) * a.group + (k.hr % a.blocks) * kAttendRows +
           r;
  };
  auto finish = [&] {
    const float vs = a.p.value_scale ? __ldg(a.p.value_scale + at.hr / a.blocks) : 1.f;
    float inv[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) inv[r] = l[r] == 0.f ? 0.f : vs / l[r];
    const int64_t r0 = row_of(at, 0);
    TY::each(o, [&](int h, int col, float x, float y) {
      if (g + h * 8 < rows && col < a.p.dim)
        store2<TO>(a.out + ((r0 + g + h * 8) * a.p.dim + col) * (int64_t)sizeof(TO), x * inv[h],
                   y * inv[h]);
    });
    if (a.lse && (lane & 3) == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (g + h * 8 < rows)
          a.lse[r0 + g + h * 8] = l[h] == 0.f ? kNegInf : kLn2 * (m[h] + log2f(l[h]));
    }
  };
  auto park = [&](int slot) {
    float *dst = a.parts + (int64_t)slot * kAttendRows * DP;
    TY::each(o, [&](int h, int col, float x, float y) {
      if (g + h * 8 < rows)
        *reinterpret_cast<float2 *>(dst + (g + h * 8) * DP + col) = make_float2(x, y);
    });
    if ((lane & 3) == 0) {
      a.ml[slot * kAttendRows + g] = make_float2(m[0], l[0]);
      a.ml[slot * kAttendRows + g + 8] = make_float2(m[1], l[1]);
    }
  };

  int4 tail = make_int4(0, 0, -1, 0);
  int stage = 0;
  for (long long t = t0; t < t1; ++t) {
    if (fresh) {
      const int h = at.hr / a.blocks, first = (at.hr % a.blocks) * kAttendRows;
      rows = min(kAttendRows, a.group - first);
      ty.load_q(a.q + at.b * a.q_stride + (int64_t)(h * a.group + first) * a.p.dim * sizeof(TO),
                rows, a.p.dim, qs);
      c = a.scale_log2 * (a.p.key_scale ? __ldg(a.p.key_scale + h) : 1.f);
      fresh = false;
    }
    cp_wait<STAGES - 2>();
    __syncwarp();  // the tile has landed, and the stage before it is free
    const int into = stage == 0 ? STAGES - 1 : stage - 1;
    advance(into);

    const uint32_t ks = ring_u + stage * L::kStage, vs = ks + L::kTile;
    const unsigned vis = bits[warp][stage];
    float s[TT / 8][4];
#pragma unroll
    for (int n = 0; n < TT / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    ty.scores(s, ks, qs);
    constexpr unsigned kAll = TT == 32 ? FULL : (1u << (TT % 32)) - 1u;
    const unsigned my = vis >> (2 * (lane & 3));
    float top[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int n = 0; n < TT / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[n][i] *= c;
        if ((vis & kAll) != kAll && !((my >> (8 * n + (i & 1))) & 1u)) s[n][i] = kNegInf;
        top[i >> 1] = fmaxf(top[i >> 1], s[n][i]);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 2));
      // weights are 2^(s - m); kShift makes the largest 2^kShift
      top[r] = fmaxf(m[r], top[r] - TY::kShift);
    }
    if (__any_sync(FULL, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float f = exp2f(m[r] - (top[r] == kNegInf ? 0.f : top[r]));
        l[r] *= f;
        m[r] = top[r];
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          o[n][2 * r] *= f;
          o[n][2 * r + 1] *= f;
        }
      }
    }
    const float u0 = m[0] == kNegInf ? 0.f : m[0], u1 = m[1] == kNegInf ? 0.f : m[1];
#pragma unroll
    for (int n = 0; n < TT / 8; ++n) {
      s[n][0] = exp2f(s[n][0] - u0);
      s[n][1] = exp2f(s[n][1] - u0);
      s[n][2] = exp2f(s[n][2] - u1);
      s[n][3] = exp2f(s[n][3] - u1);
      l[0] += s[n][0] + s[n][1];
      l[1] += s[n][2] + s[n][3];
    }
    ty.outputs(o, s, vs);

    stage = stage + 1 == STAGES ? 0 : stage + 1;
    if (at.tile + 1 == at.s.count) {  // the segment ends here
      if (!joined) {
        sum_l();
        if (whole) finish();
        else park(2 * w);
        reset();
      }
      fresh = whole = true;
      if (t + 1 < t1) {
        at.next(a, TT);
        seg = t + 1;
      }
    } else if (t + 1 < t1) {
      ++at.tile;
    } else if (!joined) {  // the segment goes on in the next warp
      sum_l();
      park(whole ? 2 * w + 1 : 2 * w);
      if (whole)
        tail = make_int4(at.b, at.hr, cache_last_warp(total, warps, seg + at.s.count), 0);
    }
  }

  // ---- a CTA inside one segment: its warps' sums in one ----------------------
  const bool all = __syncthreads_or(t0 < t1 && joined);
  if (all) {
    sum_l();
    float *mine = reinterpret_cast<float *>(ring);
    TY::each(o, [&](int h, int col, float x, float y) {
      *reinterpret_cast<float2 *>(mine + (g + h * 8) * L::kJoinPitch + col) = make_float2(x, y);
    });
    if ((lane & 3) == 0) {
      jml[warp][g] = make_float2(m[0], l[0]);
      jml[warp][g + 8] = make_float2(m[1], l[1]);
    }
    // warp 0 of such a CTA has tiles: its cursor names the segment
    __shared__ int4 sseg;
    __shared__ int srows;
    if (threadIdx.x == 0) {
      sseg = make_int4(at.b, at.hr, 0, 0);
      srows = rows;
      const bool starts = seg == cta0, ends = seg + at.s.count == cta1;
      sseg.z = starts && ends ? 1 : 0;
      sseg.w = starts ? 2 * wa + 1 : 2 * wa;
      if (starts && !ends)
        tail = make_int4(at.b, at.hr, cache_last_warp(total, warps, seg + at.s.count), 0);
    }
    __syncthreads();
    const int4 sg = sseg;
    const int h = sg.y / a.blocks;
    const float vs = a.p.value_scale ? __ldg(a.p.value_scale + h) : 1.f;
    const int64_t r0 =
        (int64_t)sg.x * a.heads + h * a.group + (sg.y % a.blocks) * (int64_t)kAttendRows;
    for (int i = threadIdx.x; i < srows * (DP / 2); i += WARPS * 32) {
      const int row = i / (DP / 2), col = (i - row * (DP / 2)) * 2;
      float top = kNegInf;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) top = fmaxf(top, jml[k][row].x);
      const float u = top == kNegInf ? 0.f : top;
      float x = 0.f, y = 0.f, sum = 0.f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        const float f = exp2f(jml[k][row].x - u);
        const float2 v = *reinterpret_cast<const float2 *>(
            smem + k * L::kWarp + (row * L::kJoinPitch + col) * 4);
        sum = fmaf(jml[k][row].y, f, sum);
        x = fmaf(v.x, f, x);
        y = fmaf(v.y, f, y);
      }
      if (sg.z) {
        const float inv = sum == 0.f ? 0.f : vs / sum;
        if (col < a.p.dim)
          store2<TO>(a.out + ((r0 + row) * a.p.dim + col) * (int64_t)sizeof(TO), x * inv, y * inv);
        if (col == 0 && a.lse) a.lse[r0 + row] = sum == 0.f ? kNegInf : kLn2 * (top + log2f(sum));
      } else {
        *reinterpret_cast<float2 *>(a.parts + ((int64_t)sg.w * kAttendRows + row) * DP + col) =
            make_float2(x, y);
        if (col == 0) a.ml[sg.w * kAttendRows + row] = make_float2(top, sum);
      }
    }
    // the other warps' slots hold nothing
    if (warp > 0 && lane < kAttendRows && w < warps)
      a.ml[2 * w * kAttendRows + lane] = make_float2(kNegInf, 0.f);
  }
  if (lane == 0) a.tails[w] = tail;
}

// Joins the parts of the segments that begin in one CTA's warps: a warp to a
// query row, two passes over the parts (their maximum, then their sums).
template <typename TO, int DP, int WARPS>
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ AttendArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch();
  constexpr int V = DP / 32;  // columns of a lane, 2 (DP = 64), 4 or 8
  for (int i = warp; i < WARPS * kAttendRows; i += 8) {
    const int w = blockIdx.x * WARPS + i / kAttendRows, row = i % kAttendRows;
    const int4 t = a.tails[w];
    if (t.z < 0) continue;
    const int h = t.y / a.blocks, first = (t.y % a.blocks) * kAttendRows;
    if (row >= a.group - first) continue;
    const int n = t.z - w + 1;  // parts
    auto slot = [&](int k) { return k == 0 ? 2 * w + 1 : 2 * (w + k); };
    float top = kNegInf;
    for (int k = lane; k < n; k += 32) top = fmaxf(top, a.ml[slot(k) * kAttendRows + row].x);
    top = warp_max(top);
    const float u = top == kNegInf ? 0.f : top;
    float acc[V] = {}, sum = 0.f;
    for (int k0 = 0; k0 < n; k0 += 32) {
      float f = 0.f;
      if (k0 + lane < n) {
        const float2 ml = a.ml[slot(k0 + lane) * kAttendRows + row];
        f = exp2f(ml.x - u);
        sum += ml.y * f;
      }
      const int most = min(32, n - k0);
#pragma unroll 4
      for (int k = 0; k < most; ++k) {
        const float fk = __shfl_sync(FULL, f, k);
        if (fk == 0.f) continue;  // an empty slot's sums are not set
        const float *src =
            a.parts + ((int64_t)slot(k0 + k) * kAttendRows + row) * DP + lane * V;
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 v = *reinterpret_cast<const float2 *>(src + e);
          acc[e] = fmaf(v.x, fk, acc[e]);
          acc[e + 1] = fmaf(v.y, fk, acc[e + 1]);
        }
      }
    }
    sum = warp_sum(sum);
    const float vs = a.p.value_scale ? __ldg(a.p.value_scale + h) : 1.f;
    const float inv = sum == 0.f ? 0.f : vs / sum;
    const int64_t r = (int64_t)t.x * a.heads + h * a.group + first + row;
#pragma unroll
    for (int e = 0; e < V; e += 2)
      if (lane * V + e < a.p.dim)
        store2<TO>(a.out + (r * a.p.dim + lane * V + e) * (int64_t)sizeof(TO), acc[e] * inv,
                   acc[e + 1] * inv);
    if (lane == 0 && a.lse) a.lse[r] = sum == 0.f ? kNegInf : kLn2 * (top + log2f(sum));
  }
}

template <typename TY, typename TO, int WARPS, int STAGES>
cudaError_t launch(const AttendArgs &a, cudaStream_t st) {
  using L = Layout<TY, WARPS, STAGES>;
  auto *kernel = k_attend<TY, TO, WARPS, STAGES>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_k(true, kernel, dim3(kAttendCtas), dim3(WARPS * 32), L::kSmem, st, a);
  if (e != cudaSuccess) return e;
  return launch_k(true, k_join<TO, TY::DP, WARPS>, dim3(kAttendCtas), dim3(256), 0, st, a);
}

}  // namespace attend
}  // namespace fwpkm
