// kernels_cache_attend.cuh -- attention of one token of each sequence over a
// paged cache.  Per query head, over the visible tokens t in tiles:
//   o = sum 2^(c s_t - m) v_t,   l = sum 2^(c s_t - m),   s_t = q.k_t,
// c = scale log2(e); where a tile brings a score well above the reference m, o
// and l are first scaled to a new one.  At the end out = o / l and lse =
// ln 2 (m + log2 l): one pass over the cache.
//
// Every cached byte is read once and takes only heads/kv_heads products, so
// HBM bandwidth bounds it (8 query heads to a cached bf16 head: 8 flops a byte,
// 52 TFLOP/s at the measured 6.55 TB/s).  What counts is that all SMs read all
// the time, whatever the lengths are, and that the work per byte stays small:
//   - The line of all tiles is cut evenly over the warps (cache_schedule.cuh).
//   - A warp streams its piece through a ring of its own in shared memory
//     (cp.async, a unit being a tile's keys or its values), across the ends of
//     segments, and waits for no other warp: the loop has no CTA barrier.
//   - The products run on mma.sync with the TOKENS as the rows of the A operand
//     (16) and the query heads of one cached head as the columns of B (8): up to
//     8 heads fill it, where heads as rows would leave half of it or more empty,
//     and the outputs take 8 columns of registers, so that up to 16 warps fit an
//     SM.  (Heads as rows on 8 warps: 118 us where this takes 101, 126 where 64.)
//     The tcgen05 path would need 64 or 128 rows of queries; a decode step has
//     one to a few, and this holds the work under the time of the bytes up to 16
//     heads to a cached one.
// Parts of segments that a cut falls into are joined in the CTA where they lie
// next to each other, the rest by k_join through the workspace.
//
// Measured (B200, calls back to back, the cache larger than the L2): 131072
// bf16 tokens x 8 cached heads of 128, 0.54 GB, 101 us, 5.3 TB/s, 81% of the
// measured copy rate; 1.17 GB of e4m3 in 32 ragged sequences 231 us, 77%, at the
// board's power limit (211 us, 85%, in runs too short to reach it); one cached fp32
// head of 256 in 1 M tokens, 2.15 GB, 340 us for 4 query heads, 96%, and 385 for 8,
// 85%.  What is left at the large sizes: SMs in GPCs with more SMs get less bandwidth
// each (equal pieces end between 71 and 97 us), 3 us before the first load and 5 at
// the end.
#pragma once
#include <cuda_fp16.h>

#include <atomic>

#include "cache_schedule.cuh"
#include "fwpkm_cache_internal.cuh"

namespace fwpkm {
namespace attend {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -__builtin_huge_valf();
// In place of a factor 0, which would make a masked score (-infinity) no number: the
// least number above it, which no score of 32 bits feels.
constexpr float kLeastFactor = __FLT_DENORM_MIN__;
// Warps of a CTA that take pieces, at the least (where it has so many): the
// sums of those join in shared memory.  (One sequence of 1024 tokens: 12.6 us
// with 1 to 8, 16.6 with 12.)
constexpr int kLeastPerCta = 8;
// A tile's scores may bring weights this much (base 2) above the largest one at the
// time of the reference before the sums are scaled to a new one: weights stay
// under 2^(kShift + kSlack).  kShift is -kSlack where values may be as large as 32
// bits hold, so that no weight is above 1 and no sum leaves their range that
// would not with weights of the softmax.
constexpr float kSlack = 6.f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const char *src, bool ok) {
  const int n = ok ? 16 : 0;  // 0: nothing is read, zeros are written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const char *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
// The same into sums of their own.
__device__ __forceinline__ void mma_bf16_new(float (&d)[4], const unsigned (&a)[4], unsigned b0,
                                             unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16_new(float (&d)[4], const unsigned (&a)[4], unsigned b0,
                                            unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// c += a, rounded to nearest, two in one instruction.
__device__ __forceinline__ void add4(float (&c)[4], const float (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2)
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(c[i]), "+f"(c[i + 1])
        : "f"(a[i]), "f"(a[i + 1]));
}
// 2^x for x <= 0 or about so; results under 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const unsigned *>(&h);
}
__device__ __forceinline__ unsigned pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const unsigned *>(&h);
}
// Four 8-bit floats as 16-bit ones, exactly: the low two and the high two.
__device__ __forceinline__ void e4m3_f16(unsigned v, unsigned &lo, unsigned &hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
__device__ __forceinline__ unsigned transpose8(unsigned a) {  // of an 8 x 8 matrix of 16 bits
  unsigned d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Two multiply-adds in one instruction, c += a * b, each rounded as fmaf does.
struct alignas(8) Pair {
  float x, y;
};
__device__ __forceinline__ void fma2(Pair &c, const Pair &a, const Pair &b) {
  uint64_t cc = *reinterpret_cast<uint64_t *>(&c);
  asm("fma.rn.f32x2 %0, %1, %2, %0;"
      : "+l"(cc)
      : "l"(*reinterpret_cast<const uint64_t *>(&a)), "l"(*reinterpret_cast<const uint64_t *>(&b)));
  c = *reinterpret_cast<Pair *>(&cc);
}
// log sum e^s from a reference and a sum in base 2.
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? kNegInf : kLn2 * (m + log2f(l));
}

// ---------------------------------------------------------------------------
// Element types.  Each holds the queries, reference m, sum l and outputs o of
// one segment, and works on a tile of TT tokens in two steps:
//   scores(keys, visible)   weights 2^(c s - m) of the tile's tokens, kept
//   outputs(values)         o += weights x values
// Its outputs are kParts groups of 32 lanes x 4 floats; float e of group i
// and a lane belongs to head head_of and head element col_of.
// ---------------------------------------------------------------------------

// What the two tensor-core types share.  Thread (g = lane/4, t = lane%4).  s
// and p: tokens 16n + g (+ 8), heads 8h + 2t (+ 1), the accumulator layout of
// mma.m16n8.  o: head elements as rows, heads as columns.
// The tensor cores cut what a product's sum has beyond 32 bits, which over
// thousands of tokens adds up in one direction (to 2^-25 of o a product): they sum
// a tile, and an addition of its own, rounded to nearest, takes that into o.  It
// costs 0.5 to 1% with 8 bf16 heads, 2 to 8% with 8 e4m3 ones (8 cached heads of 128,
// 1.17 GB: 208 and 211 us; of 256, 0.83 GB: 156 and 166), up to 9% with 32.
// QS: the queries lie in shared memory, in the order in which the products take
// them, where the outputs need the registers.
template <typename Self, int DP_, int TT_, int NT_>
struct Mma {
  static constexpr int DP = DP_, TT = TT_, NT = NT_, HEADS = 8 * NT_;
  static constexpr bool QS = DP * NT > 256;
  static constexpr int kQuery = QS ? DP / 16 * NT * 256 : 0;  // bytes of a warp's queries
  static constexpr int kParts = DP / 16 * NT;
  unsigned q[QS ? 1 : DP / 16][QS ? 1 : NT][2];
  char *qs;  // shared memory of this warp's queries
  float c[NT][2], m[NT][2], l[NT][2];
  float o[DP / 16][NT][4];
  unsigned hi[TT / 16][NT][2];

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      m[h][0] = m[h][1] = kNegInf;
      l[h][0] = l[h][1] = 0.f;
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) o[n][h][0] = o[n][h][1] = o[n][h][2] = o[n][h][3] = 0.f;
    }
  }
  __device__ __forceinline__ void set_q(int k, int h, unsigned x, unsigned y) {
    if constexpr (QS) {
      reinterpret_cast<uint2 *>(qs)[(k * NT + h) * 32 + (threadIdx.x & 31)] = make_uint2(x, y);
    } else {
      q[k][h][0] = x;
      q[k][h][1] = y;
    }
  }
  __device__ __forceinline__ uint2 get_q(int k, int h) const {
    if constexpr (QS)
      return reinterpret_cast<const uint2 *>(qs)[(k * NT + h) * 32 + (threadIdx.x & 31)];
    else
      return make_uint2(q[k][h][0], q[k][h][1]);
  }
  // s: products; on return weights, in the same places.  shift: the largest
  // weight is 2^shift when the reference is new.
  __device__ __forceinline__ void weigh(float (&s)[TT / 16][NT][4], unsigned vis, float shift) {
    const int g = (threadIdx.x & 31) >> 2;
    if (vis != FULL) {
#pragma unroll
      for (int n = 0; n < TT / 16; ++n)
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          if (!((vis >> (16 * n + g)) & 1u)) s[n][h][0] = s[n][h][1] = kNegInf;
          if (!((vis >> (16 * n + 8 + g)) & 1u)) s[n][h][2] = s[n][h][3] = kNegInf;
        }
    }
    float top[NT][2];
    bool over = false;
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(s[0][h][e], s[0][h][2 + e]);
#pragma unroll
        for (int n = 1; n < TT / 16; ++n) x = fmaxf(x, fmaxf(s[n][h][e], s[n][h][2 + e]));
        top[h][e] = x;
        over |= fmaf(x, c[h][e], -m[h][e]) > shift + kSlack;
      }
    if (__any_sync(FULL, over)) {
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = top[h][e];
          x = fmaxf(x, __shfl_xor_sync(FULL, x, 4));
          x = fmaxf(x, __shfl_xor_sync(FULL, x, 8));
          x = fmaxf(x, __shfl_xor_sync(FULL, x, 16));
          x = fmaxf(m[h][e], fmaf(x, c[h][e], -shift));
          const float f = ex2(m[h][e] - (x == kNegInf ? 0.f : x));
          m[h][e] = x;
          l[h][e] *= f;
#pragma unroll
          for (int n = 0; n < DP / 16; ++n) {
            o[n][h][e] *= f;
            o[n][h][2 + e] *= f;
          }
        }
    }
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float u = m[h][e] == kNegInf ? 0.f : m[h][e];
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < TT / 16; ++n) {
          s[n][h][e] = ex2(fmaf(s[n][h][e], c[h][e], -u));
          s[n][h][2 + e] = ex2(fmaf(s[n][h][2 + e], c[h][e], -u));
          sum += s[n][h][e] + s[n][h][2 + e];
        }
        l[h][e] += sum;
      }
  }
  // The warp's l: each thread has summed its own tokens.
  __device__ __forceinline__ void total() {
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[h][e] += __shfl_xor_sync(FULL, l[h][e], 4);
        l[h][e] += __shfl_xor_sync(FULL, l[h][e], 8);
        l[h][e] += __shfl_xor_sync(FULL, l[h][e], 16);
      }
  }
  __device__ __forceinline__ float4 part(int i) const {
    const float(&x)[4] = o[i / NT][i % NT];
    return make_float4(x[0], x[1], x[2], x[3]);
  }
  // f(head, m, l) once for each head
  template <typename F>
  __device__ __forceinline__ void stats(F &&f) const {
    if ((threadIdx.x & 31) < 4)
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) f(8 * h + 2 * (threadIdx.x & 3) + e, m[h][e], l[h][e]);
  }
  __device__ __forceinline__ static int head_of(int i, int lane, int e) {
    return 8 * (i % NT) + 2 * (lane & 3) + (e & 1);
  }
  __device__ __forceinline__ static int col_of(int i, int lane, int e) {
    return i / NT * 16 + Self::row_elem((lane >> 2) + 8 * (e >> 1));
  }
  // The segment's result; vs: the values' scale.
  __device__ __forceinline__ void finish(__nv_bfloat16 *out, float *lse, int rows, int dim,
                                         float vs) {
    total();
    float inv[NT][2];
#pragma unroll
    for (int h = 0; h < NT; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        inv[h][e] = l[h][e] == 0.f ? 0.f : vs / l[h][e];
        if (l[h][e] == 0.f)  // nothing was weighed: 0, whatever the values are
#pragma unroll
          for (int n = 0; n < DP / 16; ++n) o[n][h][e] = o[n][h][2 + e] = 0.f;
      }
    static_cast<Self *>(this)->write(out, rows, dim, inv);
    if (lse)
      stats([&](int h, float mh, float lh) {
        if (h < rows) lse[h] = log_sum(mh, lh);
      });
  }
};

// bf16: weights go in as two bf16 parts, so that rounding them costs nothing
// of the result's accuracy (one part alone would add an error of the size of
// the final rounding).  The second product is hidden behind the loads.
template <int DP_, int TT_, int NT_>
struct Bf16 : Mma<Bf16<DP_, TT_, NT_>, DP_, TT_, NT_> {
  using B = Mma<Bf16<DP_, TT_, NT_>, DP_, TT_, NT_>;
  using Out = __nv_bfloat16;
  static constexpr int DP = DP_, TT = TT_, NT = NT_, ESZ = 2, PITCH = DP * 2 + 16;
  static constexpr int kDtype = FWPKM_BF16;
  static constexpr float kShift = -kSlack;
  unsigned lo[TT / 16][NT][2];

  // Head element of row r of an output tile's 16.
  __device__ __forceinline__ static int row_elem(int r) { return r; }
  __device__ __forceinline__ void load_q(const char *qp, int rows, int dim, float f) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    const unsigned flip = f < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        unsigned x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 8 * h + g, c = k * 16 + t * 2 + i * 8;
          x[i] = row < rows && c < dim
                     ? flip ^ __ldg(reinterpret_cast<const unsigned *>(qp + (row * dim + c) * 2))
                     : 0u;
        }
        this->set_q(k, h, x[0], x[1]);
      }
#pragma unroll
    for (int h = 0; h < NT; ++h) this->c[h][0] = this->c[h][1] = fmaxf(fabsf(f), kLeastFactor);
  }
  __device__ __forceinline__ void scores(const char *ks, unsigned vis) {
    const int lane = threadIdx.x & 31;
    const uint32_t a0 = smem_u32(ks) + ((lane & 7) + ((lane >> 3) & 1) * 8) * PITCH + (lane >> 4) * 16;
    float s[TT / 16][NT][4] = {};
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
#pragma unroll
      for (int n = 0; n < TT / 16; ++n) {
        unsigned a[4];
        ldsm4(a, a0 + n * 16 * PITCH + k * 32);
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          const uint2 q = this->get_q(k, h);
          mma_bf16(s[n][h], a, q.x, q.y);
        }
      }
    this->weigh(s, vis, kShift);
#pragma unroll
    for (int n = 0; n < TT / 16; ++n)
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = s[n][h][2 * i], y = s[n][h][2 * i + 1];
          const unsigned w = pack_bf16(x, y);
          this->hi[n][h][i] = transpose8(w);
          lo[n][h][i] = transpose8(
              pack_bf16(x - __uint_as_float(w << 16), y - __uint_as_float(w & 0xffff0000u)));
        }
  }
  __device__ __forceinline__ void outputs(const char *vs) {
    const int lane = threadIdx.x & 31;
    const uint32_t a0 = smem_u32(vs) + ((lane & 7) + (lane >> 4) * 8) * PITCH + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int n = 0; n < DP / 16; ++n) {
      float x[NT][4];  // the tile's sums
#pragma unroll
      for (int k = 0; k < TT / 16; ++k) {
        unsigned a[4];
        ldsm4t(a, a0 + k * 16 * PITCH + n * 32);
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          if (k == 0) mma_bf16_new(x[h], a, lo[k][h][0], lo[k][h][1]);
          else mma_bf16(x[h], a, lo[k][h][0], lo[k][h][1]);
          mma_bf16(x[h], a, this->hi[k][h][0], this->hi[k][h][1]);
        }
      }
#pragma unroll
      for (int h = 0; h < NT; ++h) add4(this->o[n][h], x[h]);
    }
  }
  // The finished rows: out + row * dim, for the block's first `rows` heads.
  __device__ __forceinline__ void write(Out *out, int rows, int dim, const float (&inv)[NT][2]) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < DP / 16; ++n)
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const unsigned w = transpose8(pack_bf16(this->o[n][h][2 * i] * inv[h][0],
                                                  this->o[n][h][2 * i + 1] * inv[h][1]));
          const int row = 8 * h + g, c = n * 16 + i * 8 + t * 2;
          if (row < rows && c < dim) *reinterpret_cast<unsigned *>(out + row * dim + c) = w;
        }
  }
};

// e4m3: an 8-bit element is exact in 16-bit floats, so the products run on
// those.  A row of queries is scaled by a power of two so that its largest
// element lies in [1, 2): what a bf16 element then loses to the 16-bit range is
// under 2^-25 of the largest, no more than the 32-bit sum.  Weights are held
// 2^8 too large (kShift), which keeps all down to 2^-22 of the largest above
// the 16-bit format's smallest normal number, and go in as two parts, 22 bits: one
// part alone, 11 bits, left errors of 2^-12 of the terms, which show where an
// output is far smaller than they are.  With up to 8 heads to a cached one the
// second product takes no time by itself (8 cached heads of 128 with 8 query heads
// each, 1.17 GB: 205 us with one, 200 with two) but power: at the board's limit up to
// 6%.  Padded widths take 8% longer, 16 heads to a cached one 11%.
// ldmatrix moves pairs of 8-bit elements: a lane gets 4 neighbouring elements
// of a token's keys, taken as elements 2t, 2t+1, 2t+8, 2t+9 of the product's
// 16 (the queries are loaded in the same order), and 2 neighbouring elements of
// two tokens' values, which become rows g and g + 8 of the outputs.
template <int DP_, int TT_, int NT_>
struct E4m3 : Mma<E4m3<DP_, TT_, NT_>, DP_, TT_, NT_> {
  using B = Mma<E4m3<DP_, TT_, NT_>, DP_, TT_, NT_>;
  using Out = __nv_bfloat16;
  static constexpr int DP = DP_, TT = TT_, NT = NT_, ESZ = 1, PITCH = DP + 16;
  static constexpr int kDtype = FWPKM_E4M3;
  static constexpr float kShift = 8.f;
  unsigned lo[TT / 16][NT][2];

  __device__ __forceinline__ static int row_elem(int r) { return (r & 7) * 2 + (r >> 3); }
  __device__ __forceinline__ void load_q(const char *qp, int rows, int dim, float f) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      float top = 0.f;
      unsigned x[DP / 16][2];
      const int row = 8 * h + g;
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        const int c = k * 16 + t * 4;
        uint2 v = make_uint2(0u, 0u);
        if (row < rows && c < dim)
          v = __ldg(reinterpret_cast<const uint2 *>(qp + (row * dim + c) * 2));
        x[k][0] = v.x;
        x[k][1] = v.y;
        const float m0 = fmaxf(fabsf(__uint_as_float(v.x << 16)),
                               fabsf(__uint_as_float(v.x & 0xffff0000u)));
        const float m1 = fmaxf(fabsf(__uint_as_float(v.y << 16)),
                               fabsf(__uint_as_float(v.y & 0xffff0000u)));
        top = fmaxf(top, fmaxf(m0, m1));
      }
      top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
      top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
      // 2^-e and 2^e, e the exponent of the largest element kept where both
      // are normal numbers (rows of denormal numbers then have elements under
      // 1/2; beside an infinity the others do not matter, but stay finite)
      int e = (int)((__float_as_uint(top) >> 23) & 255u);
      e = e < 2 ? 2 : e > 252 ? 252 : e;
      // (f - f: a head whose scale is no number has no score that is one)
      const float down =
          __uint_as_float(((unsigned)(254 - e) << 23) | (f < 0.f ? 0x80000000u : 0u)) + (f - f);
      const float up = __uint_as_float((unsigned)e << 23);
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          x[k][i] = pack_f16(__uint_as_float(x[k][i] << 16) * down,
                             __uint_as_float(x[k][i] & 0xffff0000u) * down);
        this->set_q(k, h, x[k][0], x[k][1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)  // the factors of this thread's columns
        this->c[h][i] =
            fmaxf(fabsf(f) * __shfl_sync(FULL, up, (2 * t + i) * 4), kLeastFactor);
    }
  }
  __device__ __forceinline__ void scores(const char *ks, unsigned vis) {
    const int lane = threadIdx.x & 31;
    const uint32_t a0 = smem_u32(ks) + ((lane & 7) + ((lane >> 3) & 1) * 8) * PITCH + (lane >> 4) * 16;
    float s[TT / 16][NT][4] = {};
#pragma unroll
    for (int k = 0; k < DP / 32; ++k)
#pragma unroll
      for (int n = 0; n < TT / 16; ++n) {
        unsigned b[4];  // tokens 0-7 and 8-15 of 16 elements, then of the next 16
        ldsm4(b, a0 + n * 16 * PITCH + k * 32);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          unsigned a[4];
          e4m3_f16(b[2 * j], a[0], a[2]);
          e4m3_f16(b[2 * j + 1], a[1], a[3]);
#pragma unroll
          for (int h = 0; h < NT; ++h) {
            const uint2 q = this->get_q(2 * k + j, h);
            mma_f16(s[n][h], a, q.x, q.y);
          }
        }
      }
    this->weigh(s, vis, kShift);
#pragma unroll
    for (int n = 0; n < TT / 16; ++n)
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = s[n][h][2 * i], y = s[n][h][2 * i + 1];
          const __half2 w = __floats2half2_rn(x, y);
          this->hi[n][h][i] = transpose8(*reinterpret_cast<const unsigned *>(&w));
          lo[n][h][i] = transpose8(pack_f16(x - __low2float(w), y - __high2float(w)));
        }
  }
  __device__ __forceinline__ void outputs(const char *vs) {
    const int lane = threadIdx.x & 31;
    const uint32_t a0 = smem_u32(vs) + (lane & 15) * PITCH + (lane >> 4) * 16;
#pragma unroll
    for (int n = 0; n < DP / 32; ++n) {
      float x[2][NT][4];  // the tile's sums
#pragma unroll
      for (int k = 0; k < TT / 16; ++k) {
        unsigned b[4];  // tokens 0-7 and 8-15 of 8 pairs of elements, then of the next 8
        ldsm4t(b, a0 + k * 16 * PITCH + n * 32);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // bytes (t, 2g) (t, 2g+1) (t+1, 2g) (t+1, 2g+1): sort by element
          unsigned a[4];
          e4m3_f16(__byte_perm(b[2 * j], 0, 0x3120), a[0], a[1]);
          e4m3_f16(__byte_perm(b[2 * j + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
          for (int h = 0; h < NT; ++h) {
            if (k == 0) mma_f16_new(x[j][h], a, lo[k][h][0], lo[k][h][1]);
            else mma_f16(x[j][h], a, lo[k][h][0], lo[k][h][1]);
            mma_f16(x[j][h], a, this->hi[k][h][0], this->hi[k][h][1]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < NT; ++h) add4(this->o[2 * n + j][h], x[j][h]);
    }
  }
  __device__ __forceinline__ void write(Out *out, int rows, int dim, const float (&inv)[NT][2]) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < DP / 16; ++n)
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        unsigned w[2];  // elements 4t, 4t + 2 and 4t + 1, 4t + 3 of the 16
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[i] = transpose8(pack_bf16(this->o[n][h][2 * i] * inv[h][0],
                                      this->o[n][h][2 * i + 1] * inv[h][1]));
        const int row = 8 * h + g, c = n * 16 + t * 4;
        if (row < rows && c < dim)
          *reinterpret_cast<uint2 *>(out + row * dim + c) =
              make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632));
      }
  }
};

// f32: the products run as plain 32-bit multiply-adds, which hold the full
// accuracy, two to an instruction; RR heads take RR of them an element, 4 flops a
// byte at 8 heads, a third of what the SMs can do in the time of the bytes.  A group of LG lanes
// has two of the heads, a lane of it DP/LG elements of their queries and outputs
// (in pieces of 4, the group's side by side).  A lane's sums of its elements, 8
// tokens x 2 heads, are summed over the group by halving: each step exchanges
// half of what a lane has left.
template <int DP_, int RR_>
struct F32 {
  using Out = float;
  static constexpr int DP = DP_, TT = 8, HEADS = RR_, RR = RR_, ESZ = 4, PITCH = DP * 4;
  static constexpr int kDtype = FWPKM_F32;
  static constexpr float kShift = -kSlack;
  static constexpr int LG = 64 / RR, V4 = DP / LG / 4;  // lanes of a group, pieces of a lane
  static constexpr int NS = 16 / LG;                    // scores of a lane: tokens of one head
  static constexpr int kParts = 2 * V4, kQuery = 0;
  static_assert(RR == 4 || RR == 8 || RR == 16, "groups of 16, 8 or 4 lanes");
  Pair q[2][V4][2], o[2][V4][2];  // element pairs
  float c, m, l;  // of head head(); l: of the lane's own tokens
  float p[NS];
  int dim;
  char *qs;  // (the queries fit the registers)

  __device__ __forceinline__ static int lane() { return threadIdx.x & 31; }
  // After the halving lane j of a group has sums j*NS .. of its 16, in the order
  // head (2), token (8).
  __device__ __forceinline__ static int head() {
    return lane() / LG * 2 + (lane() % LG) * NS / 8;
  }
  __device__ __forceinline__ static int token() { return (lane() % LG) * NS % 8; }
  __device__ __forceinline__ void reset() {
    m = kNegInf;
    l = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < V4; ++i) o[h][i][0] = o[h][i][1] = Pair{0.f, 0.f};
  }
  __device__ __forceinline__ void load_q(const char *qp, int rows, int dim_, float f) {
    dim = dim_;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < V4; ++i) {
        const int row = lane() / LG * 2 + h, e = (i * LG + lane() % LG) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < rows && e < dim)
          v = __ldg(reinterpret_cast<const float4 *>(qp + (row * dim + e) * 4));
        const float sign = f < 0.f ? -1.f : 1.f;
        q[h][i][0] = Pair{v.x * sign, v.y * sign};
        q[h][i][1] = Pair{v.z * sign, v.w * sign};
      }
    c = fmaxf(fabsf(f), kLeastFactor);
  }
  __device__ __forceinline__ static void lds4(Pair (&x)[2], const char *a) {
    const float4 v = *reinterpret_cast<const float4 *>(a);
    x[0] = Pair{v.x, v.y};
    x[1] = Pair{v.z, v.w};
  }
  __device__ __forceinline__ void scores(const char *ks, unsigned vis) {
    const char *a0 = ks + lane() % LG * 16;
    float x[16];
#pragma unroll
    for (int t0 = 0; t0 < 8; t0 += 4) {  // (four tokens' pairs of sums at a time)
      Pair sum[2][4] = {};
#pragma unroll
      for (int i = 0; i < V4; ++i) {
        if (i * LG * 4 >= dim) break;  // (only zeros from here on)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          Pair k[2];
          lds4(k, a0 + (t0 + t) * PITCH + i * LG * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) fma2(sum[h][t], q[h][i][e], k[e]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < 4; ++t) x[h * 8 + t0 + t] = sum[h][t].x + sum[h][t].y;
    }
#pragma unroll
    for (int w = LG / 2, n = 8; w > 0; w >>= 1, n >>= 1) {
      const bool up = lane() & w;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float keep = up ? x[i + n] : x[i], give = up ? x[i] : x[i + n];
        x[i] = keep + __shfl_xor_sync(FULL, give, w);
      }
    }
    float top = kNegInf;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      if (!((vis >> (token() + j)) & 1u)) x[j] = kNegInf;
      top = fmaxf(top, x[j]);
    }
    if (__any_sync(FULL, fmaf(top, c, -m) > kShift + kSlack)) {
#pragma unroll
      for (int w = 4 / NS; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, w));
      top = fmaxf(m, fmaf(top, c, -kShift));
      const float f = ex2(m - (top == kNegInf ? 0.f : top));
      m = top;
      l *= f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float fh = __shfl_sync(FULL, f, h * (LG / 2), LG);
#pragma unroll
        for (int i = 0; i < V4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) o[h][i][e] = Pair{o[h][i][e].x * fh, o[h][i][e].y * fh};
      }
    }
    const float u = m == kNegInf ? 0.f : m;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      p[j] = ex2(fmaf(x[j], c, -u));
      l += p[j];
    }
  }
  __device__ __forceinline__ void outputs(const char *vs) {
    const char *a0 = vs + lane() % LG * 16;
    float w[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < 8; ++t) w[h][t] = __shfl_sync(FULL, p[t % NS], (h * 8 + t) / NS, LG);
#pragma unroll
    for (int i = 0; i < V4; ++i) {
      if (i * LG * 4 >= dim) break;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        Pair v[2];
        lds4(v, a0 + t * PITCH + i * LG * 16);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) fma2(o[h][i][e], Pair{w[h][t], w[h][t]}, v[e]);
      }
    }
  }
  __device__ __forceinline__ void total() {
#pragma unroll
    for (int w = 4 / NS; w > 0; w >>= 1) l += __shfl_xor_sync(FULL, l, w);
  }
  __device__ __forceinline__ float4 part(int i) const {
    const Pair(&x)[2] = o[i / V4][i % V4];
    return make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
  }
  template <typename F>
  __device__ __forceinline__ void stats(F &&f) const {
    if (token() == 0) f(head(), m, l);
  }
  __device__ __forceinline__ static int head_of(int i, int ln, int) { return ln / LG * 2 + i / V4; }
  __device__ __forceinline__ static int col_of(int i, int ln, int e) {
    return (i % V4 * LG + ln % LG) * 4 + e;
  }
  __device__ __forceinline__ void finish(float *out, float *lse, int rows, int, float vs) {
    total();
    const float inv = l == 0.f ? 0.f : vs / l;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f = __shfl_sync(FULL, inv, h * (LG / 2), LG);
      if (f == 0.f)  // nothing was weighed: 0, whatever the values are
#pragma unroll
        for (int i = 0; i < V4; ++i) o[h][i][0] = o[h][i][1] = Pair{0.f, 0.f};
      const int row = lane() / LG * 2 + h;
#pragma unroll
      for (int i = 0; i < V4; ++i) {
        const int e = (i * LG + lane() % LG) * 4;
        if (row < rows && e < dim)
          *reinterpret_cast<float4 *>(out + row * dim + e) =
              make_float4(o[h][i][0].x * f, o[h][i][0].y * f, o[h][i][1].x * f, o[h][i][1].y * f);
      }
    }
    if (lse)
      stats([&](int h, float mh, float lh) {
        if (h < rows) lse[h] = log_sum(mh, lh);
      });
  }
};

// ---------------------------------------------------------------------------

// Lengths of the sequences within what the table can hold: those that fit lie
// in shared memory.
struct Lengths {
  const AttendArgs &a;
  const int *kept;
  int keep;
  __device__ __forceinline__ static int get(const AttendArgs &a, int b, bool &bad) {
    return cache_length(__ldg(a.s.lengths + b), a.s.table_width, a.p.page_size, bad);
  }
  __device__ __forceinline__ int operator()(int b) const {
    bool bad;
    return b < keep ? kept[b] : get(a, b, bad);
  }
};

// A tile's place on the line.
struct Cursor {
  int b, hr, tile;  // sequence, cached head * blocks + block, tile of the segment
  int left;         // tiles of the segment in the warp's piece, from this one on
  Span s;
  int64_t seg;      // first unit of the segment
  __device__ __forceinline__ void enter(const Lengths &len, int tile_tokens) {
    s = cache_span(len(b), len.a.window, tile_tokens);
  }
  // To the next segment, in a piece that ends before unit `end`.
  __device__ __forceinline__ void next_segment(const Lengths &len, int tile_tokens, int64_t end,
                                               int extra) {
    seg += (int64_t)s.count + extra;
    tile = left = 0;
    if (seg >= end) return;
    if (++hr == len.a.p.kv_heads * len.a.blocks) {
      hr = 0;
      ++b;
      enter(len, tile_tokens);
    }
    left = tiles_before(end - seg, s.count, extra);
  }
};

template <typename T>
__device__ __forceinline__ T to_out(float x);
template <>
__device__ __forceinline__ float to_out<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

template <typename TY, int WARPS, int UNITS>
struct Layout {
  static constexpr int kUnit = TY::TT * TY::PITCH;  // a tile's keys, or its values
  static constexpr int kRing = UNITS * kUnit, kWarp = kRing + TY::kQuery;
  static constexpr int kPart = TY::kParts * 128;  // floats of a part
  struct Side {
    long long before[WARPS * 32 + 1];  // tiles before each thread's sequences
    long long wsum[WARPS];
    long long last_seg[WARPS];  // first unit of the segment a warp ended in, or -1
    int4 last_at[WARPS];        // (sequence, head and block, the segment's last warp, begins)
    float2 last_ml[WARPS][TY::HEADS];  // of a warp; then, at a run's first warp, of the run
    float weight[WARPS][TY::HEADS];
    float end_weight[WARPS][TY::HEADS];
    int run_at[WARPS];
    int kept[WARPS * 32];         // lengths of the first sequences
    unsigned bits[WARPS][UNITS];  // visible tokens of the tile whose keys are there
  };
  static constexpr int kSmem = WARPS * kWarp + (int)sizeof(Side);
  static_assert(kRing >= kPart * 4, "a warp's sums fit its ring");
  static_assert(kWarp % 16 == 0 && kSmem <= 232448, "the shared memory that a CTA may have");
};

template <typename TY, int WARPS, int UNITS>
__global__ void __launch_bounds__(WARPS * 32, 1) k_attend(const __grid_constant__ AttendArgs a) {
  using L = Layout<TY, WARPS, UNITS>;
  using Out = typename TY::Out;
  constexpr int TT = TY::TT, ESZ = TY::ESZ, HEADS = TY::HEADS;
  extern __shared__ __align__(128) char smem[];
  typename L::Side &side = *reinterpret_cast<typename L::Side *>(smem + WARPS * L::kWarp);
  auto &before = side.before;
  auto &kept = side.kept;
  auto &bits = side.bits;
  auto &last_seg = side.last_seg;
  auto &last_at = side.last_at;
  auto &last_ml = side.last_ml;
  auto &weight = side.weight;
  auto &end_weight = side.end_weight;
  auto &run_at = side.run_at;

  static_assert(WARPS <= 16, "a half warp sums over the warps");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  char *ring = smem + warp * L::kWarp;
  const uint32_t ring_u = smem_u32(ring);

  if (a.p.dim < TY::DP) {  // elements behind the head's own: zeros, which no copy touches
    for (int i = lane; i < L::kRing / 16; i += 32)
      reinterpret_cast<uint4 *>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncwarp();
  }
  griddep_wait();
  griddep_launch();

  // ---- the line of units, and this warp's piece of it ---------------------
  const int chunk = (a.s.B + WARPS * 32 - 1) / (WARPS * 32);
  const int hrs = a.p.kv_heads * a.blocks;
  {
    long long mine = 0;
    for (int i = 0; i < chunk; ++i) {
      const int b = threadIdx.x * chunk + i;
      if (b >= a.s.B) break;
      bool bad;
      const int len = Lengths::get(a, b, bad);
      if (bad && blockIdx.x == 0 && a.errors) atomicOr(a.errors, (unsigned)FWPKM_CACHE_BAD_LENGTH);
      if (b < WARPS * 32) kept[b] = len;
      mine += cache_span(len, a.window, TT).count;
    }
    mine *= hrs;
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(FULL, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) side.wsum[warp] = sum;
    __syncthreads();
    long long base = lane < warp ? side.wsum[lane] : 0;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) base += __shfl_xor_sync(FULL, base, o);
    base = __shfl_sync(FULL, base, 0);
    before[threadIdx.x] = base + sum - mine;
    if (threadIdx.x == WARPS * 32 - 1) before[WARPS * 32] = base + sum;
    __syncthreads();
  }
  const Lengths lengths{a, kept, WARPS * 32};
  const long long tiles = before[WARPS * 32];
  const int extra = extra_units(tiles, gridDim.x * WARPS);
  const long long total = tiles + (long long)extra * a.s.B * hrs;
  // The segment that unit u < total falls into: its cursor, at tile 0.
  auto find = [&](long long u) {
    const long long seq_extra = (long long)extra * hrs;  // of a sequence's segments
    // the thread whose sequences u falls into: the last one with so many before it
    auto units = [&](int i) { return before[i] + seq_extra * min(i * chunk, a.s.B); };
    int i = 0;
    if (WARPS > 1) i = __popc(__ballot_sync(FULL, lane < WARPS && units(lane * 32) <= u)) - 1;
    i = i * 32 + __popc(__ballot_sync(FULL, units(i * 32 + lane) <= u)) - 1;
    Cursor c{};
    long long p = units(i);
    c.b = i * chunk;
    c.enter(lengths, TT);
    while (p + (long long)c.s.count * hrs + seq_extra <= u) {
      p += (long long)c.s.count * hrs + seq_extra;
      ++c.b;
      c.enter(lengths, TT);
    }
    const long long n = c.s.count + extra;
    c.hr = (int)((u - p) / n);
    c.seg = p + c.hr * n;
    return c;
  };
  // The line: of all units, its pieces dealt to the warps of all CTAs, or of the
  // CTA's own segments.  Piece 0 of it is that of warp `shift`; the first unit
  // is `base`.
  Line line;
  int per, shift;
  long long base;
  if (a.aligned) {
    const Line share = cut_line(total, gridDim.x);
    auto next_start = [&](long long u) {  // the first segment's start from unit u on
      if (u >= total) return total;
      const Cursor c = find(u);
      return c.seg == u ? u : c.seg + c.s.count + extra;
    };
    base = next_start(line_cut(share, blockIdx.x));
    const long long n = next_start(line_cut(share, blockIdx.x + 1)) - base;
    line = n > 0 ? piece_line(n, WARPS, extra) : Line{};
    per = WARPS;
    shift = blockIdx.x * WARPS;
  } else {
    line = piece_line(total, gridDim.x * WARPS, extra);
    per = max((line.warps + (int)gridDim.x - 1) / (int)gridDim.x, min(kLeastPerCta, WARPS));
    shift = 0;
    base = 0;
  }
  const int w0 = blockIdx.x * per, w = w0 + warp;
  const bool busy = warp < per && w - shift < line.warps;
  const long long u0 = busy ? base + line_cut(line, w - shift) : 0;
  const long long u1 = busy ? base + line_cut(line, w - shift + 1) : 0;
  auto owner = [&](long long unit) { return line_owner(line, unit - base) + shift; };

  Cursor at{};  // the tile that is computed; at.left == 0: none is left
  if (busy) {
    at = find(u0);
    at.tile = tile_from(u0 - at.seg, extra);
    at.left = tiles_before(u1 - at.seg, at.s.count, extra) - at.tile;
    if (at.tile >= at.s.count) at.next_segment(lengths, TT, u1, extra);  // behind its last
  }

  // the segment that the CTA's first warp is in the middle of: k_join's CTAs share it
  if (threadIdx.x == 0) {
    int4 id = make_int4(0, 0, -1, 0);
    if (at.left > 0 && at.tile > 0)
      id = make_int4(at.b, at.hr, owner(at.seg + tile_unit(at.s.count - 1, extra)),
                     owner(at.seg));
    a.middles[blockIdx.x] = id;
  }

  // ---- loads ---------------------------------------------------------------
  constexpr int CPR = TY::DP * ESZ / 16;    // 16-byte pieces of a padded row
  constexpr int kCopies = TT * CPR / 32;    // instructions a unit takes
  constexpr int kRows = CPR <= 32 ? 32 / CPR : 1;  // rows an instruction copies,
  constexpr int kSteps = CPR <= 32 ? 1 : CPR / 32;  // or instructions that a row takes
  const int cpr = a.p.dim * ESZ / 16;
  const bool packed = cpr == CPR && a.p.row_stride == TY::DP * ESZ;  // rows without gaps
  Cursor ld = at;  // the tile whose keys are loaded next
  int token = 0, page = -1;  // of this lane's row
  bool seen = false;
  auto look = [&] {
    token = (ld.s.first + ld.tile) * TT + (lane % TT);
    seen = token >= ld.s.lo && token < ld.s.len;
    page = seen ? __ldg(a.s.table + ld.b * a.s.table_stride + page_of(a.div, token)) : -1;
  };
  // this lane's 16 bytes of the first rows that one instruction copies
  const int64_t lane_off = (lane / CPR) * a.p.row_stride + (lane % CPR) * 16;
  const uint32_t lane_dst = ring_u + (lane / CPR) * TY::PITCH + (lane % CPR) * 16;
  int64_t off = 0;      // of this lane's row, or of its bytes where `even`
  unsigned vis = 0;     // visible tokens of the tile
  bool even = false;    // all visible, in one page: equal steps from the first row
  bool values = false;  // what comes next
  auto load = [&](int slot) {
    const char *pool = values ? a.p.values : a.p.keys;
    if (!values) {
      const bool ok = seen && (unsigned)page < (unsigned)a.p.pages;
      if (seen && !ok && a.errors && lane < TT) atomicOr(a.errors, (unsigned)FWPKM_CACHE_BAD_PAGE);
      vis = __ballot_sync(FULL, ok);
      if (lane == 0) bits[warp][slot] = vis;
      const int row = token - page_of(a.div, token) * a.p.page_size;
      const int first = __shfl_sync(FULL, row, 0);
      off = ok ? page * a.p.page_stride + (int64_t)(ld.hr / a.blocks) * a.p.head_stride +
                     (int64_t)row * a.p.row_stride
               : 0;
      even = vis == FULL && first + TT <= a.p.page_size;
      if (even) off = __shfl_sync(FULL, off, 0) + lane_off;
      // the next tile's pages are looked up while this one's values are loaded
      ++ld.tile;
      if (--ld.left == 0 && ld.tile == ld.s.count)
        ld.next_segment(lengths, TT, u1, extra);
      if (ld.left > 0) look();
    }
    if (even && packed) {
      const char *src = pool + off;
      const uint32_t dst = lane_dst + slot * L::kUnit;
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        cp_async16(dst + (i / kSteps) * kRows * TY::PITCH + (i % kSteps) * 512, src + i * 512);
    } else if (even) {
      const char *src = pool + off;
      const int64_t step = kRows * a.p.row_stride;
      const uint32_t dst = lane_dst + slot * L::kUnit;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        if (lane % CPR + (i % kSteps) * 32 < cpr)
          cp_async16(dst + (i / kSteps) * kRows * TY::PITCH + (i % kSteps) * 512,
                     src + (i % kSteps) * 512);
        if (i % kSteps == kSteps - 1) src += step;
      }
    } else {
      const uint32_t dst = ring_u + slot * L::kUnit;
#pragma unroll 2
      for (int i = 0; i < kCopies; ++i) {
        const int flat = i * 32 + lane, row = flat / CPR, c = flat % CPR;
        const int64_t ro = __shfl_sync(FULL, off, row) + c * 16;
        const bool ok = (vis >> row) & 1u;
        if (c < cpr) cp_async16(dst + row * TY::PITCH + c * 16, ok ? pool + ro : pool, ok);
      }
    }
  };
  if (ld.left > 0) look();
  auto advance = [&](int slot) {
    if (ld.left > 0 || values) {
      load(slot);
      values = !values;
    }
    cp_commit();
  };
#pragma unroll 1
  for (int i = 0; i < UNITS - 1; ++i) advance(i);

  // ---- the pass --------------------------------------------------------------
  TY ty;
  ty.qs = ring + L::kRing;
  ty.reset();
  int rows = 0;
  bool fresh = true, whole = at.tile == 0;
  auto park = [&](int slot) {
    ty.total();
    float4 *dst = reinterpret_cast<float4 *>(a.parts + (int64_t)slot * L::kPart) + lane;
#pragma unroll
    for (int i = 0; i < TY::kParts; ++i) dst[i * 32] = ty.part(i);
    ty.stats([&](int h, float m, float l) { a.ml[slot * HEADS + h] = make_float2(m, l); });
  };
  auto first_row = [&](int b, int hr) {
    return (int64_t)b * a.heads + (hr / a.blocks) * a.group + (hr % a.blocks) * HEADS;
  };

  int4 tail = make_int4(0, 0, -1, 0);
  bool open = false;  // a part is left in the registers,
  long long seg = 0;  // of the segment that begins at this unit
  int slot = 0;
  bool second = false;  // the tile's values are next
  while (at.left > 0) {
    if (fresh) {
      const int h = at.hr / a.blocks, first = (at.hr % a.blocks) * HEADS;
      rows = min(HEADS, a.group - first);
      ty.load_q(a.q + at.b * a.q_stride + (int64_t)(h * a.group + first) * a.p.dim * sizeof(Out),
                rows, a.p.dim, a.scale_log2 * (a.p.key_scale ? __ldg(a.p.key_scale + h) : 1.f));
      fresh = false;
    }
    cp_wait<UNITS - 2>();
    __syncwarp();  // the unit has landed, and the one before it is free
    advance(slot == 0 ? UNITS - 1 : slot - 1);
    const char *src = ring + slot * L::kUnit;
    if (!second) {
      ty.scores(src, bits[warp][slot]);
    } else {
      ty.outputs(src);
      open = true;
      ++at.tile;
      if (--at.left == 0) {  // the segment or the piece ends
        const int b = at.b, hr = at.hr, count = at.s.count;
        const bool end = at.tile == count;
        seg = at.seg;
        if (end) {
          at.next_segment(lengths, TT, u1, extra);
          if (whole) {
            const int64_t r = first_row(b, hr);
            ty.finish(reinterpret_cast<Out *>(a.out) + r * a.p.dim, a.lse ? a.lse + r : nullptr,
                      rows, a.p.dim, a.p.value_scale ? __ldg(a.p.value_scale + hr / a.blocks) : 1.f);
            open = false;
          } else if (at.left > 0) {
            park(2 * w);
            open = false;
          }
          if (at.left > 0) {
            ty.reset();
            fresh = whole = true;
          }
        }
        if (at.left == 0 && open) {  // what is left is joined with the CTA's other warps'
          const int last = owner(seg + tile_unit(count - 1, extra));
          if (lane == 0) last_at[warp] = make_int4(b, hr, last, whole);
          if (whole && !end) tail = make_int4(b, hr, last, 0);
        }
      }
    }
    second = !second;
    slot = slot + 1 == UNITS ? 0 : slot + 1;
  }

  // ---- the warps' last parts, joined where they are of one segment -------------
  if (lane == 0) last_seg[warp] = open ? seg : -1;
  if (open) {
    ty.total();
    __syncwarp();  // every lane has read its last tile from the ring
    float4 *mine = reinterpret_cast<float4 *>(ring) + lane;
#pragma unroll
    for (int i = 0; i < TY::kParts; ++i) mine[i * 32] = ty.part(i);
    ty.stats([&](int h, float m, float l) { last_ml[warp][h] = make_float2(m, l); });
  }
  tail.w = per;
  if (lane == 0) a.tails[blockIdx.x * WARPS + warp] = tail;
  if (!__syncthreads_or(open)) return;
  // A run is the neighbouring warps whose last parts are of one segment; its
  // first warp's slot takes its sum.  Bit k of `heads`: warp k begins a run.
  // A run that begins its segment takes in what the warp behind it has parked of
  // that segment, which is then done.
  const long long my_seg = lane < WARPS ? last_seg[lane] : -1;
  const long long left = __shfl_up_sync(FULL, my_seg, 1);
  const unsigned live = __ballot_sync(FULL, my_seg >= 0);
  const unsigned heads = __ballot_sync(FULL, my_seg >= 0 && (lane == 0 || left != my_seg));
  if (warp == 0 && (heads >> lane) & 1u) run_at[__popc(heads & lanemask_lt())] = lane;
  auto run_end = [&](int k0) {  // behind the run that begins at warp k0
    const unsigned stop = (~live | heads) & (0xfffffffeu << k0);
    return min(__ffs(stop | 1u << WARPS) - 1, WARPS);
  };
  for (int i = threadIdx.x; i < WARPS * HEADS; i += WARPS * 32) {
    const int k0 = i / HEADS, h = i % HEADS;
    if (!((heads >> k0) & 1u)) continue;
    const int k1 = run_end(k0);
    const int4 id = last_at[k0];
    const bool more = id.w && id.z == w0 + k1 && k1 < per;
    float2 end = make_float2(kNegInf, 0.f);
    if (more) end = a.ml[2 * id.z * HEADS + h];
    float top = end.x, l = 0.f;
    for (int k = k0; k < k1; ++k) top = fmaxf(top, last_ml[k][h].x);
    const float u = top == kNegInf ? 0.f : top;
    for (int k = k0; k < k1; ++k) {
      const float2 ml = last_ml[k][h];
      const float f = ex2(ml.x - u);
      weight[k][h] = f;
      l = fmaf(ml.y, f, l);
    }
    const float f = ex2(end.x - u);
    l = fmaf(end.y, f, l);
    last_ml[k0][h] = make_float2(top, l);
    end_weight[k0][h] = more ? f : 0.f;
  }
  __syncthreads();
  const int runs = __popc(heads);
  for (int p = threadIdx.x; p < runs * TY::kParts * 32; p += WARPS * 32) {
    const int k0 = run_at[p / (TY::kParts * 32)];
    const int q = p % (TY::kParts * 32), i = q >> 5, ln = q & 31;
    const int k1 = run_end(k0);
    const int4 id = last_at[k0];
    const bool begins = id.w, more = begins && id.z == w0 + k1 && k1 < per;
    const bool done = begins && (more || id.z < w0 + k1);
    const int h0 = id.y / a.blocks, block = id.y % a.blocks;
    const int n = min(HEADS, a.group - block * HEADS);
    const int to = 2 * (w0 + k0) + (begins ? 1 : 0);
    int h[4];
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = TY::head_of(i, ln, e);
    float4 end;
    if (more) end = reinterpret_cast<const float4 *>(a.parts + (int64_t)(2 * id.z) * L::kPart)[q];
#pragma unroll 4
    for (int k = k0; k < k1; ++k) {
      const float4 v = reinterpret_cast<const float4 *>(smem + k * L::kWarp)[q];
      x[0] = fmaf(v.x, weight[k][h[0]], x[0]);
      x[1] = fmaf(v.y, weight[k][h[1]], x[1]);
      x[2] = fmaf(v.z, weight[k][h[2]], x[2]);
      x[3] = fmaf(v.w, weight[k][h[3]], x[3]);
    }
    if (more) {
      x[0] = fmaf(end.x, end_weight[k0][h[0]], x[0]);
      x[1] = fmaf(end.y, end_weight[k0][h[1]], x[1]);
      x[2] = fmaf(end.z, end_weight[k0][h[2]], x[2]);
      x[3] = fmaf(end.w, end_weight[k0][h[3]], x[3]);
    }
    if (done) {
      const int64_t r = first_row(id.x, id.y);
      const float vs = a.p.value_scale ? __ldg(a.p.value_scale + h0) : 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = TY::col_of(i, ln, e);
        const float2 ml = last_ml[k0][h[e]];
        if (h[e] < n && c < a.p.dim)
          reinterpret_cast<Out *>(a.out)[(r + h[e]) * a.p.dim + c] =
              to_out<Out>(ml.y == 0.f ? 0.f : x[e] * (vs / ml.y));
        if (a.lse && h[e] < n && c == 0) a.lse[r + h[e]] = log_sum(ml.x, ml.y);
      }
      if (q == 0) a.tails[blockIdx.x * WARPS + k0].z = -1;
    } else {
      reinterpret_cast<float4 *>(a.parts + (int64_t)to * L::kPart)[q] =
          make_float4(x[0], x[1], x[2], x[3]);
      if (q < HEADS) {
        a.ml[to * HEADS + q] = last_ml[k0][q];
        // the slot that k_join may look for at the run's last warp holds nothing
        if (k1 - k0 > 1) a.ml[2 * (w0 + k1 - 1) * HEADS + q] = make_float2(kNegInf, 0.f);
      }
    }
  }
}

// Joins the parts of segments that lie in more than one CTA's slots.  The CTAs whose
// warps have a part share a segment's groups of 32 x 4 floats out; a group with
// few parts is one warp's, one with many is summed by all warps of the CTA.
constexpr int kJoinWarps = 16, kJoinFew = 6;
template <typename TY, int WARPS>
__global__ void __launch_bounds__(kJoinWarps * 32) k_join(const __grid_constant__ AttendArgs a) {
  using Out = typename TY::Out;
  constexpr int HEADS = TY::HEADS, kPart = TY::kParts * 128;
  __shared__ float sum[kJoinWarps][12][32];  // of each warp and lane: m, l and x of 4 floats
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch();
  // lane i: the segment that begins in warp i; lane 31: the one that goes on here
  const int cta = blockIdx.x;
  int4 mine = make_int4(0, 0, -1, 0);
  if (lane < WARPS) mine = a.tails[cta * WARPS + lane];
  else if (lane == 31) mine = a.middles[cta];
  const int per = __shfl_sync(FULL, mine.w, 0);
  if (lane < WARPS) mine.w = cta * per + lane;
  unsigned left = __ballot_sync(FULL, mine.z >= 0);
  int turn = 0;  // single-warp groups dealt out so far
  for (; left; left &= left - 1) {
    const int from = __ffs(left) - 1;
    const int b = __shfl_sync(FULL, mine.x, from), hr = __shfl_sync(FULL, mine.y, from);
    const int last = __shfl_sync(FULL, mine.z, from), w = __shfl_sync(FULL, mine.w, from);
    const int c0 = w / per, c1 = last / per;
    // parts: the first warp's; the first warp's of each later CTA; the last warp's
    const int n = 1 + c1 - c0 + (last % per != 0);
    const int h0 = hr / a.blocks, block = hr % a.blocks;
    const int rows = min(HEADS, a.group - block * HEADS);
    const int64_t r = (int64_t)b * a.heads + h0 * a.group + block * HEADS;
    const float vs = a.p.value_scale ? __ldg(a.p.value_scale + h0) : 1.f;
    const bool many = n > kJoinFew;
    for (int i = cta - c0; i < TY::kParts; i += c1 - c0 + 1) {
      if (!many && turn++ % kJoinWarps != warp) continue;
      int h[4];
      float top[4], x[4] = {0.f, 0.f, 0.f, 0.f}, l[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[e] = TY::head_of(i, lane, e);
        top[e] = kNegInf;
      }
      const int dk = many ? kJoinWarps : 1;
      for (int kb = many ? warp : 0; kb < n; kb += 4 * dk) {  // four parts at a time
        float2 ml[4][4];
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = kb + j * dk;
          if (k < n) {
            const int slot = k == 0 ? 2 * w + 1 : k <= c1 - c0 ? 2 * (c0 + k) * per : 2 * last;
#pragma unroll
            for (int e = 0; e < 4; ++e) ml[j][e] = a.ml[slot * HEADS + h[e]];
            v[j] = reinterpret_cast<const float4 *>(a.parts + (int64_t)slot * kPart)[i * 32 + lane];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) ml[j][e] = make_float2(kNegInf, 0.f);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float t = top[e];
#pragma unroll
          for (int j = 0; j < 4; ++j) t = fmaxf(t, ml[j][e].x);
          const float u = t == kNegInf ? 0.f : t, f = ex2(top[e] - u);
          top[e] = t;
          l[e] *= f;
          x[e] *= f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float g = ex2(ml[j][e].x - u);
            l[e] = fmaf(ml[j][e].y, g, l[e]);
            // an empty slot's sums are not set
            if (ml[j][e].y != 0.f)
              x[e] = fmaf(e == 0 ? v[j].x : e == 1 ? v[j].y : e == 2 ? v[j].z : v[j].w, g, x[e]);
          }
        }
      }
      if (many) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[warp][e][lane] = top[e];
          sum[warp][4 + e][lane] = l[e];
          sum[warp][8 + e][lane] = x[e];
        }
        __syncthreads();
        if (warp < 4) {  // warp e: float e
          const int e = warp;
          float t = kNegInf, xe = 0.f, le = 0.f;
#pragma unroll
          for (int k = 0; k < kJoinWarps; ++k) t = fmaxf(t, sum[k][e][lane]);
          const float u = t == kNegInf ? 0.f : t;
#pragma unroll
          for (int k = 0; k < kJoinWarps; ++k) {
            const float f = ex2(sum[k][e][lane] - u);
            le = fmaf(sum[k][4 + e][lane], f, le);
            xe = fmaf(sum[k][8 + e][lane], f, xe);
          }
          const int he = TY::head_of(i, lane, e), c = TY::col_of(i, lane, e);
          if (he < rows) {
            if (c < a.p.dim)
              reinterpret_cast<Out *>(a.out)[(r + he) * a.p.dim + c] =
                  to_out<Out>(le == 0.f ? 0.f : xe * (vs / le));
            if (a.lse && c == 0) a.lse[r + he] = log_sum(t, le);
          }
        }
        __syncthreads();
        continue;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = TY::col_of(i, lane, e);
        if (h[e] >= rows) continue;
        if (c < a.p.dim)
          reinterpret_cast<Out *>(a.out)[(r + h[e]) * a.p.dim + c] =
              to_out<Out>(l[e] == 0.f ? 0.f : x[e] * (vs / l[e]));
        if (a.lse && c == 0) a.lse[r + h[e]] = log_sum(top[e], l[e]);
      }
    }
  }
}

// Attributes of the kernels, set once a device.  k_join asks for the shared
// memory split that k_attend runs with: a multiprocessor changes its split only
// when it is idle, which would keep the join from starting early.
template <typename TY, int WARPS, int UNITS>
cudaError_t prepare() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(k_attend<TY, WARPS, UNITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Layout<TY, WARPS, UNITS>::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_attend<TY, WARPS, UNITS>,
                             cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_join<TY, WARPS>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <typename TY, int WARPS, int UNITS>
cudaError_t launch(AttendArgs a, cudaStream_t st) {
  cudaError_t e = prepare<TY, WARPS, UNITS>();
  if (e != cudaSuccess) return e;
  const AttendShape s = attend_shape(TY::kDtype, a.p.dim, a.group);
  if (s.warps != WARPS || s.heads != TY::HEADS || s.part != TY::kParts * 128)
    return cudaErrorInvalidConfiguration;  // the workspace has another layout
  a.blocks = (a.group + TY::HEADS - 1) / TY::HEADS;
  // Where no segment can have more than four tiles for each of a CTA's warps, a CTA
  // takes whole ones and the second kernel falls away.  In a graph, whole and divided
  // (bf16 heads of 128): 64 tokens of 8 cached heads 10.4 us and 12.4, 300 sequences
  // of 64 tokens and one head 12.6 and 15.8, 256 ragged ones of up to 704 and 4 heads
  // 53.6 and 54.9.  What it loses is where a few segments of that length meet idle
  // CTAs, or somewhat more of them than CTAs: one sequence of 736 tokens 16.7 and
  // 14.7, 148, 160 and 300 segments of it 20.8 and 21.9, 27.0 and 25.4, 35.0 and 34.9.
  // As calls of their own, small ones gain the second launch's host time (one of 512:
  // 15.4 and 16.8).  Beyond the limit, one sequence of 2048 would take 29 and 12.6.
  a.aligned = a.tokens / TY::TT + 2 <= 4 * WARPS;
  e = launch_k(true, k_attend<TY, WARPS, UNITS>, dim3(kAttendCtas), dim3(WARPS * 32),
               Layout<TY, WARPS, UNITS>::kSmem, st, a);
  if (e != cudaSuccess) return e;
  if (a.aligned) return cudaSuccess;  // each CTA finishes its segments
  return launch_k(true, k_join<TY, WARPS>, dim3(kAttendCtas), dim3(kJoinWarps * 32), 0,
                  st, a);
}

}  // namespace attend
}  // namespace fwpkm
