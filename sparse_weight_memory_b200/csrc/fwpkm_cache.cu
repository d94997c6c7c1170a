// fwpkm_cache.cu -- host side of the paged key-value cache's C ABI
// (include/fwpkm_cache.h): argument checks, then the launches.  Nothing is
// allocated, kept or synchronised.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "fwpkm_cache_internal.cuh"

using namespace fwpkm;

namespace {

fwpkm_status fail(fwpkm_status st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

int elem_size(int dtype) { return dtype == FWPKM_F32 ? 4 : dtype == FWPKM_BF16 ? 2 : 1; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

constexpr int64_t kMaxRows = 1ll << 22;   // B * heads
constexpr int kMaxHeads = 4096, kMaxKvHeads = 1024;
constexpr int64_t kMaxStride = 1ll << 40;  // elements

// What both calls and the workspace size need of the cache.
fwpkm_status check_kind(const char *who, const fwpkm_cache *c) {
  if (!c) return fail(FWPKM_EINVAL, "%s: cache is NULL", who);
  if (c->dtype != FWPKM_F32 && c->dtype != FWPKM_BF16 && c->dtype != FWPKM_E4M3)
    return fail(FWPKM_EINVAL, "%s: cache dtype must be FWPKM_F32, FWPKM_BF16 or FWPKM_E4M3", who);
  const int unit = c->dtype == FWPKM_E4M3 ? 16 : 8;
  if (c->dim < unit || c->dim > FWPKM_CACHE_MAX_DIM || c->dim % unit)
    return fail(FWPKM_ESHAPE, "%s: dim=%d must be a multiple of %d, %d .. %d", who, c->dim, unit,
                unit, FWPKM_CACHE_MAX_DIM);
  if (c->kv_heads < 1 || c->kv_heads > kMaxKvHeads)
    return fail(FWPKM_ESHAPE, "%s: kv_heads=%d must be 1 .. %d", who, c->kv_heads, kMaxKvHeads);
  return FWPKM_OK;
}

fwpkm_status check_pool(const char *who, const fwpkm_cache *c, CachePool *p) {
  fwpkm_status rc = check_kind(who, c);
  if (rc) return rc;
  if (!c->keys || !c->values) return fail(FWPKM_EINVAL, "%s: keys or values is NULL", who);
  if (!aligned16(c->keys) || !aligned16(c->values))
    return fail(FWPKM_EINVAL, "%s: keys and values must be 16-byte aligned", who);
  if (c->pages < 1 || c->pages > 0x7fffffffll)
    return fail(FWPKM_ESHAPE, "%s: pages=%lld must be 1 .. 2^31 - 1", who, (long long)c->pages);
  if (c->page_size < 1) return fail(FWPKM_ESHAPE, "%s: page_size must be >= 1", who);
  const int es = elem_size(c->dtype);
  const int64_t strides[3] = {c->page_stride, c->head_stride, c->row_stride};
  const int64_t counts[3] = {c->pages, c->kv_heads, c->page_size};
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0 || strides[i] > kMaxStride || (strides[i] * es) % 16)
      return fail(FWPKM_ESHAPE, "%s: strides must be 0 .. 2^40 elements and whole 16-byte units",
                  who);
    // the pool's last byte must have a 63-bit offset
    if (strides[i] && (counts[i] - 1) > ((1ll << 60) / es) / strides[i])
      return fail(FWPKM_ESHAPE, "%s: the pool's strides reach beyond 2^60 bytes", who);
  }
  if ((c->key_scale || c->value_scale) && c->dtype != FWPKM_E4M3)
    return fail(FWPKM_EINVAL, "%s: only an FWPKM_E4M3 cache has scales", who);
  if (!aligned4(c->key_scale) || !aligned4(c->value_scale))
    return fail(FWPKM_EINVAL, "%s: scales must be 4-byte aligned", who);
  p->keys = static_cast<char *>(c->keys);
  p->values = static_cast<char *>(c->values);
  p->page_stride = c->page_stride * es;
  p->head_stride = c->head_stride * es;
  p->row_stride = c->row_stride * es;
  p->key_scale = c->key_scale;
  p->value_scale = c->value_scale;
  p->pages = (int)c->pages;
  p->page_size = c->page_size;
  p->kv_heads = c->kv_heads;
  p->dim = c->dim;
  return FWPKM_OK;
}

fwpkm_status check_batch(const char *who, const fwpkm_cache_batch *b, CacheBatch *s) {
  if (!b) return fail(FWPKM_EINVAL, "%s: batch is NULL", who);
  if (b->B < 1 || b->B > kMaxRows) return fail(FWPKM_ESHAPE, "%s: B must be 1 .. 2^22", who);
  if (b->table_width < 1) return fail(FWPKM_ESHAPE, "%s: table_width must be >= 1", who);
  if (b->table_stride < 0 || b->table_stride > kMaxStride)
    return fail(FWPKM_ESHAPE, "%s: table_stride must be 0 .. 2^40", who);
  if (!b->table || !b->lengths) return fail(FWPKM_EINVAL, "%s: table or lengths is NULL", who);
  if (!aligned4(b->table) || !aligned4(b->lengths))
    return fail(FWPKM_EINVAL, "%s: table and lengths must be 4-byte aligned", who);
  s->table = b->table;
  s->lengths = b->lengths;
  s->table_stride = b->table_stride;
  s->B = b->B;
  s->table_width = b->table_width;
  return FWPKM_OK;
}

// Rows of `stride` elements holding `width` of them each.
fwpkm_status check_rows(const char *who, const char *what, const void *p, int64_t stride,
                        int64_t width, int es, int64_t rows) {
  if (!p) return fail(FWPKM_EINVAL, "%s: %s is NULL", who, what);
  if (!aligned16(p)) return fail(FWPKM_EINVAL, "%s: %s must be 16-byte aligned", who, what);
  if ((rows > 1 && stride < width) || stride < 0 || stride > kMaxStride || (stride * es) % 16)
    return fail(FWPKM_ESHAPE, "%s: the row stride of %s must be at least a row and whole 16-byte "
                "units", who, what);
  return FWPKM_OK;
}

}  // namespace

extern "C" fwpkm_status fwpkm_cache_append(const fwpkm_cache *cache,
                                           const fwpkm_cache_batch *batch, int rows, int in_dtype,
                                           const void *k, int64_t k_stride, const void *v,
                                           int64_t v_stride, const void *q, int64_t q_stride,
                                           void *q_out, int64_t q_out_stride, int heads,
                                           const int32_t *starts, int rotary, int style,
                                           const float *freqs, uint32_t *device_errors,
                                           void *stream) {
  const char *who = "cache_append";
  AppendArgs a{};
  fwpkm_status rc = check_pool(who, cache, &a.p);
  if (rc) return rc;
  if ((rc = check_batch(who, batch, &a.s))) return rc;
  if (in_dtype != FWPKM_F32 && in_dtype != FWPKM_BF16)
    return fail(FWPKM_EINVAL, "%s: in_dtype must be FWPKM_F32 or FWPKM_BF16", who);
  if (rows < 0) return fail(FWPKM_ESHAPE, "%s: rows must be >= 0", who);
  if (!starts && rows != a.s.B)
    return fail(FWPKM_ESHAPE, "%s: without starts there is one row a sequence (rows=%d, B=%d)",
                who, rows, a.s.B);
  if (rotary < 0 || rotary > a.p.dim || rotary % 16)
    return fail(FWPKM_ESHAPE, "%s: rotary=%d must be a multiple of 16 up to dim=%d", who, rotary,
                a.p.dim);
  if (style != FWPKM_ROTATE_HALVES && style != FWPKM_ROTATE_PAIRS)
    return fail(FWPKM_EINVAL, "%s: style must be FWPKM_ROTATE_HALVES or FWPKM_ROTATE_PAIRS", who);
  if (rotary && !freqs) return fail(FWPKM_EINVAL, "%s: freqs is NULL", who);
  if (!aligned4(starts) || !aligned4(freqs) || !aligned4(device_errors))
    return fail(FWPKM_EINVAL, "%s: starts, freqs and device_errors must be 4-byte aligned", who);
  if ((q == nullptr) != (q_out == nullptr))
    return fail(FWPKM_EINVAL, "%s: q and q_out must both be given, or neither", who);
  if (q && (heads < 1 || heads > kMaxHeads))
    return fail(FWPKM_ESHAPE, "%s: heads=%d must be 1 .. %d", who, heads, kMaxHeads);
  if (rows == 0) return FWPKM_OK;
  const int es = elem_size(in_dtype);
  const int64_t kv_width = (int64_t)a.p.kv_heads * a.p.dim;
  if ((rc = check_rows(who, "k", k, k_stride, kv_width, es, rows))) return rc;
  if ((rc = check_rows(who, "v", v, v_stride, kv_width, es, rows))) return rc;
  if (q) {
    const int64_t width = (int64_t)heads * a.p.dim;
    if ((rc = check_rows(who, "q", q, q_stride, width, es, rows))) return rc;
    if ((rc = check_rows(who, "q_out", q_out, q_out_stride, width, es, rows))) return rc;
    if (q == q_out && q_stride != q_out_stride)
      return fail(FWPKM_EINVAL, "%s: q_out at q's place needs q's stride", who);
  }
  a.k = static_cast<const char *>(k);
  a.v = static_cast<const char *>(v);
  a.q = static_cast<const char *>(q);
  a.q_out = static_cast<char *>(q_out);
  a.k_stride = k_stride * es;
  a.v_stride = v_stride * es;
  a.q_stride = q_stride * es;
  a.q_out_stride = q_out_stride * es;
  a.starts = starts;
  a.freqs = freqs;
  a.errors = device_errors;
  a.rows = rows;
  a.heads = q ? heads : 0;
  a.rotary = rotary;
  a.pairs = style == FWPKM_ROTATE_PAIRS;
  const cudaError_t e =
      launch_cache_append(a, in_dtype, cache->dtype, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess)
    return fail(FWPKM_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return FWPKM_OK;
}

// More warps hide more latency, as long as the outputs and queries of a
// segment's heads fit their registers.  One cached head for 8 query heads, in
// sequences of up to 40435 tokens, rings as deep as the shared memory allows: bf16
// heads of 128 (1.03 GB) on 8, 10, 12 and 16 warps 191, 191, 185 and 191 us; of 64
// (0.78 GB) 148, 148, 144 and 142; e4m3 heads of 128 (0.78 GB) 145, 163, 150 and,
// with spills, 438; of 256 (0.83 GB) on 8 166 and, with spills, on 12 533.
// More than 8 query heads to a cached one are one segment of 16 or 32, since every
// further segment reads the cached head again, unless that spills so much that two
// segments take less: 32 heads to a cached e4m3 one of 128 (0.78 GB) 730 us as one
// segment, 372 as two, 16 to one of 256 (0.83 GB) 640 and 312; 32 to one of 64
// (0.39 GB) 202 as one and 217 as two.
fwpkm::AttendShape fwpkm::attend_shape(int cache_dtype, int dim, int group) {
  const int dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  if (cache_dtype == FWPKM_F32) {
    const int heads = group <= 4 ? 4 : group <= 8 || dp == 256 ? 8 : 16;
    const int warps = heads == 16 || dp == 256 ? 8 : dp == 64 ? 16 : 12;
    return {warps, heads, heads * dp};
  }
  const bool e4m3 = cache_dtype == FWPKM_E4M3;
  const int most = !e4m3 ? (dp == 256 ? 16 : 32) : dp == 64 ? 32 : dp == 128 ? 16 : 8;
  const int heads = group <= 8 || most == 8 ? 8 : group <= 16 || most == 16 ? 16 : 32;
  int warps = 16;
  if (dp * heads >= 128 * 16 || (dp == 128 && e4m3)) warps = 8;
  else if (dp == 128 || heads > 8) warps = 12;
  return {warps, heads, heads * dp};
}

namespace {

// The workspace: parts, their (m, l), the tails and middles.
struct Workspace {
  int64_t ml, tails, middles, bytes;
};
Workspace layout(int cache_dtype, int dim, int group) {
  const AttendShape s = attend_shape(cache_dtype, dim, group);
  const int64_t warps = (int64_t)kAttendCtas * s.warps;
  Workspace w;
  w.ml = 2 * warps * s.part * (int64_t)sizeof(float);
  w.tails = w.ml + 2 * warps * s.heads * (int64_t)sizeof(float2);
  w.middles = w.tails + warps * (int64_t)sizeof(int4);
  w.bytes = w.middles + kAttendCtas * (int64_t)sizeof(int4);
  return w;
}

fwpkm_status check_heads(const char *who, const fwpkm_cache *c, int B, int heads) {
  if (B < 1) return fail(FWPKM_ESHAPE, "%s: B must be >= 1", who);
  if (heads < 1 || heads > kMaxHeads || heads % c->kv_heads)
    return fail(FWPKM_ESHAPE, "%s: heads=%d must be a multiple of kv_heads=%d, up to %d", who,
                heads, c->kv_heads, kMaxHeads);
  if ((int64_t)B * heads > kMaxRows)
    return fail(FWPKM_ESHAPE, "%s: B * heads = %lld must be <= 2^22", who, (long long)B * heads);
  return FWPKM_OK;
}

}  // namespace

extern "C" int64_t fwpkm_cache_attend_workspace(const fwpkm_cache *cache, int B, int heads) {
  const char *who = "cache_attend_workspace";
  fwpkm_status rc = check_kind(who, cache);
  if (rc == FWPKM_OK) rc = check_heads(who, cache, B, heads);
  return rc ? (int64_t)rc : layout(cache->dtype, cache->dim, heads / cache->kv_heads).bytes;
}

extern "C" fwpkm_status fwpkm_cache_attend(const fwpkm_cache *cache,
                                           const fwpkm_cache_batch *batch, int heads, int q_dtype,
                                           const void *q, int64_t q_stride, float scale,
                                           int window, void *out, float *lse, void *workspace,
                                           int64_t workspace_bytes, uint32_t *device_errors,
                                           void *stream) {
  const char *who = "cache_attend";
  AttendArgs a{};
  fwpkm_status rc = check_pool(who, cache, &a.p);
  if (rc) return rc;
  if ((rc = check_batch(who, batch, &a.s))) return rc;
  if ((rc = check_heads(who, cache, a.s.B, heads))) return rc;
  if (q_dtype != FWPKM_F32 && q_dtype != FWPKM_BF16)
    return fail(FWPKM_EINVAL, "%s: q_dtype must be FWPKM_F32 or FWPKM_BF16", who);
  if ((q_dtype == FWPKM_F32) != (cache->dtype == FWPKM_F32))
    return fail(FWPKM_EUNSUPPORTED, "%s: an FWPKM_F32 cache takes FWPKM_F32 queries, the others "
                "FWPKM_BF16 ones", who);
  const int es = elem_size(q_dtype);
  if ((rc = check_rows(who, "q", q, q_stride, (int64_t)heads * a.p.dim, es, a.s.B))) return rc;
  if (!out || !aligned16(out))
    return fail(FWPKM_EINVAL, "%s: out must be given and 16-byte aligned", who);
  if (out == q) return fail(FWPKM_EINVAL, "%s: out must not be q", who);
  if (!aligned4(lse) || !aligned4(device_errors))
    return fail(FWPKM_EINVAL, "%s: lse and device_errors must be 4-byte aligned", who);
  const float scale_log2 = scale * 1.4426950408889634f;  // scores in base 2
  if (!std::isfinite(scale_log2))
    return fail(FWPKM_EINVAL, "%s: scale must be finite, and times log2(e) too", who);
  if (window < 0) return fail(FWPKM_EINVAL, "%s: window must be >= 0", who);
  const Workspace w = layout(cache->dtype, cache->dim, heads / cache->kv_heads);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < w.bytes)
    return fail(FWPKM_EINVAL, "%s: workspace must be 256-byte aligned and hold %lld bytes", who,
                (long long)w.bytes);
  char *ws = static_cast<char *>(workspace);
  a.q = static_cast<const char *>(q);
  a.q_stride = q_stride * es;
  a.out = static_cast<char *>(out);
  a.lse = lse;
  a.parts = reinterpret_cast<float *>(ws);
  a.ml = reinterpret_cast<float2 *>(ws + w.ml);
  a.tails = reinterpret_cast<int4 *>(ws + w.tails);
  a.middles = reinterpret_cast<int4 *>(ws + w.middles);
  a.errors = device_errors;
  a.scale_log2 = scale_log2;
  a.heads = heads;
  a.group = heads / a.p.kv_heads;
  a.window = window;
  a.div = page_div(a.p.page_size);
  a.tokens = (int64_t)a.s.table_width * a.p.page_size;
  if (window > 0 && window < a.tokens) a.tokens = window;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == FWPKM_F32    ? launch_cache_attend_f32(a, st)
                        : cache->dtype == FWPKM_BF16 ? launch_cache_attend_bf16(a, st)
                                                     : launch_cache_attend_e4m3(a, st);
  if (e != cudaSuccess)
    return fail(FWPKM_ECUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return FWPKM_OK;
}
