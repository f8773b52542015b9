// C ABI of the paged key/value cache operators: argument validation, choice of
// the kernel family, launch.  Declarations and the meaning of every argument:
// include/sdpa.h.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>

#include "paged.cuh"

namespace sdpa {
namespace {

constexpr long long kMaxStride = 1LL << 40;
// tokens of a sequence and rows of a batch: positions less a window stay inside 32 bits
constexpr long long kMaxTokens = 1LL << 30;

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t cache_esz(int dtype) { return dtype == SDPA_CACHE_F32 ? 4 : dtype == SDPA_CACHE_BF16 ? 2 : 1; }
bool is_codes(int dtype) { return dtype == SDPA_CACHE_E4M3 || dtype == SDPA_CACHE_INT8; }
bool stride_ok(const sdpa_strides_t& s) {
  return s.b >= 1 && s.h >= 1 && s.t >= 1 && s.b <= kMaxStride && s.h <= kMaxStride && s.t <= kMaxStride;
}
bool stride_ok(const sdpa_rows_t& s) { return s.t >= 1 && s.h >= 1 && s.t <= kMaxStride && s.h <= kMaxStride; }

// Addresses [lo, hi) of a tensor; lo > hi: it does not end inside the address space.
struct Span {
  uintptr_t lo, hi;
  bool fits() const { return lo <= hi; }
};
// Strides go to 2^40 and extents to 2^31: counted in 128 bits.
Span span_of(const void* p, __int128 elems, size_t esz) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (p == nullptr || elems <= 0) return {a, a};
  const __int128 end = (__int128)a + elems * (__int128)esz;
  return end > (__int128)INT64_MAX ? Span{1, 0} : Span{a, (uintptr_t)end};
}
bool meet(const Span& a, const Span& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
__int128 last3(const sdpa_strides_t& s, long long nb, long long nh, long long nt, long long d) {
  return nb <= 0 || nh <= 0 || nt <= 0 ? 0 : (__int128)(nb - 1) * s.b + (__int128)(nh - 1) * s.h + (__int128)(nt - 1) * s.t + d;
}
__int128 last2(const sdpa_rows_t& s, long long nt, long long nh, long long d) {
  return nt <= 0 || nh <= 0 ? 0 : (__int128)(nt - 1) * s.t + (__int128)(nh - 1) * s.h + d;
}

// What a cache occupies: pages, and the scales of codes.
struct CacheSpans {
  Span part[4];
  bool fits() const { return part[0].fits() && part[1].fits() && part[2].fits() && part[3].fits(); }
  bool meets(const Span& s) const { return meet(s, part[0]) || meet(s, part[1]) || meet(s, part[2]) || meet(s, part[3]); }
};
CacheSpans spans_of(const sdpa_cache_t& c) {
  auto axis = [&](const void* p, const sdpa_strides_t& st, long long d, size_t esz) {
    return span_of(p, last3(st, c.num_pages, c.Hkv, c.page_size, d), esz);
  };
  const bool codes = is_codes(c.dtype);
  return {{axis(c.k, c.k_strides, c.d, cache_esz(c.dtype)), axis(c.v, c.v_strides, c.d, cache_esz(c.dtype)),
           axis(codes ? c.k_scale : nullptr, c.k_scale_strides, 1, 4),
           axis(codes ? c.v_scale : nullptr, c.v_scale_strides, 1, 4)}};
}
// What the kernels read of a batch.
struct BatchSpans {
  Span part[3];
  bool fits() const { return part[0].fits() && part[1].fits() && part[2].fits(); }
  bool meets(const Span& s) const { return meet(s, part[0]) || meet(s, part[1]) || meet(s, part[2]); }
  bool meets(const CacheSpans& c) const { return c.meets(part[0]) || c.meets(part[1]) || c.meets(part[2]); }
};

int check_cache(const sdpa_cache_t* c, CacheView* v, CacheSpans* pool) {
  if (c == nullptr) return SDPA_ERR_INVALID_ARG;
  if (c->dtype < SDPA_CACHE_F32 || c->dtype > SDPA_CACHE_INT8) return SDPA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->Hkv < 1) return SDPA_ERR_INVALID_ARG;
  if (!(c->d == 16 || c->d == 64 || c->d == 128)) return SDPA_ERR_UNSUPPORTED;
  if (c->k == nullptr || c->v == nullptr) return SDPA_ERR_INVALID_ARG;
  if (!stride_ok(c->k_strides) || !stride_ok(c->v_strides)) return SDPA_ERR_INVALID_ARG;
  if (is_codes(c->dtype)) {
    if (c->k_scale == nullptr || c->v_scale == nullptr) return SDPA_ERR_INVALID_ARG;
    if (!stride_ok(c->k_scale_strides) || !stride_ok(c->v_scale_strides)) return SDPA_ERR_INVALID_ARG;
    if (!aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4)) return SDPA_ERR_MISALIGNED;
  }
  const size_t esz = cache_esz(c->dtype);
  if (!aligned_to(c->k, esz) || !aligned_to(c->v, esz)) return SDPA_ERR_MISALIGNED;
  *pool = spans_of(*c);
  if (!pool->fits()) return SDPA_ERR_INVALID_ARG;
  memset(v, 0, sizeof(*v));
  v->k = c->k; v->v = c->v;
  v->kp = c->k_strides.b; v->kh = c->k_strides.h; v->kt = c->k_strides.t;
  v->vp = c->v_strides.b; v->vh = c->v_strides.h; v->vt = c->v_strides.t;
  if (is_codes(c->dtype)) {
    v->ks = c->k_scale; v->vs = c->v_scale;
    v->ksp = c->k_scale_strides.b; v->ksh = c->k_scale_strides.h; v->kst = c->k_scale_strides.t;
    v->vsp = c->v_scale_strides.b; v->vsh = c->v_scale_strides.h; v->vst = c->v_scale_strides.t;
  }
  v->dtype = c->dtype; v->num_pages = c->num_pages; v->page_size = c->page_size; v->Hkv = c->Hkv; v->d = c->d;
  v->fd_page = make_fastdiv((uint32_t)c->page_size);
  return SDPA_OK;
}

int check_batch(const sdpa_batch_t* s, const CacheView& c, bool rows, BatchView* v, BatchSpans* read) {
  if (s == nullptr) return SDPA_ERR_INVALID_ARG;
  if (s->B < 0 || s->max_pages < 0 || s->table_stride < s->max_pages) return SDPA_ERR_INVALID_ARG;
  if ((long long)s->max_pages * c.page_size > kMaxTokens) return SDPA_ERR_UNSUPPORTED;
  if (s->B > 0 && s->kv_lens == nullptr) return SDPA_ERR_INVALID_ARG;
  if (s->B > 0 && s->max_pages > 0 && s->page_table == nullptr) return SDPA_ERR_INVALID_ARG;
  if (!aligned_to(s->page_table, 4) || !aligned_to(s->kv_lens, 4) || !aligned_to(s->cu_q, 4)) return SDPA_ERR_MISALIGNED;
  *read = {{span_of(s->max_pages > 0 ? s->page_table : nullptr, (__int128)(s->B - 1) * s->table_stride + s->max_pages, 4),
            span_of(s->kv_lens, s->B, 4), span_of(rows ? s->cu_q : nullptr, s->B + 1LL, 4)}};
  if (!read->fits()) return SDPA_ERR_INVALID_ARG;
  memset(v, 0, sizeof(*v));
  v->table = s->page_table; v->table_stride = s->table_stride; v->max_pages = s->max_pages;
  v->kv_lens = s->kv_lens; v->B = s->B;
  if (rows) {
    if (s->total_q < 0 || s->max_q < 0) return SDPA_ERR_INVALID_ARG;
    if (s->total_q > kMaxTokens) return SDPA_ERR_UNSUPPORTED;
    if (s->cu_q == nullptr && s->total_q != s->B) return SDPA_ERR_INVALID_ARG;
    if (s->B == 0 && s->total_q > 0) return SDPA_ERR_INVALID_ARG;
    v->cu_q = s->cu_q; v->total_q = s->total_q;
    v->max_q = s->cu_q == nullptr ? 1 : s->max_q < s->total_q ? s->max_q : s->total_q;
  }
  return SDPA_OK;
}

int build_paged(const void* q, const sdpa_rows_t* qs, const sdpa_cache_t* cache, const sdpa_batch_t* batch, void* out,
                const sdpa_rows_t* os, sdpa_dtype_t dtype, int Hq, float scale, int window, float softcap,
                const float* slopes, float* lse, PagedParams* p) {
  memset(p, 0, sizeof(*p));
  if (dtype != SDPA_F32 && dtype != SDPA_BF16) return SDPA_ERR_INVALID_ARG;
  CacheSpans pool;
  BatchSpans read;
  int rc = check_cache(cache, &p->c, &pool);
  if (rc == SDPA_OK) rc = check_batch(batch, p->c, true, &p->s, &read);
  if (rc != SDPA_OK) return rc;
  if (Hq < 1 || Hq % p->c.Hkv != 0) return SDPA_ERR_INVALID_ARG;
  if (Hq > 65535) return SDPA_ERR_UNSUPPORTED;
  if (!is_codes(p->c.dtype) && (p->c.dtype == SDPA_CACHE_F32) != (dtype == SDPA_F32)) return SDPA_ERR_UNSUPPORTED;
  if (!isfinite(scale) || !isfinite(softcap) || softcap < 0.f || window < 0) return SDPA_ERR_INVALID_ARG;
  const int d = p->c.d;
  const sdpa_rows_t dense = {(int64_t)Hq * d, d};
  const sdpa_rows_t a = qs ? *qs : dense, o = os ? *os : dense;
  if (!stride_ok(a) || !stride_ok(o)) return SDPA_ERR_INVALID_ARG;
  p->q = q; p->out = out; p->lse = lse; p->slopes = slopes;
  p->qt = a.t; p->qh = a.h; p->ot = o.t; p->oh = o.h;
  p->Hq = Hq; p->group = Hq / p->c.Hkv;
  p->scale = scale;
  // 1 / c stays finite, so that a score of 0 stays 0; below this a capped score is as good as 0 anyway
  p->softcap = softcap > 0.f ? fmaxf(softcap, 1e-37f) : 0.f;
  // a window that no sequence of the table can leave is none
  p->window = window >= (long long)p->s.max_pages * p->c.page_size ? 0 : window;
  const int T = p->s.total_q;
  if (T == 0) return SDPA_OK;
  if (q == nullptr || out == nullptr) return SDPA_ERR_INVALID_ARG;
  const size_t esz = dtype == SDPA_F32 ? 4 : 2;
  if (!aligned_to(q, esz) || !aligned_to(out, esz) || !aligned_to(lse, 4) || !aligned_to(slopes, 4))
    return SDPA_ERR_MISALIGNED;
  const Span sq = span_of(q, last2(a, T, Hq, d), esz), so = span_of(out, last2(o, T, Hq, d), esz);
  const Span sl = span_of(lse, (long long)T * Hq, 4);
  const Span ss = span_of(slopes, Hq, 4);
  if (!sq.fits() || !so.fits() || !sl.fits() || meet(so, sl)) return SDPA_ERR_INVALID_ARG;
  for (const Span& s : {so, sl})
    if (meet(s, sq) || meet(s, ss) || pool.meets(s) || read.meets(s)) return SDPA_ERR_INVALID_ARG;
  return SDPA_OK;
}

// Which kernels a call takes.  A sequence's rows per kv head decide: the
// decode kernel has those of up to kDecodeRows, the tensor-core kernel (the
// exact kernel where a layout keeps that one out) the others.  The host only
// knows the bound max_q, so a batch that may hold both kinds launches both
// kernels, and each leaves out the other's sequences; a single sequence that
// may be long goes to the tensor-core kernel whatever it turns out to be.
struct Plan {
  int status;
  bool decode, tc, exact;
  int limit;  // rows up to which sequences are the decode kernel's, for the others
  size_t decode_ws, tc_ws;
  int64_t ws_bytes;
};

Plan make_plan(const PagedParams& p, sdpa_dtype_t dtype, int path) {
  Plan r;
  memset(&r, 0, sizeof(r));
  const int dec = paged_decode_check(p, dtype), tc = paged_tc_check(p, dtype);
  const bool all_few = (long long)p.s.max_q * p.group <= kDecodeRows;
  switch (path) {
    case SDPA_PAGED_EXACT: r.exact = true; break;
    case SDPA_PAGED_DECODE:
      r.status = dec != SDPA_OK ? dec : all_few ? SDPA_OK : SDPA_ERR_UNSUPPORTED;
      r.decode = true;
      break;
    case SDPA_PAGED_TCGEN05:
      r.status = tc;
      r.tc = true;
      break;
    default:
      r.decode = dec == SDPA_OK && (all_few || p.s.B > 1 || tc != SDPA_OK);
      if (!(r.decode && all_few)) (tc == SDPA_OK ? r.tc : r.exact) = true;
  }
  if (r.status != SDPA_OK) return r;
  r.limit = r.decode ? kDecodeRows : 0;
  if (r.decode) r.decode_ws = (paged_decode_workspace(p) + 255) / 256 * 256;
  if (r.tc) r.tc_ws = paged_tc_workspace(p, r.limit);
  r.ws_bytes = (int64_t)(r.decode_ws + r.tc_ws);
  return r;
}

}  // namespace
}  // namespace sdpa

using namespace sdpa;

extern "C" int sdpa_cache_write(const sdpa_cache_t* cache, const sdpa_batch_t* batch, const void* k,
                                const sdpa_rows_t* k_strides, const void* v, const sdpa_rows_t* v_strides,
                                sdpa_dtype_t dtype, cudaStream_t stream) {
  CacheView c;
  BatchView s;
  if (dtype != SDPA_F32 && dtype != SDPA_BF16) return SDPA_ERR_INVALID_ARG;
  CacheSpans pool;
  BatchSpans read;
  int rc = check_cache(cache, &c, &pool);
  if (rc == SDPA_OK) rc = check_batch(batch, c, true, &s, &read);
  if (rc != SDPA_OK) return rc;
  if (!is_codes(c.dtype) && (c.dtype == SDPA_CACHE_F32) != (dtype == SDPA_F32)) return SDPA_ERR_UNSUPPORTED;
  const sdpa_rows_t dense = {(int64_t)c.Hkv * c.d, c.d};
  const sdpa_rows_t ks = k_strides ? *k_strides : dense, vs = v_strides ? *v_strides : dense;
  if (!stride_ok(ks) || !stride_ok(vs)) return SDPA_ERR_INVALID_ARG;
  if (s.total_q == 0) return SDPA_OK;
  if ((long long)s.total_q * 2 * c.Hkv > 0x7fffffffLL) return SDPA_ERR_UNSUPPORTED;
  if (k == nullptr || v == nullptr) return SDPA_ERR_INVALID_ARG;
  const size_t esz = dtype == SDPA_F32 ? 4 : 2;
  if (!aligned_to(k, esz) || !aligned_to(v, esz)) return SDPA_ERR_MISALIGNED;
  const Span sk = span_of(k, last2(ks, s.total_q, c.Hkv, c.d), esz), sv = span_of(v, last2(vs, s.total_q, c.Hkv, c.d), esz);
  if (!sk.fits() || !sv.fits() || pool.meets(sk) || pool.meets(sv) || read.meets(pool)) return SDPA_ERR_INVALID_ARG;
  int* err = error_word();
  if (err == nullptr) return SDPA_ERR_CUDA;
  return launch_cache_write(c, s, k, ks.t, ks.h, v, vs.t, vs.h, dtype, err, stream) == cudaSuccess ? SDPA_OK
                                                                                                  : SDPA_ERR_CUDA;
}

extern "C" int sdpa_cache_read(const sdpa_cache_t* cache, const sdpa_batch_t* batch, void* k_out,
                               const sdpa_strides_t* k_strides, void* v_out, const sdpa_strides_t* v_strides,
                               sdpa_dtype_t dtype, int T, cudaStream_t stream) {
  CacheView c;
  BatchView s;
  if (dtype != SDPA_F32 && dtype != SDPA_BF16) return SDPA_ERR_INVALID_ARG;
  if (T < 0) return SDPA_ERR_INVALID_ARG;
  CacheSpans pool;
  BatchSpans read;
  int rc = check_cache(cache, &c, &pool);
  if (rc == SDPA_OK) rc = check_batch(batch, c, false, &s, &read);
  if (rc != SDPA_OK) return rc;
  if (T > kMaxTokens) return SDPA_ERR_UNSUPPORTED;
  if (!is_codes(c.dtype) && (c.dtype == SDPA_CACHE_F32) != (dtype == SDPA_F32)) return SDPA_ERR_UNSUPPORTED;
  const sdpa_strides_t dense = {(int64_t)c.Hkv * T * c.d, (int64_t)T * c.d, c.d};
  const sdpa_strides_t ks = k_strides ? *k_strides : dense, vs = v_strides ? *v_strides : dense;
  if (s.B == 0 || T == 0) return SDPA_OK;
  if (!stride_ok(ks) || !stride_ok(vs)) return SDPA_ERR_INVALID_ARG;
  if ((long long)s.B * 2 * c.Hkv * ((T + 31) / 32) > 0x7fffffffLL) return SDPA_ERR_UNSUPPORTED;
  if (k_out == nullptr || v_out == nullptr) return SDPA_ERR_INVALID_ARG;
  const size_t esz = dtype == SDPA_F32 ? 4 : 2;
  if (!aligned_to(k_out, esz) || !aligned_to(v_out, esz)) return SDPA_ERR_MISALIGNED;
  const Span ok = span_of(k_out, last3(ks, s.B, c.Hkv, T, c.d), esz), ov = span_of(v_out, last3(vs, s.B, c.Hkv, T, c.d), esz);
  if (!ok.fits() || !ov.fits()) return SDPA_ERR_INVALID_ARG;
  for (const Span& s : {ok, ov})
    if (pool.meets(s) || read.meets(s)) return SDPA_ERR_INVALID_ARG;
  // the outputs may interleave, as views of one tensor; rows that begin less than a row apart are not two
  if (std::max(ok.lo, ov.lo) - std::min(ok.lo, ov.lo) < c.d * esz) return SDPA_ERR_INVALID_ARG;
  int* err = error_word();
  if (err == nullptr) return SDPA_ERR_CUDA;
  return launch_cache_read(c, s, k_out, ks, v_out, vs, dtype, T, err, stream) == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

extern "C" int sdpa_fwd_paged(const void* q, const sdpa_rows_t* q_strides, const sdpa_cache_t* cache,
                          const sdpa_batch_t* batch, void* out, const sdpa_rows_t* out_strides, sdpa_dtype_t dtype,
                          int Hq, float scale, int window, float softcap, const float* slopes, float* lse, int path,
                          void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  if (path < SDPA_PAGED_AUTO || path > SDPA_PAGED_TCGEN05) return SDPA_ERR_INVALID_ARG;
  PagedParams p;
  const int rc = build_paged(q, q_strides, cache, batch, out, out_strides, dtype, Hq, scale, window, softcap, slopes, lse, &p);
  if (rc != SDPA_OK) return rc;
  if (p.s.total_q == 0) return SDPA_OK;
  const Plan plan = make_plan(p, dtype, path);
  if (plan.status != SDPA_OK) return plan.status;
  if (plan.ws_bytes > 0) {
    if (workspace == nullptr || workspace_bytes < plan.ws_bytes) return SDPA_ERR_CAPACITY;
    if (!aligned_to(workspace, 16)) return SDPA_ERR_MISALIGNED;
  }
  p.err = error_word();
  if (p.err == nullptr) return SDPA_ERR_CUDA;
  if (plan.decode && launch_paged_decode(p, workspace, stream) != cudaSuccess) return SDPA_ERR_CUDA;
  if (plan.tc && launch_paged_tc(p, plan.limit, static_cast<char*>(workspace) + plan.decode_ws, stream) != cudaSuccess)
    return SDPA_ERR_CUDA;
  if (plan.exact) {
    p.skip_rows = plan.limit;
    if (launch_paged_exact(p, dtype, stream) != cudaSuccess) return SDPA_ERR_CUDA;
  }
  return SDPA_OK;
}

extern "C" int64_t sdpa_fwd_paged_workspace(const sdpa_cache_t* cache, const sdpa_batch_t* batch, const void* q,
                                            const sdpa_rows_t* q_strides, const void* out,
                                            const sdpa_rows_t* out_strides, sdpa_dtype_t dtype, int Hq, int window,
                                            int path) {
  if (path < SDPA_PAGED_AUTO || path > SDPA_PAGED_TCGEN05) return SDPA_ERR_INVALID_ARG;
  PagedParams p;
  const int rc = build_paged(q, q_strides, cache, batch, const_cast<void*>(out), out_strides, dtype, Hq, 1.f, window, 0.f,
                             nullptr, nullptr, &p);
  if (rc != SDPA_OK) return rc;
  if (p.s.total_q == 0) return 0;
  const Plan plan = make_plan(p, dtype, path);
  return plan.status != SDPA_OK ? plan.status : plan.ws_bytes;
}
