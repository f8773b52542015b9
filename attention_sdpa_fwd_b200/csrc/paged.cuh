// Shared definitions of the paged key/value cache operators: the kernels'
// view of a cache and of a ragged batch over it, and the device-side reading
// of lengths and page numbers, checked before anything is addressed with them.
//
// A page number outside the pool, a length the table cannot hold or a query
// range outside the packed rows comes from device memory the host never sees,
// so every build checks them: the bad value sets ERR_INDEX in the error word
// and is replaced by one that stays in bounds (page 0, the nearest length).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "sm100.cuh"

namespace sdpa {

constexpr float kScaleFloor = 9.313225746154785e-10f;  // 2^-30: no row's scale is smaller

struct CacheView {
  void* k;
  void* v;
  float* ks;  // scales of 8-bit codes, else NULL
  float* vs;
  long long kp, kh, kt, vp, vh, vt;          // element strides: page, head, token
  long long ksp, ksh, kst, vsp, vsh, vst;    // of the scales
  int dtype, num_pages, page_size, Hkv, d;
  FastDiv fd_page;
};

struct BatchView {
  const int* table;
  long long table_stride;
  const int* kv_lens;
  const int* cu_q;  // NULL: one query row per sequence
  int max_pages, B, total_q, max_q;
};

struct PagedParams {
  CacheView c;
  BatchView s;
  const void* q;
  void* out;
  float* lse;           // optional [total_q, Hq]
  const float* slopes;  // optional [Hq]
  long long qt, qh, ot, oh;  // element strides: token, head
  int Hq, group;
  float scale, softcap;  // softcap 0: none
  int window;            // 0: none
  int skip_rows;         // the exact kernel leaves out sequences of 1 .. skip_rows (token, head) rows per kv head
  int* err;
};

// What the kernels know of one sequence: its packed rows [q0, q0 + n) and its
// L tokens in the cache; query row i stands at position L - n + i.
struct Seq {
  int q0, n, L;
};

__device__ __forceinline__ void index_error(int* err) {
  if (err != nullptr) atomicOr(err, ERR_INDEX);
}

__device__ __forceinline__ int seq_len(const BatchView& s, const CacheView& c, int b, int* err) {
  const int L = ld_prior(s.kv_lens + b);
  const long long cap = (long long)s.max_pages * c.page_size;
  if (L < 0 || L > cap) {
    index_error(err);
    return L < 0 ? 0 : (int)cap;
  }
  return L;
}

__device__ __forceinline__ Seq seq_of(const BatchView& s, const CacheView& c, int b, int* err) {
  Seq r;
  if (s.cu_q == nullptr) {
    r.q0 = b;
    r.n = 1;
  } else {
    const int a = ld_prior(s.cu_q + b), e = ld_prior(s.cu_q + b + 1);
    const bool ok = a >= 0 && e >= a && e <= s.total_q && e - a <= s.max_q;
    r.q0 = ok ? a : 0;
    r.n = ok ? e - a : 0;
    if (!ok) index_error(err);
  }
  r.L = seq_len(s, c, b, err);
  return r;
}

// Page of token t of sequence b as the table has it; a bad one becomes -1 in
// good_page.  (Apart, so that a load may be on its way long before its use.)
__device__ __forceinline__ int page_entry(const BatchView& s, const CacheView& c, int b, int t) {
  return ld_prior(s.table + (long long)b * s.table_stride + fdiv((uint32_t)t, c.fd_page));
}
__device__ __forceinline__ int good_page(const CacheView& c, int p, int* err) {
  if ((unsigned)p < (unsigned)c.num_pages) return p;
  index_error(err);
  return -1;
}
__device__ __forceinline__ int page_or_bad(const BatchView& s, const CacheView& c, int b, int t, int* err) {
  return good_page(c, page_entry(s, c, b, t), err);
}
__device__ __forceinline__ int page_of(const BatchView& s, const CacheView& c, int b, int t, int* err) {
  return max(0, page_or_bad(s, c, b, t, err));
}

// Keys [lo, hi) a query at position pos sees.
__device__ __forceinline__ void seen(const PagedParams& p, int pos, int& lo, int& hi) {
  hi = pos + 1;  // <= L
  lo = p.window > 0 ? max(0, hi - p.window) : 0;
}

// Code pairs to f16 pairs (exact): two e4m3 in the low 16 bits; two signed
// bytes u0, u1 as f16 1024 + (u ^ 128) minus 1152.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
// bytes at selectors 0..3 of x ^ 0x80808080 already applied by the caller
__device__ __forceinline__ uint32_t biased_bytes_to_half2(uint32_t x, uint32_t sel) {
  const uint32_t r = __byte_perm(x, 0x64646464u, sel);
  __half2 h;
  memcpy(&h, &r, 4);
  h = __hsub2(h, __half2{__half_raw{0x6480}, __half_raw{0x6480}});  // 1152
  uint32_t o;
  memcpy(&o, &h, 4);
  return o;
}

// 1 / x to within one rounding step (2^-23 relative); x = inf gives 0.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A capped score c tanh(x / c).  c - 2 c / (1 + e^(2 x / c)) may be off by c 2^-19
// (the exponential, up to eight roundings and the reciprocal, times 2 c) whatever
// x is, for the two terms cancel: 2^-12 at this cap, half of what rounding a
// weight to f16 may do, a sixteenth of it to bf16.
constexpr float kPlainCap = 128.f;
// Above it: tanh's series where |x| <= c / 3, cut off at 2^-22.7 of the score;
// beyond that c is less than 3.2 times what comes out.  In all 2^-19 of it.
// (2048 rows behind 6144, bf16: 645 us, the plain form 494.)  x is in any unit,
// c and ic = 1 / c in the same.
__device__ __forceinline__ float cap_any(float x, float c, float ic) {
  const float z = x * ic, z2 = z * z;
  const float series = fmaf(z2, fmaf(z2, fmaf(z2, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f);
  const float far = fmaf(-2.f * c, rcp_approx(1.f + sm100::ex2_approx(z * (2.f * 1.4426950408889634f))), c);
  return fabsf(z) <= 1.f / 3.f ? fmaf(x * z2, series, x) : far;  // NaN: far
}

// One element of a cache row as fp32.
__device__ __forceinline__ float cache_elem(float x) { return x; }
__device__ __forceinline__ float cache_elem(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float cache_elem(__nv_fp8_e4m3 x) { return float(x); }
__device__ __forceinline__ float cache_elem(int8_t x) { return (float)x; }
template <typename C> struct is_code { static constexpr bool value = sizeof(C) == 1; };

cudaError_t launch_cache_write(const CacheView& c, const BatchView& s, const void* k, long long kt, long long kh,
                               const void* v, long long vt, long long vh, sdpa_dtype_t dtype, int* err,
                               cudaStream_t stream);
cudaError_t launch_cache_read(const CacheView& c, const BatchView& s, void* k, const sdpa_strides_t& ks, void* v,
                              const sdpa_strides_t& vs, sdpa_dtype_t dtype, int T, int* err, cudaStream_t stream);
cudaError_t launch_paged_exact(const PagedParams& p, sdpa_dtype_t dtype, cudaStream_t stream);
// Sequences of up to this many (token, head) rows per kv head are the decode kernel's.
constexpr int kDecodeRows = 32;
int paged_decode_check(const PagedParams& p, sdpa_dtype_t dtype);  // SDPA_OK or why it cannot take the layout
size_t paged_decode_workspace(const PagedParams& p);
cudaError_t launch_paged_decode(const PagedParams& p, void* ws, cudaStream_t stream);
// The tensor-core kernel; `limit`: sequences of 1 .. limit rows are left to the decode kernel.
int paged_tc_check(const PagedParams& p, sdpa_dtype_t dtype);
size_t paged_tc_workspace(const PagedParams& p, int limit);
cudaError_t launch_paged_tc(const PagedParams& p, int limit, void* ws, cudaStream_t stream);
int* error_word();  // device error word of the current device, NULL if it cannot be had

}  // namespace sdpa
