// Writing new keys and values into a paged cache, and reading sequences back.
//
// An 8-bit cache holds one f32 scale per (token, head) row of d elements:
//   s = max(fl(amax / Q), 2^-30),  Q = 448 (e4m3) or 127 (int8)
//   code = round_to_type(fl(x / s)), ties to even, saturated;  value = code * s
// with fl the rounding to fp32 (IEEE division), so the codes are the same
// wherever they are computed.  amax skips NaN elements; those become the NaN
// code (e4m3) or 0 (int8).  The floor keeps every scale and its reciprocal a
// normal number and bounds how far apart two scales of ordinary rows can be.
//
// Both are HBM-bound: each element is read once and written once.  A row is
// held by a group of neighbouring lanes, 16 bytes of the wider side each, so
// its amax is a few shuffles and nothing is staged; a warp keeps several rows
// in flight to cover the latency of their loads.
#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "pdl_launch.cuh"

namespace sdpa {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsAhead = 4;  // rows a lane group has in flight

// Sequence of packed row t: the last b with cu[b] <= t (0 if there is none),
// searched by the whole warp, 32 boundaries at a time.
__device__ __forceinline__ int find_seq(const int* cu, int B, int t, int lane) {
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, i < n && ld_prior(cu + lo + i) <= t);
    const int k = max(0, __popc(le) - 1);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// fl(x / s) for the many x of a row, from r = fl(1 / s): q = fl(x r) is within
// an ulp, and q + fl(x - q s) r, both fused, is the correctly rounded quotient
// unless s's significand is all ones (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  Three operations
// an element where a division is tens (8190 tokens of 12 heads to int8: 20 us
// for the launch, 33 with divisions and an index computation per piece).
// r = 0 asks for the division: all-ones significands, and scales so large that
// r or the remainder could leave the normal range.  (Small x can make the
// remainder inexact only where the code is 0 either way: s >= 2^-30.)
__device__ __forceinline__ float row_reciprocal(float s) {
  const bool plain = s < 1e30f && (__float_as_uint(s) & 0x7fffffu) != 0x7fffffu;
  return plain ? __frcp_rn(s) : 0.f;
}
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}
// y = fl(x / s) to the code.  |y| <= Q by the choice of s, so nothing saturates;
// adding 1.5 2^23 leaves the integer nearest to y, ties to even, in the low bits.
template <typename C>
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d) {
  if constexpr (std::is_same<C, int8_t>::value) {
    auto low = [](float y) { return y == y ? __float_as_uint(y + 12582912.f) : 0u; };
    return __byte_perm(__byte_perm(low(a), low(b), 0x0040), __byte_perm(low(c), low(d), 0x0040), 0x5410);
  } else {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
}
// The E elements of a 16-byte piece as fp32.
__device__ __forceinline__ float piece_elem(const uint32_t (&w)[4], int n, float) { return __uint_as_float(w[n]); }
__device__ __forceinline__ float piece_elem(const uint32_t (&w)[4], int n, __nv_bfloat16) {
  return __uint_as_float(n & 1 ? w[n >> 1] & 0xffff0000u : w[n >> 1] << 16);
}
// Their largest magnitude; NaN elements are passed over.
__device__ __forceinline__ float piece_amax(const uint32_t (&w)[4], float) {
  float m = 0.f;
#pragma unroll
  for (int n = 0; n < 4; ++n) m = fmaxf(m, fabsf(__uint_as_float(w[n])));
  return m;
}
__device__ __forceinline__ float piece_amax(const uint32_t (&w)[4], __nv_bfloat16) {
  __nv_bfloat162 m = __float2bfloat162_rn(0.f), x;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    memcpy(&x, &w[n], 4);
    m = __hmax2(m, __habs2(x));
  }
  return fmaxf(__low2float(m), __high2float(m));
}
template <typename T, typename C, int E>
__device__ __forceinline__ void encode_piece(const uint32_t (&w)[4], float s, uint32_t (&out)[E * sizeof(C) / 4]) {
  if constexpr (is_code<C>::value) {
    const float r = row_reciprocal(s);
    float q[E];
#pragma unroll
    for (int n = 0; n < E; ++n) q[n] = quotient(piece_elem(w, n, T()), s, r);
    if (r == 0.f) {
#pragma unroll
      for (int n = 0; n < E; ++n) q[n] = __fdiv_rn(piece_elem(w, n, T()), s);
    }
#pragma unroll
    for (int n = 0; n < E; n += 4) out[n / 4] = codes_of<C>(q[n], q[n + 1], q[n + 2], q[n + 3]);
  } else {
    static_assert(std::is_same<T, C>::value, "copied as it is");
#pragma unroll
    for (int n = 0; n < 4; ++n) out[n] = w[n];
  }
}
template <typename C> constexpr float code_max() { return std::is_same<C, int8_t>::value ? 127.f : 448.f; }

struct WriteArgs {
  CacheView c;
  BatchView s;
  const void* k;
  const void* v;
  long long kt, kh, vt, vh;
  int vec;   // sources and cache rows allow whole-piece accesses
  int tb;    // tokens of a block
  int ppt;   // 16-byte pieces of a token: 2 Hkv D / E
  int per;   // pieces of a token a block's threads have at once, a multiple of a row's
  int side;  // tokens side by side
  FastDiv fd_per;
  int* err;
};

constexpr int kMaxTok = 32;  // tokens of a block at most
constexpr int kAhead = 4;    // pieces a thread has in flight

// T: elements given, C: elements kept.  A block takes tb tokens, all heads of k
// and v.  A thread keeps its place in a token (16 bytes of one row) and walks
// the tokens, so rows and heads are divided once.  While its first pieces are on
// their way one warp looks up where the tokens go.
template <typename T, typename C, int D>
__global__ void __launch_bounds__(kThreads, 5) cache_write_kernel(const __grid_constant__ WriteArgs a) {
  constexpr int E = 16 / sizeof(T);  // elements of a piece
  constexpr int G = D / E;           // pieces (neighbouring lanes) of a row
  __shared__ int s_page[kMaxTok], s_off[kMaxTok];
  sm100::grid_dep_launch();
  sm100::grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int t0 = blockIdx.x * a.tb;
  const int ntok = min(a.tb, a.s.total_q - t0);
  const int tl = (int)fdiv((uint32_t)tid, a.fd_per), pc = tid - tl * a.per;
  bool looked_up = false;
  for (int c = 0; c < a.ppt; c += a.per) {
    const int row = (c + pc) / G;  // k heads, then v heads
    const bool mine = tl < a.side && c + pc < a.ppt;
    const bool is_v = row >= a.c.Hkv;
    const int h = is_v ? row - a.c.Hkv : row;
    const long long st = is_v ? a.vt : a.kt, dp = is_v ? a.c.vp : a.c.kp, dt = is_v ? a.c.vt : a.c.kt;
    const T* src = static_cast<const T*>(is_v ? a.v : a.k) + h * (is_v ? a.vh : a.kh) + t0 * st + (tid % G) * E;
    C* dst = static_cast<C*>(is_v ? a.c.v : a.c.k) + h * (is_v ? a.c.vh : a.c.kh) + (tid % G) * E;
    for (int base = 0; base < ntok; base += a.side * kAhead) {
      uint32_t x[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int t = base + u * a.side + tl;
        if (mine && t < ntok) {
          const T* at = src + t * st;
          if (a.vec) {
            const uint4 raw = ld_prior(reinterpret_cast<const uint4*>(at));
            x[u][0] = raw.x; x[u][1] = raw.y; x[u][2] = raw.z; x[u][3] = raw.w;
          } else {
            alignas(16) T e[E];
#pragma unroll
            for (int n = 0; n < E; ++n) e[n] = at[n];
            memcpy(x[u], e, 16);
          }
        } else {
          x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0;
        }
      }
      if (!looked_up) {
        looked_up = true;
        if (tid < 32) {
          const int first = a.s.cu_q ? find_seq(a.s.cu_q, a.s.B, t0, lane) : 0;
          if (lane < ntok) {
            const int t = t0 + lane;
            int b = t, page = -1, off = 0;
            if (a.s.cu_q)
              for (b = first; b + 1 < a.s.B && ld_prior(a.s.cu_q + b + 1) <= t;) ++b;
            const Seq q = seq_of(a.s, a.c, b, a.err);
            // rows behind the last sequence and rows without a place are left out
            if (t >= q.q0 && t < q.q0 + q.n) {
              const int pos = q.L - q.n + (t - q.q0);
              if (pos < 0) {
                index_error(a.err);
              } else {
                page = page_or_bad(a.s, a.c, b, pos, a.err);
                off = pos - (int)fdiv((uint32_t)pos, a.c.fd_page) * a.c.page_size;
              }
            }
            s_page[lane] = page;
            s_off[lane] = off;
          }
        }
        __syncthreads();
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        float s = 1.f;
        if (is_code<C>::value) {
          float m = piece_amax(x[u], T());
#pragma unroll
          for (int o = 1; o < G; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          // fl(m / Q) the same way: neither Q's significand is all ones
          constexpr float Q = code_max<C>();
          s = m < 1e30f && m > 1e-20f ? quotient(m, Q, 1.f / Q) : __fdiv_rn(m, Q);
          s = fmaxf(s, kScaleFloor);
        }
        const int t = base + u * a.side + tl;
        if (!mine || t >= ntok) continue;
        const long long page = s_page[t];
        if (page < 0) continue;
        const int off = s_off[t];
        C* out = dst + page * dp + off * dt;
        constexpr int W = E * sizeof(C) / 4;
        uint32_t y[W];
        encode_piece<T, C, E>(x[u], s, y);
        if (a.vec) {
          if constexpr (W == 4) *reinterpret_cast<uint4*>(out) = make_uint4(y[0], y[1], y[2], y[3]);
          else if constexpr (W == 2) *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[1]);
          else *reinterpret_cast<uint32_t*>(out) = y[0];
        } else {
          alignas(16) C e[E];
          memcpy(e, y, sizeof(e));
#pragma unroll
          for (int n = 0; n < E; ++n) out[n] = e[n];
        }
        if (is_code<C>::value && tid % G == 0) {
          if (is_v) a.c.vs[page * a.c.vsp + h * a.c.vsh + off * a.c.vst] = s;
          else a.c.ks[page * a.c.ksp + h * a.c.ksh + off * a.c.kst] = s;
        }
      }
    }
  }
}

struct ReadArgs {
  CacheView c;
  BatchView s;
  void* k;
  void* v;
  sdpa_strides_t ks, vs;
  int T, chunks;  // chunks: blocks along the tokens of one (sequence, k or v, head)
  int vec;
  FastDiv fd_chunks, fd_h;
  int* err;
};

template <int N>
struct alignas(N) Bytes {
  uint8_t b[N];
};
// 32 bytes at once: one store per lane where the row's codes were one load
__device__ __forceinline__ void store32(void* p, const void* src) {
  const uint32_t* s = static_cast<const uint32_t*>(src);
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(s[0]), "r"(s[1]), "r"(s[2]),
               "r"(s[3]), "r"(s[4]), "r"(s[5]), "r"(s[6]), "r"(s[7])
               : "memory");
}

// C: elements kept, T: elements given out.  A block takes a run of tokens of
// one (sequence, k or v, head): rows that follow each other in a page and in
// the output.  A lane has 16 bytes of T of a row, 32 from 8-bit codes to bf16.
template <typename C, typename T>
constexpr int read_elems() {
  return sizeof(C) == 1 && sizeof(T) == 2 ? 16 : 16 / sizeof(T);
}
template <typename C, typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int E = read_elems<C, T>();
  constexpr int G = D / E;
  constexpr int RB = kThreads / G;  // rows of a block side by side
  sm100::grid_dep_launch();
  sm100::grid_dep_wait();
  const uint32_t z = fdiv(blockIdx.x, a.fd_chunks);
  const int chunk = (int)(blockIdx.x - z * a.chunks);
  const uint32_t z2 = fdiv(z, a.fd_h);
  const int h = (int)(z - z2 * a.c.Hkv);
  const bool is_v = z2 & 1;
  const int b = (int)(z2 >> 1);
  const int L = min(seq_len(a.s, a.c, b, a.err), a.T);
  const int t0 = chunk * (RB * kRowsAhead);
  if (t0 >= L) return;
  const int e0 = (threadIdx.x % G) * E;
  const C* src = static_cast<const C*>(is_v ? a.c.v : a.c.k) + h * (is_v ? a.c.vh : a.c.kh) + e0;
  const float* sc = is_v ? a.c.vs : a.c.ks;
  if (is_code<C>::value) sc += h * (is_v ? a.c.vsh : a.c.ksh);
  const long long sp = is_v ? a.c.vp : a.c.kp, stk = is_v ? a.c.vt : a.c.kt;
  const long long ssp = is_v ? a.c.vsp : a.c.ksp, sst = is_v ? a.c.vst : a.c.kst;
  const sdpa_strides_t os = is_v ? a.vs : a.ks;
  T* dst = static_cast<T*>(is_v ? a.v : a.k) + (long long)b * os.b + (long long)h * os.h + e0;
  int page[kRowsAhead];
#pragma unroll
  for (int u = 0; u < kRowsAhead; ++u) {
    const int t = t0 + u * RB + threadIdx.x / G;
    page[u] = t < L ? page_of(a.s, a.c, b, t, a.err) : 0;
  }
  alignas(16) C raw[kRowsAhead][E];
  float s[kRowsAhead];
#pragma unroll
  for (int u = 0; u < kRowsAhead; ++u) {
    const int t = t0 + u * RB + threadIdx.x / G;
    if (t < L) {
      const int off = t - (int)fdiv((uint32_t)t, a.c.fd_page) * a.c.page_size;
      const C* row = src + page[u] * sp + off * stk;
      if (a.vec) {
        using V = Bytes<E * sizeof(C)>;
        if constexpr (E * sizeof(C) == 16) *reinterpret_cast<uint4*>(raw[u]) = ld_prior(reinterpret_cast<const uint4*>(row));
        else *reinterpret_cast<V*>(raw[u]) = *reinterpret_cast<const V*>(row);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) raw[u][i] = row[i];
      }
      s[u] = is_code<C>::value ? sc[page[u] * ssp + off * sst] : 1.f;
    }
  }
#pragma unroll
  for (int u = 0; u < kRowsAhead; ++u) {
    const int t = t0 + u * RB + threadIdx.x / G;
    if (t < L) {
      alignas(32) T y[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float f = cache_elem(raw[u][i]);
        y[i] = from_f32<T>(is_code<C>::value ? f * s[u] : f);
      }
      T* o = dst + (long long)t * os.t;
      if (a.vec) {
        if constexpr (E * sizeof(T) == 32) store32(o, y);
        else *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(y);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = y[i];
      }
    }
  }
}

// base and strides (in elements of esz bytes) all multiples of n bytes
bool mult(const void* p, long long a, long long b, long long c, int esz, int n) {
  return reinterpret_cast<uintptr_t>(p) % n == 0 && (a * esz) % n == 0 && (b * esz) % n == 0 && (c * esz) % n == 0;
}

template <typename T, typename C, int D>
cudaError_t write_one(WriteArgs& a, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  const int nb = E * sizeof(C);
  a.vec = mult(a.k, a.kt, a.kh, 0, sizeof(T), 16) && mult(a.v, a.vt, a.vh, 0, sizeof(T), 16) &&
          mult(a.c.k, a.c.kp, a.c.kh, a.c.kt, sizeof(C), nb) && mult(a.c.v, a.c.vp, a.c.vh, a.c.vt, sizeof(C), nb);
  a.ppt = 2 * a.c.Hkv * (D / E);
  const int rounds = (a.ppt + kThreads - 1) / kThreads;
  a.per = rounds == 1 ? a.ppt : ((a.ppt + rounds - 1) / rounds + 31) / 32 * 32;
  a.side = std::max(1, std::min(kMaxTok / kAhead, kThreads / a.per));
  a.fd_per = make_fastdiv((uint32_t)a.per);
  // a token per block while that does not fill the SMs, beyond that up to as
  // many as the block's threads have pieces in flight for
  a.tb = std::max(1, std::min(a.side * kAhead, a.s.total_q / (4 * num_sms())));
  const int threads = (a.side * a.per + 31) / 32 * 32;
  return launch_serialized(cache_write_kernel<T, C, D>, dim3((unsigned)((a.s.total_q + a.tb - 1) / a.tb)),
                           dim3((unsigned)threads), 0, stream, a);
}
template <typename T, typename C>
cudaError_t write_d(WriteArgs& a, cudaStream_t stream) {
  switch (a.c.d) {
    case 16: return write_one<T, C, 16>(a, stream);
    case 64: return write_one<T, C, 64>(a, stream);
    case 128: return write_one<T, C, 128>(a, stream);
  }
  return cudaErrorInvalidValue;
}

template <typename C, typename T, int D>
cudaError_t read_one(ReadArgs& a, cudaStream_t stream) {
  constexpr int E = read_elems<C, T>(), RB = kThreads / (D / E);
  const int nb = E * sizeof(C), no = E * sizeof(T);
  a.vec = mult(a.k, a.ks.b, a.ks.h, a.ks.t, sizeof(T), no) && mult(a.v, a.vs.b, a.vs.h, a.vs.t, sizeof(T), no) &&
          mult(a.c.k, a.c.kp, a.c.kh, a.c.kt, sizeof(C), nb) && mult(a.c.v, a.c.vp, a.c.vh, a.c.vt, sizeof(C), nb);
  a.chunks = (a.T + RB * kRowsAhead - 1) / (RB * kRowsAhead);
  a.fd_chunks = make_fastdiv((uint32_t)a.chunks);
  const long long grid = (long long)a.s.B * 2 * a.c.Hkv * a.chunks;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_serialized(cache_read_kernel<C, T, D>, dim3((unsigned)grid), dim3(kThreads), 0, stream, a);
}
template <typename C, typename T>
cudaError_t read_d(ReadArgs& a, cudaStream_t stream) {
  switch (a.c.d) {
    case 16: return read_one<C, T, 16>(a, stream);
    case 64: return read_one<C, T, 64>(a, stream);
    case 128: return read_one<C, T, 128>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_write(const CacheView& c, const BatchView& s, const void* k, long long kt, long long kh,
                               const void* v, long long vt, long long vh, sdpa_dtype_t dtype, int* err,
                               cudaStream_t stream) {
  WriteArgs a;
  a.c = c; a.s = s; a.k = k; a.v = v; a.kt = kt; a.kh = kh; a.vt = vt; a.vh = vh; a.err = err;
  const bool f = dtype == SDPA_F32;
  switch (c.dtype) {
    case SDPA_CACHE_F32: return write_d<float, float>(a, stream);
    case SDPA_CACHE_BF16: return write_d<__nv_bfloat16, __nv_bfloat16>(a, stream);
    case SDPA_CACHE_E4M3:
      return f ? write_d<float, __nv_fp8_e4m3>(a, stream) : write_d<__nv_bfloat16, __nv_fp8_e4m3>(a, stream);
    case SDPA_CACHE_INT8: return f ? write_d<float, int8_t>(a, stream) : write_d<__nv_bfloat16, int8_t>(a, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_cache_read(const CacheView& c, const BatchView& s, void* k, const sdpa_strides_t& ks, void* v,
                              const sdpa_strides_t& vs, sdpa_dtype_t dtype, int T, int* err, cudaStream_t stream) {
  ReadArgs a;
  a.c = c; a.s = s; a.k = k; a.v = v; a.ks = ks; a.vs = vs; a.T = T; a.err = err;
  a.fd_h = make_fastdiv((uint32_t)c.Hkv);
  const bool f = dtype == SDPA_F32;
  switch (c.dtype) {
    case SDPA_CACHE_F32: return read_d<float, float>(a, stream);
    case SDPA_CACHE_BF16: return read_d<__nv_bfloat16, __nv_bfloat16>(a, stream);
    case SDPA_CACHE_E4M3:
      return f ? read_d<__nv_fp8_e4m3, float>(a, stream) : read_d<__nv_fp8_e4m3, __nv_bfloat16>(a, stream);
    case SDPA_CACHE_INT8: return f ? read_d<int8_t, float>(a, stream) : read_d<int8_t, __nv_bfloat16>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
