// Attention over a paged cache for sequences with few new rows: at most 32
// (token, head) rows share a kv head (one new token, or a few drafted ones).
//
// HBM-bound: every key and value of the batch is read once, 4 d operations per
// (row, key) are far below what the bytes leave room for.  So the work is laid
// out by bytes, not by sequences:
//
//  * Work is counted in tiles, a step of KS keys for each of a CTA's warps, of
//    one (sequence, kv head), all of these units in one row; CTA c of G takes tiles [T c / G, T (c+1) / G), T from
//    a scan of the lengths at its start.  Every CTA streams the same number of
//    bytes whatever the lengths are.  A unit that ends up in several CTAs
//    leaves unnormalised parts (O, max, sum) in the workspace, at most two per
//    CTA, and paged_merge_kernel, launched behind, adds them in a fixed order: no
//    atomics, no state between calls.
//  * Each warp runs on its own: it copies KS keys and values at a time with
//    16-byte cp.async into its own ring of NST stages and never waits for
//    another warp before the end of a unit.  Keys outside the visible range are
//    filled with zeros without being read (their pages may be gone).
//  * S^T = K.Q^T and O^T += V^T.P^T are mma.sync m16n8k16 tiles of 16 keys (16
//    columns of V) by 8 rows: the few rows are the narrow side, K and V are
//    converted once whatever the number of rows, and P^T becomes the second
//    product's operand by a transpose of 8 x 8 blocks in registers.  (With the
//    rows on the 16-wide side, as it was first, a unit of 4 rows took twice the
//    products, exponentials and registers.)  At this arithmetic intensity the
//    tensor pipe is far from its limit and register fragments save the trips
//    through tensor memory.
//
// 8-bit codes go to f16 without rounding (every e4m3 and int8 value is one).
// The order of d inside S's sum and of O's columns is free, so a lane takes the
// codes of its fragments as 16-byte runs of a row: K[key][c D/4 ..] feeds all
// k-steps of lane c of a quad, V[key][n D/8 ..] rows n and n + 8 of every V^T
// tile, two keys interleaved by byte permutes.  q is scaled by a power of two per row
// that puts its largest element in [2^14, 2^15), so f16 keeps it to 2^-39 of
// that.  K's scale multiplies the score's column; V's goes into the exponent:
//     t_j = x_j log2e + log2 vs_j,  p_j = 2^(t_j - m),  m = max t
//     out = sum p_j code_j / sum p_j (1 / vs_j)
// p_j is kept within 2^15 (f16) by m, which may lag 2^3 behind, and offset by
// 2^12, so that a weight down to 2^-26 of the largest keeps f16's 11 bits and
// none is off by more than 2^-37 of it; the sums are fp32.  Beside bf16 values the
// weights are bf16 too (one mma takes both operands in one type, and bf16 values
// do not fit f16): 2^-8 of a weight, which takes the error of a batch's outputs
// from 1.7e-3, their own rounding, to 2.3e-3 of their size.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "paged.cuh"
#include "pdl_launch.cuh"
#include "softmax_tile.cuh"

namespace sdpa {
namespace {

using namespace sm100;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// log2 units the running max may lag behind the largest score, and the offset
// of P (f16 P: 2^(12 + 3) is below its largest number)
template <bool F16> constexpr float kLag = F16 ? 3.f : 8.f;
template <bool F16> constexpr float kOffset = F16 ? 12.f : 0.f;

// KV types
enum { KV_BF16 = 0, KV_E4M3 = 1, KV_INT8 = 2 };

struct DecodeArgs {
  PagedParams p;
  int limit;   // sequences of up to this many rows are this kernel's
  int whole;   // one CTA per unit, nothing split
  // strides of a page (bytes; of the scales elements) and of a token, 32 bits each
  uint32_t kp, vp, kt, vt, ksp, vsp, kst, vst;
  int dense;   // a page's rows of a head follow each other
  float* ws_o;      // [2 * CTAs][rows][D]
  float2* ws_ml;    // [2 * CTAs][rows]
  int4* ws_unit;    // [units] CTAs that share a unit: first, last, slot of the first (0 or 1)
};

// NT: 8-row tiles of a unit.
template <int KV, int D, int NT>
struct Cfg {
  static constexpr bool kCodes = KV != KV_BF16;
  static constexpr int kElem = kCodes ? 1 : 2;
  static constexpr int KS = !kCodes && D == 128 ? 16 : 32;       // keys of a warp's step
  static constexpr int kRow = D * kElem;
  static constexpr int kTile = KS * kRow;                        // K (or V) of a step
  static constexpr int kScales = kCodes ? 2 * KS * 4 : 0;        // ks, vs
  static constexpr int kStage = 2 * kTile + kScales;
  static constexpr bool kQSmem = NT > 1;                         // Q fragments in shared memory
  static constexpr int kCtas = kCodes && NT < 3 ? 3 : 2;         // of an SM
  static constexpr int NST = kCodes ? (D == 128 ? (kCtas == 3 ? 2 : 3) : 3) : 3;
  static constexpr int kRows = 8 * NT;
  static constexpr int kPitch = D + 4;
  static constexpr int kRing = kWarps * NST * kStage;
  static constexpr int kMergeBytes = kWarps * kRows * kPitch * 4;
  static constexpr int kQ = kQSmem ? NT * (D / 16) * 32 * 8 : 0;
  static constexpr int kBig = kRing > kMergeBytes ? kRing : kMergeBytes;
  static constexpr int oQ = kBig;
  static constexpr int oSk = oQ + kQ;                            // [kWarps][KS] float4: ks, log2 vs, 1 / vs of a step
  static constexpr int oML = oSk + (kCodes ? kWarps * KS * 16 : 0);  // [kWarps][kRows] float2
  static constexpr int kTotal = oML + kWarps * kRows * 8;
  static constexpr int kKeys = kWarps * KS;                      // keys of a tile
  static_assert(kCtas * (kTotal + 1024) <= 233472, "shared memory of an SM");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_if(uint32_t dst, const void* src, bool live) {  // zeros where not live, nothing read
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool live) {
  const int n = live ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}

// An 8 x 8 matrix of 16-bit elements, a row's pair per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// four codes to two f16 pairs
template <int KV>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KV == KV_E4M3) {
    e4m3x4_to_half2(w, lo, hi);
  } else {
    w ^= 0x80808080u;
    lo = biased_bytes_to_half2(w, 0x4140);
    hi = biased_bytes_to_half2(w, 0x4342);
  }
}

// Where 16-byte piece i of row `key` of a step's K / V tile is kept: an XOR of
// the piece within its 128-byte line that spreads the 8 lanes of a phase of
// the fragment loads over all banks.
template <int KV, int D>
__device__ __forceinline__ uint32_t k_off(int key, int piece) {
  if (KV == KV_BF16) return key * (D * 2) + ((piece ^ (key & 7)) << 4);
  return D == 128 ? key * 128 + ((piece ^ (key & 1)) << 4) : key * 64 + (piece << 4);
}
template <int KV, int D>
__device__ __forceinline__ uint32_t v_off(int key, int piece) {
  if (KV == KV_BF16) return key * (D * 2) + ((piece ^ (key & 7)) << 4);
  const int lin = D == 128 ? piece : (key & 1) * 4 + piece;
  return (D == 128 ? key : key >> 1) * 128 + ((lin ^ (((key >> 1) & 3) << 1)) << 4);
}

struct Unit {
  Seq s;
  int rows;      // n * group, 0 if they are too many for this kernel
  int lo16, hi;  // first key (rounded down to 16) and end of what any row sees
  int lo;
  int nt;        // tiles
};

template <int TK>
__device__ __forceinline__ Unit unit_of(const DecodeArgs& a, int b) {
  Unit u;
  u.s = seq_of(a.p.s, a.p.c, b, a.p.err);
  u.rows = u.s.n <= a.limit / a.p.group ? u.s.n * a.p.group : 0;  // 0: none, or not this kernel's
  u.hi = u.s.L;
  u.lo = a.p.window > 0 ? max(0, u.s.L - u.s.n + 1 - a.p.window) : 0;
  u.lo16 = u.lo & ~15;
  u.nt = u.rows > 0 && u.hi > u.lo ? (u.hi - u.lo16 + TK - 1) / TK : 0;
  return u;
}

// a / b, mostly of numbers that fit 32 bits
__device__ __forceinline__ long long div64(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// CTA that owns tile f of T split over G
__device__ __forceinline__ int owner(long long f, long long T, int G) { return (int)div64((f + 1) * G - 1, T); }

// MOD: 0 plain scores, 1 capped or with slopes, 2 the same for caps above
// kPlainCap (an instance of its own: as a branch in 1 it cost every call of that
// registers and 75.8 us against 73.8, 16 sequences of 4096, 5 drafts, slopes).
template <int KV, int D, int NT, int MOD>
__global__ void __launch_bounds__(kThreads, (Cfg<KV, D, NT>::kCtas)) paged_decode_kernel(const __grid_constant__ DecodeArgs a) {
  using C = Cfg<KV, D, NT>;
  constexpr bool F16 = KV != KV_BF16;
  constexpr int KS = C::KS, NST = C::NST;
  constexpr float kShift = kOffset<F16>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_b;
  __shared__ long long s_scan[kWarps], s_F;
  const PagedParams& p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = lane >> 2, c = lane & 3;
  grid_dep_wait();
  grid_dep_launch();  // the merge may start: it reads nothing of this call's inputs that still changes

  const int G = gridDim.x;
  int b;
  long long F, cur, end, T = 0;
  int work_ctas = G;
  if (a.whole) {
    b = blockIdx.x / p.c.Hkv;
    F = 0;
    const int nt = unit_of<C::kKeys>(a, b).nt;
    cur = (long long)(blockIdx.x - b * p.c.Hkv) * nt;
    end = cur + nt;
  } else {
    // tiles of all sequences: each thread a run of sequences, then a scan
    const int per = (p.s.B + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int i = 0; i < per; ++i) {
      const int bb = tid * per + i;
      if (bb < p.s.B) mine += unit_of<C::kKeys>(a, bb).nt;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_scan[warp] = incl;
    if (tid == 0) { s_b = p.s.B; s_F = 0; }
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += s_scan[w];
      total += s_scan[w];
    }
    T = total * p.c.Hkv;
    // at least two tiles to a CTA
    work_ctas = (int)min((long long)G, max(1LL, T / 2));
    cur = blockIdx.x < work_ctas ? div64(T * blockIdx.x, work_ctas) : T;
    end = blockIdx.x < work_ctas ? div64(T * (blockIdx.x + 1), work_ctas) : T;
    long long at = (incl - mine) * p.c.Hkv;
    if (cur < end && cur >= at && cur < at + mine * p.c.Hkv) {
      int bb = tid * per;
      for (;; ++bb) {
        const long long w = (long long)unit_of<C::kKeys>(a, bb).nt * p.c.Hkv;
        if (cur < at + w) break;
        at += w;
      }
      s_b = bb;
      s_F = at;
    }
    __syncthreads();
    b = s_b;
    F = s_F;
  }
  const long long begin = cur;

  const uint32_t ring = smem_u32(smem) + warp * (NST * C::kStage);
  float* mrg = reinterpret_cast<float*>(smem);
  float2* s_ml = reinterpret_cast<float2*>(smem + C::oML);

  while (cur < end && b < p.s.B) {
    const Unit u = unit_of<C::kKeys>(a, b);
    if (u.nt == 0) { ++b; continue; }
    const int hk = (int)div64(cur - F, u.nt);
    const int tile0 = (int)((cur - F) - (long long)hk * u.nt);
    const int ntile = (int)min((long long)(u.nt - tile0), end - cur);
    const int base = u.lo16 + tile0 * C::kKeys + warp * KS;  // this warp's first key
    const int khi = u.hi, klo = u.lo;

    // ---- the ring: one step is KS keys and values of this warp
    constexpr int kPieces = C::kRow / 16;  // of a row
    constexpr int kPass = 32 / kPieces;    // rows the warp copies at once
    constexpr int kGroups = KS / 16;       // runs of 16 tokens, each inside a page
    const int piece = lane % kPieces, r0 = lane / kPieces;
    const uint8_t* kp = static_cast<const uint8_t*>(p.c.k) + (long long)hk * p.c.kh * C::kElem + r0 * a.kt + piece * 16;
    const uint8_t* vp = static_cast<const uint8_t*>(p.c.v) + (long long)hk * p.c.vh * C::kElem + r0 * a.vt + piece * 16;
    const float* ksp = F16 ? p.c.ks + (long long)hk * p.c.ksh : nullptr;
    const float* vsp = F16 ? p.c.vs + (long long)hk * p.c.vsh : nullptr;
    // Page numbers are fetched 32 runs at a time, a lane per run, one such span
    // ahead of its use.
    constexpr int kSpan = 32 / kGroups;
    auto fetch = [&](int span) {
      const int step = span * kSpan + lane / kGroups;
      const int t = base + step * C::kKeys + 16 * (lane % kGroups);
      return step < ntile && t < khi && t + 16 > klo ? page_entry(p.s, p.c, b, t) : 0;
    };
    int pages = fetch(0), pages_next = fetch(1);
    // Q's rows are on their way before the pages are waited for: row r of the
    // unit is token r / group, head r % group
    uint32_t qw[NT][D / 8];  // of row t * 8 + quad: this lane's D / 4 elements, in pairs
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = t * 8 + quad;
      const int i = r / p.group, g = r - i * p.group;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (long long)(u.s.q0 + i) * p.qt +
                                 (long long)(hk * p.group + g) * p.qh;
      if constexpr (F16) {
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (r < u.rows) x = ld_prior(reinterpret_cast<const uint4*>(src + c * (D / 4) + k * 8));
          qw[t][4 * k] = x.x; qw[t][4 * k + 1] = x.y; qw[t][4 * k + 2] = x.z; qw[t][4 * k + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
          qw[t][k] = r < u.rows ? ld_prior(reinterpret_cast<const unsigned int*>(src + 16 * (k >> 1) + 8 * (k & 1) + 2 * c)) : 0u;
      }
    }
    pages = max(0, good_page(p.c, pages, p.err));
    // The next step: where this lane's first row of each run is, and its key's
    // scales.  Inside a page 32 bits do (the host checks that).
    const uint8_t *kq[kGroups], *vq[kGroups];
    const float *ksq, *vsq;
    auto lookup = [&](int step) {
      if (step > 0 && step % kSpan == 0) {
        pages = max(0, good_page(p.c, pages_next, p.err));
        pages_next = fetch(step / kSpan + 1);
      }
      const int t0 = base + step * C::kKeys;
      uint32_t off = t0 - fdiv((uint32_t)t0, p.c.fd_page) * p.c.page_size;
      if constexpr (F16) {
        const uint32_t pg = __shfl_sync(0xffffffffu, pages, (step % kSpan) * kGroups + lane / 16);
        uint32_t o = off + lane;
        if (o >= (uint32_t)p.c.page_size) o -= p.c.page_size;  // the second run's page (a page has 16 tokens or more)
        ksq = ksp + (uint64_t)pg * a.ksp + o * a.kst;
        vsq = vsp + (uint64_t)pg * a.vsp + o * a.vst;
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const uint32_t pg = __shfl_sync(0xffffffffu, pages, (step % kSpan) * kGroups + g);
        kq[g] = kp + (uint64_t)pg * a.kp + off * a.kt;
        vq[g] = vp + (uint64_t)pg * a.vp + off * a.vt;
        off += 16;
        if (off >= (uint32_t)p.c.page_size) off -= p.c.page_size;
      }
    };
    auto issue = [&](int step) {
      if (step < ntile) {
        const uint32_t st = ring + (step % NST) * C::kStage;
        const int t0 = base + step * C::kKeys;
        if (a.dense && t0 >= klo && t0 + KS <= khi) {
          // rows of a page that follow each other, all of them seen: constant offsets
#pragma unroll
          for (int i = 0; i < KS / kPass; ++i) {
            const int r = i * kPass, g = r / 16;
            cp16(st + k_off<KV, D>(r + r0, piece), kq[g] + (r % 16) * C::kRow);
            cp16(st + C::kTile + v_off<KV, D>(r + r0, piece), vq[g] + (r % 16) * C::kRow);
          }
          if constexpr (F16) {  // KS == 32: a lane per key
            cp4(st + 2 * C::kTile + lane * 4, ksq, true);
            cp4(st + 2 * C::kTile + (KS + lane) * 4, vsq, true);
          }
        } else {
#pragma unroll 4
          for (int i = 0; i < KS / kPass; ++i) {
            const int r = i * kPass, g = r / 16;
            const bool live = t0 + r + r0 >= klo && t0 + r + r0 < khi;
            const uint8_t *kr = g == 0 ? kq[0] : kq[kGroups - 1], *vr = g == 0 ? vq[0] : vq[kGroups - 1];
            cp16_if(st + k_off<KV, D>(r + r0, piece), kr + (r % 16) * a.kt, live);
            cp16_if(st + C::kTile + v_off<KV, D>(r + r0, piece), vr + (r % 16) * a.vt, live);
          }
          if constexpr (F16) {
            const bool live = t0 + lane >= klo && t0 + lane < khi;
            cp4(st + 2 * C::kTile + lane * 4, ksq, live);
            cp4(st + 2 * C::kTile + (KS + lane) * 4, vsq, live);
          }
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) {
      lookup(i);
      issue(i);
    }
    lookup(NST - 1);

    // ---- Q^T as B fragments
    uint32_t qf[C::kQSmem ? 1 : D / 16][2];
    uint32_t* s_q = reinterpret_cast<uint32_t*>(smem + C::oQ);
    float* s_x = reinterpret_cast<float*>(s_ml);  // a row's power of two, until the parts need the place
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t (&w)[D / 8] = qw[t];
      if constexpr (F16) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^k with top 2^k in [2^14, 2^15), k within what a float holds
        const int ex = top > 0.f && top < INFINITY ? min(126, max(-126, 141 - (int)(__float_as_uint(top) >> 23))) : 0;
        const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
        if (c == 0) s_x[warp * C::kRows + t * 8 + quad] = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const __half2 hh = __floats2half2_rn(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xffff0000u) * up);
          memcpy(&w[k], &hh, 4);
        }
      }
      // pairs 2s and 2s + 1 are b0 and b1 of k-step s
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        if constexpr (!C::kQSmem) {
          qf[s][0] = w[2 * s];
          qf[s][1] = w[2 * s + 1];
        } else if (s % kWarps == warp) {  // every warp has the same: each writes a share
          *reinterpret_cast<uint2*>(s_q + ((t * (D / 16) + s) * 32 + lane) * 2) = make_uint2(w[2 * s], w[2 * s + 1]);
        }
      }
    }
    if constexpr (C::kQSmem) __syncthreads();
    else __syncwarp();
    // this lane's columns of S^T: rows t * 8 + 2 c + e
    float xscale[NT][2];  // what turns an accumulator into its score
    float slope[MOD ? NT : 1][2];
    int pos[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = t * 8 + 2 * c + e;
        const int i = r / p.group, g = r - i * p.group;
        pos[t][e] = u.s.L - u.s.n + i;
        if constexpr (MOD) slope[t][e] = p.slopes && r < u.rows ? ld_prior(p.slopes + hk * p.group + g) : 0.f;
        xscale[t][e] = p.scale * (F16 ? s_x[warp * C::kRows + r] : 1.f);
        if constexpr (!MOD) xscale[t][e] *= kLog2e;
      }

    float o[NT][D / 16][4];
    float mx[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mx[t][0] = mx[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[t][i][k] = 0.f;
    }
    const int pos_first = u.s.L - u.s.n, pos_last = u.s.L - 1;
    const float icap = MOD == 2 ? 1.f / p.softcap : MOD && p.softcap > 0.f ? 2.f * kLog2e / p.softcap : 0.f;

    for (int step = 0; step < ntile; ++step) {
      cp_wait<NST - 2>();
      __syncwarp();
      const uint32_t st = ring + (step % NST) * C::kStage;
      const int t0 = base + step * C::kKeys;
      float* sc = reinterpret_cast<float*>(smem + (st - smem_u32(smem)) + 2 * C::kTile);
      float4* sk = reinterpret_cast<float4*>(smem + C::oSk) + warp * KS;
      if constexpr (F16) {
        // what this lane's key needs: ks, log2 vs, 1 / vs; a key not read counts as scale 1
        const int t = t0 + lane;
        const float vs = t >= klo && t < khi ? sc[KS + lane] : 1.f;
        float lg;
        asm("lg2.approx.f32 %0, %1;" : "=f"(lg) : "f"(vs));
        sk[lane] = make_float4(sc[lane], lg, rcp_approx(vs), 0.f);
      }
      issue(step + NST - 1);
      lookup(step + NST);
      if (t0 >= khi || t0 + KS <= klo) continue;  // nothing of it is seen
      if constexpr (F16) __syncwarp();
      const bool edge = t0 + KS - 1 > pos_first || t0 < klo || (p.window > 0 && t0 <= pos_last - p.window);
      // 16 keys at a time, a rolled loop: unrolled it costs 40 registers and an
      // occupancy step
#pragma unroll 1
      for (int k0 = 0; k0 < KS; k0 += 16) {
        // ---- S^T = K.Q^T, 16 keys by 8 rows
        float s[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[t][k] = 0.f;
        auto q_frag = [&](int t, int ss) {
          if constexpr (C::kQSmem) return lds8(smem_u32(s_q) + ((t * (D / 16) + ss) * 32 + lane) * 8);
          else return make_uint2(qf[ss][0], qf[ss][1]);
        };
        if constexpr (F16) {
          uint32_t w[2][D / 16];
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
              const uint4 x = lds16(st + k_off<KV, D>(k0 + y * 8 + quad, c * (D / 64) + i));
              w[y][4 * i] = x.x; w[y][4 * i + 1] = x.y; w[y][4 * i + 2] = x.z; w[y][4 * i + 3] = x.w;
            }
#pragma unroll
          for (int ss = 0; ss < D / 16; ++ss) {
            uint32_t a4[4];
            codes4<KV>(w[0][ss], a4[0], a4[2]);
            codes4<KV>(w[1][ss], a4[1], a4[3]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint2 q = q_frag(t, ss);
              mma<F16>(s[t], a4, q.x, q.y);
            }
          }
        } else {
#pragma unroll
          for (int ss = 0; ss < D / 16; ++ss) {
            uint32_t a4[4];
            ldsm4(st + k_off<KV, D>(k0 + (lane & 15), 2 * ss + (lane >> 4)), a4);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint2 q = q_frag(t, ss);
              mma<F16>(s[t], a4, q.x, q.y);
            }
          }
        }
        // ---- scores in log2 units; this lane's keys are k0 + quad and + 8
        float iv[2] = {1.f, 1.f}, ks2[2] = {1.f, 1.f}, lv2[2] = {0.f, 0.f};
        if constexpr (F16) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float4 x = sk[k0 + y * 8 + quad];
            ks2[y] = x.x;
            lv2[y] = x.y;
            iv[y] = x.z;
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e = k & 1, y2 = k >> 1;
            if constexpr (MOD) {
              float y = s[t][k] * xscale[t][e] * ks2[y2];
              if constexpr (MOD == 2) y = cap_any(y, p.softcap, icap);
              else if (p.softcap > 0.f)  // c tanh(y / c) = c - 2 c / (1 + e^(2 y / c))
                y = fmaf(-2.f * p.softcap, rcp_approx(1.f + ex2_approx(y * icap)), p.softcap);
              y = fmaf(slope[t][e], (float)(t0 + k0 + y2 * 8 + quad - pos[t][e]), y);
              s[t][k] = fmaf(y, kLog2e, lv2[y2]);
            } else if constexpr (F16) {
              s[t][k] = fmaf(s[t][k] * ks2[y2], xscale[t][e], lv2[y2]);
            } else {
              s[t][k] *= xscale[t][e];
            }
          }
        if (edge) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = t0 + k0 + (k >> 1) * 8 + quad;
              if (j > pos[t][k & 1] || (p.window > 0 && j <= pos[t][k & 1] - p.window)) s[t][k] = -INFINITY;
            }
        }
        // ---- the running max: only when a score passes it by the lag are the lanes compared
        bool grow = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) grow |= fmaxf(s[t][e], s[t][2 + e]) > mx[t][e] + kLag<F16>;  // from -inf too
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(s[t][e], s[t][2 + e]);
#pragma unroll
              for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              if (top > mx[t][e] + kLag<F16>) {
                const float al = ex2_approx(mx[t][e] - top);
                mx[t][e] = top;
                l[t][e] *= al;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  o[t][i][e] *= al;
                  o[t][i][2 + e] *= al;
                }
              }
            }
        }
        // ---- P^T as B fragments: a row's two keys in one register by a transpose
        uint32_t pf[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float ms[2] = {mx[t][0] == -INFINITY ? 0.f : mx[t][0] - kShift,
                               mx[t][1] == -INFINITY ? 0.f : mx[t][1] - kShift};
          float w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[k] = ex2_approx(s[t][k] - ms[k & 1]);
            if constexpr (F16) l[t][k & 1] = fmaf(w[k], iv[k >> 1], l[t][k & 1]);
            else l[t][k & 1] += w[k];
          }
          uint32_t lo, hi;
          if constexpr (F16) {
            const __half2 h0 = __floats2half2_rn(w[0], w[1]), h1 = __floats2half2_rn(w[2], w[3]);
            memcpy(&lo, &h0, 4);
            memcpy(&hi, &h1, 4);
          } else {
            lo = pack_bf16x2(w[0], w[1]);
            hi = pack_bf16x2(w[2], w[3]);
          }
          pf[t][0] = transpose8(lo);
          pf[t][1] = transpose8(hi);
        }
        // ---- O^T += V^T.P^T
        const uint32_t vt = st + C::kTile;
        if constexpr (F16) {
          constexpr int W = D / 32;  // words of a lane's run of a row
          uint32_t w[4][W];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = k0 + 2 * c + (x & 1) + (x >> 1) * 8;
            if constexpr (D == 128) {
              const uint4 y = lds16(vt + v_off<KV, D>(key, quad));
              w[x][0] = y.x; w[x][1] = y.y; w[x][W - 2] = y.z; w[x][W - 1] = y.w;
            } else {
              const uint2 y = lds8(vt + v_off<KV, D>(key, quad >> 1) + (quad & 1) * 8);
              w[x][0] = y.x; w[x][1] = y.y;
            }
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
            // columns 4 i .. 4 i + 3 of the run: two tiles, column 2 j in rows 0-7, 2 j + 1 in rows 8-15
            uint32_t a4[2][4];
            codes4<KV>(__byte_perm(w[0][i], w[1][i], 0x5140), a4[0][0], a4[0][1]);
            codes4<KV>(__byte_perm(w[0][i], w[1][i], 0x7362), a4[1][0], a4[1][1]);
            codes4<KV>(__byte_perm(w[2][i], w[3][i], 0x5140), a4[0][2], a4[0][3]);
            codes4<KV>(__byte_perm(w[2][i], w[3][i], 0x7362), a4[1][2], a4[1][3]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int y = 0; y < 2; ++y) mma<F16>(o[t][2 * i + y], a4[y], pf[t][0], pf[t][1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t a4[4];
            ldsm4t(vt + v_off<KV, D>(k0 + (lane & 7) + (lane >> 4) * 8, 2 * i + ((lane >> 3) & 1)), a4);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma<F16>(o[t][i], a4, pf[t][0], pf[t][1]);
          }
        }
      }
    }
    cp_wait<0>();

    // ---- the warps' parts into one
    __syncthreads();  // every ring is drained: its space holds the parts now
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], x);
        if (quad == 0) s_ml[warp * C::kRows + t * 8 + 2 * c + e] = make_float2(mx[t][e], l[t][e]);
      }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = t * 8 + 2 * c + e;
        float top = -INFINITY;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w * C::kRows + r].x);
        const float f = mx[t][e] == -INFINITY ? 0.f : ex2_approx(mx[t][e] - top);
        float* dst = mrg + (warp * C::kRows + r) * C::kPitch;
        if (r < u.rows) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            if constexpr (F16) {
              *reinterpret_cast<float2*>(dst + (D / 8) * quad + 2 * i) = make_float2(o[t][i][e] * f, o[t][i][2 + e] * f);
            } else {
              dst[16 * i + quad] = o[t][i][e] * f;
              dst[16 * i + 8 + quad] = o[t][i][2 + e] * f;
            }
          }
        }
      }
    __syncthreads();
    const bool complete = ntile == u.nt;
    const long long slot = 2LL * blockIdx.x + (cur == begin ? 0 : 1);
    if (!a.whole && tile0 == 0 && tid == 0)
      a.ws_unit[(long long)b * p.c.Hkv + hk] =
          make_int4(blockIdx.x, owner(cur + u.nt - 1, T, work_ctas), cur == begin ? 0 : 1, 0);
    for (int i = tid; i < u.rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), x = (i - r * (D / 4)) * 4;
      float top = -INFINITY, den = 0.f;
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w * C::kRows + r].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w * C::kRows + r];
        den = fmaf(ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top), ml.y, den);
        const float4 y = *reinterpret_cast<const float4*>(mrg + (w * C::kRows + r) * C::kPitch + x);
        acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
      }
      if (!complete) {
        *reinterpret_cast<float4*>(a.ws_o + (slot * C::kRows + r) * D + x) = acc;
        if (x == 0) a.ws_ml[slot * C::kRows + r] = make_float2(top, den);
      } else {
        const int tok = r / p.group, h = hk * p.group + r - tok * p.group;
        const float inv = den != 0.f ? 1.f / den : 0.f;
        uint2 y;
        y.x = pack_bf16x2(acc.x * inv, acc.y * inv);
        y.y = pack_bf16x2(acc.z * inv, acc.w * inv);
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (long long)(u.s.q0 + tok) * p.ot + (long long)h * p.oh;
        *reinterpret_cast<uint2*>(dst + x) = y;
        if (x == 0 && p.lse)
          p.lse[(long long)(u.s.q0 + tok) * p.Hq + h] = den != 0.f ? (top - kShift) * kLn2 + logf(den) : -INFINITY;
      }
    }
    __syncthreads();  // before the next unit's copies land in the ring
    cur += ntile;
    if (cur - F == (long long)u.nt * p.c.Hkv) { F = cur; ++b; }
  }

  // rows that see nothing at all
  for (int unit = blockIdx.x; unit < p.s.B * p.c.Hkv; unit += G) {
    const int bb = unit / p.c.Hkv, hk = unit - bb * p.c.Hkv;
    const Unit u = unit_of<C::kKeys>(a, bb);
    if (u.nt != 0) continue;
    if (!a.whole && tid == 0) a.ws_unit[unit] = make_int4(0, 0, 0, 0);
    if (u.rows == 0) continue;
    for (int i = tid; i < u.rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), x = (i - r * (D / 4)) * 4;
      const int tok = r / p.group, h = hk * p.group + r - tok * p.group;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (long long)(u.s.q0 + tok) * p.ot + (long long)h * p.oh;
      *reinterpret_cast<uint2*>(dst + x) = make_uint2(0, 0);
      if (x == 0 && p.lse) p.lse[(long long)(u.s.q0 + tok) * p.Hq + h] = -INFINITY;
    }
  }
}

// Adds the parts of every unit that several CTAs share: O = sum 2^(m_i - M) O_i
// over sum 2^(m_i - M) l_i.  One block per unit, latency-bound: each of its warp
// groups takes every kMergeGroups-th part, loads a part's (m, l) and O together
// and a few parts at a time, and the groups' sums are added in order.
constexpr int kMergeGroups = 4;
template <int D, int ROWS>
__global__ void __launch_bounds__(kMergeGroups * kThreads) paged_merge_kernel(const __grid_constant__ DecodeArgs a,
                                                                             float shift) {
  __shared__ float4 s_acc[kMergeGroups][kThreads];
  __shared__ float2 s_ml[kMergeGroups][kThreads];
  const PagedParams& p = a.p;
  const int b = blockIdx.x / p.c.Hkv, hk = blockIdx.x - b * p.c.Hkv;
  const int group = threadIdx.x / kThreads, tid = threadIdx.x % kThreads;
  grid_dep_wait();
  grid_dep_launch();
  const int4 w = a.ws_unit[blockIdx.x];
  const Seq s = seq_of(p.s, p.c, b, p.err);
  const int c0 = w.x, c1 = w.y;
  if (c0 == c1) return;
  const int items = s.n * p.group * (D / 4);
  for (int i0 = 0; i0 < items; i0 += kThreads) {
    const int i = min(i0 + tid, items - 1);
    const int r = i / (D / 4), x = (i - r * (D / 4)) * 4;
    float top = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAtOnce = 4;
    for (int q0 = c0 + group; q0 <= c1; q0 += kAtOnce * kMergeGroups) {
      float2 ml[kAtOnce];
      float4 y[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int q = q0 + k * kMergeGroups;
        const long long at = (2LL * min(q, c1) + (min(q, c1) == c0 ? w.z : 0)) * ROWS + r;
        ml[k] = a.ws_ml[at];
        y[k] = *reinterpret_cast<const float4*>(a.ws_o + at * D + x);
        if (q > c1) ml[k] = make_float2(-INFINITY, 0.f);
      }
      float m = top;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) m = fmaxf(m, ml[k].x);
      const float old = top == -INFINITY ? 0.f : ex2_approx(top - m);
      top = m;
      den *= old;
      acc.x *= old; acc.y *= old; acc.z *= old; acc.w *= old;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        // a part whose rows saw no key has l = 0 and O = 0; NaN in either passes on
        const float f = ml[k].x == -INFINITY ? 0.f : ex2_approx(ml[k].x - m);
        den = fmaf(f, ml[k].y, den);
        if (q0 + k * kMergeGroups <= c1) {
          acc.x = fmaf(f, y[k].x, acc.x); acc.y = fmaf(f, y[k].y, acc.y);
          acc.z = fmaf(f, y[k].z, acc.z); acc.w = fmaf(f, y[k].w, acc.w);
        }
      }
    }
    s_acc[group][tid] = acc;
    s_ml[group][tid] = make_float2(top, den);
    __syncthreads();
    if (group == 0 && i0 + tid < items) {
      float m = -INFINITY;
#pragma unroll
      for (int k = 0; k < kMergeGroups; ++k) m = fmaxf(m, s_ml[k][tid].x);
      den = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMergeGroups; ++k) {
        const float2 ml = s_ml[k][tid];
        const float4 y = s_acc[k][tid];
        const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
        den = fmaf(f, ml.y, den);
        acc.x = fmaf(f, y.x, acc.x); acc.y = fmaf(f, y.y, acc.y);
        acc.z = fmaf(f, y.z, acc.z); acc.w = fmaf(f, y.w, acc.w);
      }
      const int tok = r / p.group, h = hk * p.group + r - tok * p.group;
      const float inv = den != 0.f ? 1.f / den : 0.f;
      uint2 y;
      y.x = pack_bf16x2(acc.x * inv, acc.y * inv);
      y.y = pack_bf16x2(acc.z * inv, acc.w * inv);
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (long long)(s.q0 + tok) * p.ot + (long long)h * p.oh;
      *reinterpret_cast<uint2*>(dst + x) = y;
      if (x == 0 && p.lse)
        p.lse[(long long)(s.q0 + tok) * p.Hq + h] = den != 0.f ? (m - shift) * kLn2 + logf(den) : -INFINITY;
    }
    __syncthreads();
  }
}

// Raises a kernel's shared-memory limit once per device (`done`: a bit each).
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

template <int KV, int D, int NT>
cudaError_t decode_one(DecodeArgs& a, int mod, int ctas, cudaStream_t stream) {
  using C = Cfg<KV, D, NT>;
  auto kern = mod == 0   ? paged_decode_kernel<KV, D, NT, 0>
              : mod == 1 ? paged_decode_kernel<KV, D, NT, 1>
                         : paged_decode_kernel<KV, D, NT, 2>;
  static std::atomic<uint64_t> done[3];
  cudaError_t e = allow_smem(kern, C::kTotal, done[mod]);
  if (e != cudaSuccess) return e;
  e = launch_serialized(kern, dim3((unsigned)ctas), dim3(kThreads), (size_t)C::kTotal, stream, a);
  if (e != cudaSuccess || a.whole) return e;
  return launch_serialized(paged_merge_kernel<D, C::kRows>, dim3((unsigned)(a.p.s.B * a.p.c.Hkv)),
                           dim3(kMergeGroups * kThreads), 0, stream, a, kOffset<KV != KV_BF16>);
}
template <int KV, int D>
cudaError_t decode_rows(DecodeArgs& a, int mod, int ctas, cudaStream_t stream) {
  switch (a.limit) {
    case 8: return decode_one<KV, D, 1>(a, mod, ctas, stream);
    case 16: return decode_one<KV, D, 2>(a, mod, ctas, stream);
    case 24: return decode_one<KV, D, 3>(a, mod, ctas, stream);
    default: return decode_one<KV, D, 4>(a, mod, ctas, stream);
  }
}

// Rows a call's sequences may have here: the fewest row tiles that hold the
// bound max_q gives, at most 32 rows.
int row_limit(const PagedParams& p) {
  const long long rows = (long long)p.s.max_q * p.group;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : kDecodeRows;
}

// One resident wave.
int decode_ctas(const PagedParams& p) {
  return num_sms() * (p.c.dtype != SDPA_CACHE_BF16 && row_limit(p) <= 16 ? 3 : 2);
}

// One CTA per unit and no merge launch where splitting the keys would cost more
// than it gives: where no sequence reaches past 512 keys (one of 131 tokens: 8.5
// us against 12.4, graph replay), and, with a unit for every SM, past 1088 (32
// sequences of up to 1024, bf16: 17.9 against 22.0; 24 with drafts, e4m3: 26.7
// against 43.7; a window of 1024: 18.7 against 22.8), or past 2176 while all
// units are resident at once (32 of up to 2048, bf16: 37.6 against 41.3; beyond
// one wave the tail costs more: 64 of up to 2048, e4m3: 63.8 against 56.0).
bool whole_units(const PagedParams& p) {
  const long long cap = (long long)p.s.max_pages * p.c.page_size, units = (long long)p.s.B * p.c.Hkv;
  const long long reach = p.window > 0 ? std::min(cap, (long long)p.window + p.s.max_q + 16) : cap;
  return reach <= 512 || (units >= num_sms() && reach <= (units <= decode_ctas(p) ? 2176 : 1088));
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int paged_decode_check(const PagedParams& p, sdpa_dtype_t dtype) {
  const CacheView& c = p.c;
  if (dtype != SDPA_BF16 || c.dtype == SDPA_CACHE_F32 || c.d == 16) return SDPA_ERR_UNSUPPORTED;
  if (c.page_size % 16 != 0 || p.group > kDecodeRows) return SDPA_ERR_UNSUPPORTED;
  if ((long long)p.s.B * c.Hkv > 0x7fffffffLL) return SDPA_ERR_UNSUPPORTED;
  const long long es = c.dtype == SDPA_CACHE_BF16 ? 2 : 1;
  const long long bytes[] = {c.kp * es, c.kh * es, c.kt * es, c.vp * es, c.vh * es, c.vt * es, p.qt * 2, p.qh * 2};
  for (long long x : bytes)
    if (x % 16 != 0) return SDPA_ERR_MISALIGNED;
  // strides of a page, and offsets inside one, in 32 bits
  const long long wide[] = {c.kp * es, c.vp * es, c.kt * es, c.vt * es, c.kst, c.vst, c.kt * es * c.page_size, c.vt * es * c.page_size, c.ksp, c.vsp,
                            c.kst * c.page_size, c.vst * c.page_size};
  for (long long x : wide)
    if (x > 0x7fffffffLL) return SDPA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) | reinterpret_cast<uintptr_t>(p.q)) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(p.out) % 8 != 0 || p.ot % 4 != 0 || p.oh % 4 != 0)
    return SDPA_ERR_MISALIGNED;
  return SDPA_OK;
}

size_t paged_decode_workspace(const PagedParams& p) {
  if (whole_units(p) || p.s.total_q == 0) return 0;
  const size_t slots = 2 * (size_t)decode_ctas(p), rows = row_limit(p);
  return up256(slots * rows * p.c.d * 4) + up256(slots * rows * 8) + up256((size_t)p.s.B * p.c.Hkv * 16);
}

cudaError_t launch_paged_decode(const PagedParams& p, void* ws, cudaStream_t stream) {
  DecodeArgs a;
  memset(&a, 0, sizeof(a));
  a.p = p;
  a.limit = row_limit(p);
  a.whole = whole_units(p);
  const int ctas = a.whole ? p.s.B * p.c.Hkv : decode_ctas(p);
  if (!a.whole) {
    const size_t slots = 2 * (size_t)ctas, rows = a.limit;
    char* w = static_cast<char*>(ws);
    a.ws_o = reinterpret_cast<float*>(w);
    w += up256(slots * rows * p.c.d * 4);
    a.ws_ml = reinterpret_cast<float2*>(w);
    w += up256(slots * rows * 8);
    a.ws_unit = reinterpret_cast<int4*>(w);
  }
  const CacheView& c = p.c;
  const uint32_t es = c.dtype == SDPA_CACHE_BF16 ? 2 : 1;
  a.kp = (uint32_t)(c.kp * es); a.vp = (uint32_t)(c.vp * es); a.kt = (uint32_t)(c.kt * es); a.vt = (uint32_t)(c.vt * es);
  a.ksp = (uint32_t)c.ksp; a.vsp = (uint32_t)c.vsp; a.kst = (uint32_t)c.kst; a.vst = (uint32_t)c.vst;
  a.dense = c.kt == c.d && c.vt == c.d;
  const int mod = p.softcap > kPlainCap ? 2 : p.softcap > 0.f || p.slopes != nullptr ? 1 : 0;
  const bool wide = p.c.d == 128;
  switch (p.c.dtype) {
    case SDPA_CACHE_BF16: return wide ? decode_rows<KV_BF16, 128>(a, mod, ctas, stream) : decode_rows<KV_BF16, 64>(a, mod, ctas, stream);
    case SDPA_CACHE_E4M3: return wide ? decode_rows<KV_E4M3, 128>(a, mod, ctas, stream) : decode_rows<KV_E4M3, 64>(a, mod, ctas, stream);
    case SDPA_CACHE_INT8: return wide ? decode_rows<KV_INT8, 128>(a, mod, ctas, stream) : decode_rows<KV_INT8, 64>(a, mod, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
