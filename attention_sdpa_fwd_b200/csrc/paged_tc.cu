// Attention of chunks of new tokens over a paged cache on the tensor cores:
// TMA + tcgen05/TMEM, online softmax, for sequences whose (token, head) rows
// per kv head are too many for the decode kernel.
//
// A unit is 256 rows of one (sequence, kv head), two tiles of 128: row r of a
// tile is token r / G, query head r % G of the G heads that share the kv head,
// so a tile is full whatever G is, K and V are read once for all G heads, and
// the causal diagonal costs 128 / G tokens.  Q comes as one TMA box
// (64 columns, G heads, 128 / G tokens) per panel.  Roles, 384 threads, 512 for codes:
//   warps 0-3, 4-7  softmax of tile A, B (thread = row = TMEM lane)
//   warp  8         producer: K / V pages by TMA, one box per run of tokens
//                   inside a page, page numbers a tile ahead
//   warp  9         TMEM owner, MMA issuer
//   warps 12-15     codes: the converters (10 and 11 idle)
// The tile pipeline (S_t = Q_t.K^T, softmax, O_t += P_t.V, stale-max rescale)
// is that of the dense kernel, flash_tc.cu: at head_dim 128 P_t overwrites S_t,
// at 64 it has its own columns and S_t runs a tile ahead.
//
// 8-bit caches: raw pages land in a ring of 64-key pieces, and four converter
// warps, 32 keys of a tile each, turn codes into f16 in the K / V stages, in the
// 128-byte swizzle the MMA reads.  Every row is multiplied by its scale on the
// way, relative to a power of two 2^e of its 32 keys that puts their largest
// scale in [64, 128): code * scale 2^-e is below 57344 and is rounded
// once, to f16 (2^-11; the scale enters as a sum of two f16), eight times finer
// than the bf16 the cache stands in for.  What the softmax warps see of it is a
// factor 2^ek for 32 scores and, for V, an offset ev of 32 exponents:
//     p_j = 2^(x_j log2e + ev - m),  out = sum p_j v_j 2^-ev / sum p_j 2^-ev
// (Scales by column there, exact, cost three shared-memory vectors per row and
// tile and twice the time.)  The softmax warps scale their Q row in place by a
// power of two into f16, its largest element to [2^14, 2^15).  P is f16 as in
// the decode kernel: at most 2^15, offset by 2^12; beside bf16 values it is bf16,
// for the reason given there.
//
// Units of one launch differ in length (causal), so later query blocks, the
// longer ones, start first.  When there are fewer units than SMs every unit's
// keys are split into parts that write (O, max, sum) to the workspace, and a
// second kernel adds them in order: no atomics, nothing kept between calls.
#include <math.h>
#include <string.h>

#include <mutex>

#include "paged.cuh"
#include "pdl_launch.cuh"
#include "softmax_tile.cuh"
#include "tmap.h"

namespace sdpa {
namespace {

using namespace sm100;

// Codes take four more warps, the converters.
template <int KV> constexpr int kThreadsOf = KV == 0 ? 384 : 512;
constexpr int kRows = 128;           // of a tile
constexpr int BN = 128;              // keys of a tile
constexpr int kHalf = 64;            // keys of a raw piece
constexpr int kMaxSplit = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
template <int KV> constexpr int kRegsLaunch = KV == 0 ? 168 : 128;  // registers a thread is launched with

enum { KV_BF16 = 0, KV_E4M3 = 1, KV_INT8 = 2 };

struct TcPagedArgs {
  CUtensorMap tq;      // (d, head, token), box 64 x G x tokens of a tile
  CUtensorMap tk, tv;  // (d, token of a page, head, page), box (64 | d) x box_rows
  PagedParams p;
  int tok;             // tokens of a tile: 128 / G
  int box_rows;        // tokens of a K / V box
  int limit;           // sequences of up to this many rows are the decode kernel's (0: none)
  int n_split;
  float* ws_o;         // [units][n_split][D / 4][256] float4
  float2* ws_ml;       // [units][n_split][256]
  FastDiv fd_split, fd_hkv, fd_g;
};

template <int KV, int D>
struct TcLayout {
  static constexpr bool kCodes = KV != KV_BF16;
  static constexpr int NS = D == 64 ? 3 : 2;
  static constexpr int NR = 4;                      // raw pieces; even: each converter has its own
  static constexpr int SR = D == 64 ? 8 : 4;        // tiles whose exponents are kept: see the converters
  static constexpr int kPanels = D / 64;
  static constexpr int kQBytes = kPanels * kRows * 128;
  static constexpr int kKVBytes = kPanels * BN * 128;
  static constexpr int kRaw = kCodes ? kHalf * D : 0;
  static constexpr int oQ = 0;
  static constexpr int oK = oQ + 2 * kQBytes;
  static constexpr int oV = oK + NS * kKVBytes;
  static constexpr int oRaw = oV + NS * kKVBytes;
  static constexpr int oSc = oRaw + NR * kRaw;       // [SR][4] float4: 2^ek, ev, 2^-ev of 32 keys
  static constexpr int oBar = oSc + (kCodes ? SR * 4 * 16 : 0);
  static constexpr int kBars = 4 * NS + 16 + 2 * NR + SR;
  static constexpr int kTotal = oBar + kBars * 8 + 64;
  static constexpr int kAlloc = kTotal + 1024;
  static_assert(kAlloc <= 232448, "shared memory budget");
};

// What a CTA works on.
struct TcUnit {
  Seq s;
  int b, hk;
  int tok0;      // first token of the unit
  int lo, hi;    // keys any of its rows sees
  int jb, je;    // their tiles
};

__device__ __forceinline__ int blocks_of(const TcPagedArgs& a, int b) {
  const Seq s = seq_of(a.p.s, a.p.c, b, a.p.err);
  if (s.n <= a.limit / a.p.group) return 0;
  return (s.n + 2 * a.tok - 1) / (2 * a.tok);
}

// Unit `unit` of the launch, blocks numbered from the last one down; false past
// the last.  The whole CTA takes part.
template <int kThreads>
__device__ __forceinline__ bool find_unit(const TcPagedArgs& a, int unit, TcUnit& u) {
  __shared__ int s_part[kThreads / 32], s_found[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blk = (int)fdiv((uint32_t)unit, a.fd_hkv);
  u.hk = unit - blk * a.p.c.Hkv;
  if (a.p.s.B == 1) {
    const int n = blocks_of(a, 0);
    if (blk >= n) return false;
    u.b = 0;
    u.tok0 = (n - 1 - blk) * 2 * a.tok;
  } else {
    const int per = (a.p.s.B + kThreads - 1) / kThreads;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < a.p.s.B) mine += blocks_of(a, b);
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_part[warp] = incl;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) incl += s_part[w];
      total += s_part[w];
    }
    if (blk >= total) return false;
    const int want = total - 1 - blk;
    int at = incl - mine;
    if (want >= at && want < incl) {
      int b = tid * per;
      for (;; ++b) {
        const int n = blocks_of(a, b);
        if (want < at + n) break;
        at += n;
      }
      s_found[0] = b;
      s_found[1] = want - at;
    }
    __syncthreads();
    u.b = s_found[0];
    u.tok0 = s_found[1] * 2 * a.tok;
  }
  u.s = seq_of(a.p.s, a.p.c, u.b, a.p.err);
  const int first = u.s.L - u.s.n + u.tok0, last = u.s.L - u.s.n + min(u.tok0 + 2 * a.tok, u.s.n) - 1;
  u.hi = max(0, last + 1);
  u.lo = a.p.window > 0 ? max(0, first + 1 - a.p.window) : 0;
  u.jb = u.lo / BN;
  u.je = u.hi > u.lo ? (u.hi + BN - 1) / BN : u.jb;
  return true;
}

// The smaller, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// Four scores x in log2 units to c tanh(x / c) = c - 2 c / (1 + 2^(2 x / c)),
// one reciprocal for the four: 1 / a = b c d / (a b c d).  The exponent is kept
// below 30, where tanh is 1 - 2^-29, so that the product stays finite.
// (The multi-function unit bounds capped scores: 2.25 operations a score
// instead of 3.)  A NaN reaches all four.
__device__ __forceinline__ void cap4(uint64_t& x, uint64_t& y, float cap_in, float cap_out) {
  float v[4], a[4];
  f2_split(x, v[0], v[1]);
  f2_split(y, v[2], v[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = 1.f + ex2_approx(min_nan(v[i] * cap_in, 30.f));
  const float ab = a[0] * a[1], cd = a[2] * a[3];
  const float r = rcp_approx(ab * cd) * (-2.f * cap_out);
  const float rab = r * cd, rcd = r * ab;
  x = f2(fmaf(rab, a[1], cap_out), fmaf(rab, a[0], cap_out));
  y = f2(fmaf(rcd, a[3], cap_out), fmaf(rcd, a[2], cap_out));
}

// MOD: 0 plain scores and a positive scale, 1 with slopes (which may be zero), 2
// capped and with slopes, 3 the same for caps above kPlainCap.
template <int KV, int D, int MOD>
__global__ void __launch_bounds__(kThreadsOf<KV>, 1) paged_tc_kernel(const __grid_constant__ TcPagedArgs args) {
  using L = TcLayout<KV, D>;
  constexpr bool kCodes = L::kCodes;
  constexpr bool kPSep = D == 64;
  constexpr int NS = L::NS, NR = L::NR, SR = L::SR;
  constexpr float kLag = kCodes ? 3.f : 8.f, kOffset = kCodes ? 12.f : 0.f;
  // setmaxnreg: what the softmax warpgroups get the other one (codes: two) gave up
  constexpr int kRegsSoftmax = kCodes ? 192 : 216, kRegsOther = kCodes ? 64 : 72;
  static_assert(256 * kRegsSoftmax + (kThreadsOf<KV> - 256) * kRegsOther <= kThreadsOf<KV> * kRegsLaunch<KV>, "register split");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem + L::oQ;
  uint8_t* sK = smem + L::oK;
  uint8_t* sV = smem + L::oV;
  uint8_t* sRaw = smem + L::oRaw;
  float4* sSc = reinterpret_cast<float4*>(smem + L::oSc);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::oBar);
  uint64_t* k_full = bars;
  uint64_t* v_full = bars + NS;
  uint64_t* k_empty = bars + 2 * NS;
  uint64_t* v_empty = bars + 3 * NS;
  uint64_t* q_full = bars + 4 * NS;
  uint64_t* q_ready = q_full + 1;   // codes: Q rows are f16
  uint64_t* s_full = q_full + 2;    // [2]
  uint64_t* p_full = q_full + 4;    // [2]
  uint64_t* o_done = q_full + 6;    // [2]
  uint64_t* s_free = q_full + 8;    // [2]
  uint64_t* o_ready = q_full + 10;  // [2]
  uint64_t* fin = q_full + 12;
  uint64_t* raw_full = q_full + 16;
  uint64_t* raw_empty = raw_full + NR;
  uint64_t* sc_full = raw_empty + NR;  // [SR]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + L::kBars);
  int* abort_flag = reinterpret_cast<int*>(tslot + 1);

  const PagedParams& p = args.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dep_wait();
  grid_dep_launch();
  const int unit = (int)fdiv(blockIdx.x, args.fd_split);
  const int sidx = blockIdx.x - unit * args.n_split;
  TcUnit u;
  if (!find_unit<kThreadsOf<KV>>(args, unit, u)) return;
  const int span = u.je - u.jb;
  const int j_begin = u.jb + (int)fdiv((uint32_t)(span * sidx), args.fd_split);
  const int n_tiles = u.jb + (int)fdiv((uint32_t)(span * (sidx + 1)), args.fd_split) - j_begin;
  const int klo = u.lo, khi = u.hi;
  // tiles of this CTA that hold rows outside [klo, khi)
  auto edge_tile = [&](int j) { return j * BN < klo || j * BN + BN > khi; };

  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < L::kBars; ++i) mbar_init(&bars[i], 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&p_full[t], kRows);
      mbar_init(&s_free[t], kRows);
    }
    mbar_init(q_ready, 2 * kRows);
    if (kCodes) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(&k_full[i], 4);
        mbar_init(&v_full[i], 4);
      }
      for (int i = 0; i < NR; ++i) mbar_init(&raw_empty[i], 2);
      for (int i = 0; i < SR; ++i) mbar_init(&sc_full[i], 4);
    }
    fence_mbar_init();
    if (n_tiles > 0) {
      tma_prefetch_desc(&args.tk);
      tma_prefetch_desc(&args.tv);
      mbar_expect_tx(q_full, 2 * L::kPanels * args.tok * p.group * 128);
      for (int t = 0; t < 2; ++t)
        for (int pn = 0; pn < L::kPanels; ++pn)
          tma_load_3d(sQ + t * L::kQBytes + pn * kRows * 128, &args.tq, q_full, pn * 64, u.hk * p.group,
                      u.s.q0 + u.tok0 + t * args.tok);
    }
  }
  if (warp == 9) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  volatile int* abort_v = abort_flag;
  auto wait_all = [](bool v) { return __all_sync(0xffffffffu, v) != 0; };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsOther));
    if (warp == 8 && n_tiles > 0) {
      // ------------------------------------------------------------ producer
      // Lane i has box i of a tile (bf16) or of a half (codes); its page number
      // is fetched an item ahead.
      constexpr int kItem = kCodes ? kHalf : BN;  // keys of what one barrier phase brings
      const int rows = args.box_rows, boxes = kItem / rows;
      auto page_at = [&](int key) {  // of the box that starts at `key`; past the pool: zeros
        return lane < boxes && key + rows > klo && key < khi ? page_of(p.s, p.c, u.b, max(key, klo), p.err)
                                                             : p.c.num_pages;
      };
      auto box_key = [&](int key0) { return key0 + lane * rows; };
      auto in_page = [&](int key) { return key - (int)fdiv((uint32_t)key, p.c.fd_page) * p.c.page_size; };
      bool ok = true;
      int k_issued = 0, v_issued = 0, r_issued = 0;
      if constexpr (!kCodes) {
        auto load = [&](bool is_v, int jj, int page) {
          const int s = jj % NS, use = jj / NS;
          if (use > 0) ok = wait_all(mbar_wait(is_v ? &v_empty[s] : &k_empty[s], (use - 1) & 1, abort_v, p.err));
          if (!ok) return;
          uint64_t* bar = is_v ? &v_full[s] : &k_full[s];
          if (lane == 0) mbar_expect_tx(bar, L::kKVBytes);
          __syncwarp();
          if (lane < boxes) {
            uint8_t* dst = (is_v ? sV : sK) + s * L::kKVBytes + lane * rows * 128;
            const int y = in_page(box_key((j_begin + jj) * BN));
            for (int pn = 0; pn < L::kPanels; ++pn)
              tma_load_4d(dst + pn * BN * 128, is_v ? &args.tv : &args.tk, bar, pn * 64, y, u.hk, page);
          }
          (is_v ? v_issued : k_issued) = jj + 1;
        };
        int pg = page_at(box_key(j_begin * BN)), pg_prev = 0;
        for (int jj = 0; jj < n_tiles && ok; ++jj) {
          const int next = jj + 1 < n_tiles ? page_at(box_key((j_begin + jj + 1) * BN)) : 0;
          load(false, jj, pg);
          if (ok && jj > 0) load(true, jj - 1, pg_prev);
          pg_prev = pg;
          pg = next;
        }
        if (ok) load(true, n_tiles - 1, pg_prev);
        if (!ok) {  // abandoned: what is in flight lands before the CTA leaves
          mbar_wait(q_full, 0, nullptr, p.err);
          for (int jj = max(0, k_issued - NS); jj < k_issued; ++jj)
            mbar_wait(&k_full[jj % NS], (jj / NS) & 1, nullptr, p.err);
          for (int jj = max(0, v_issued - NS); jj < v_issued; ++jj)
            mbar_wait(&v_full[jj % NS], (jj / NS) & 1, nullptr, p.err);
        }
      } else {
        auto load = [&](bool is_v, int key0, int page) {
          const int s = r_issued % NR, use = r_issued / NR;
          if (use > 0) ok = wait_all(mbar_wait(&raw_empty[s], (use - 1) & 1, abort_v, p.err));
          if (!ok) return;
          if (lane == 0) mbar_expect_tx(&raw_full[s], L::kRaw);
          __syncwarp();
          if (lane < boxes)
            tma_load_4d(sRaw + s * L::kRaw + lane * rows * D, is_v ? &args.tv : &args.tk, &raw_full[s], 0,
                        in_page(box_key(key0)), u.hk, page);
          ++r_issued;
        };
        int pg[2];
        for (int x = 0; x < 2; ++x) pg[x] = page_at(box_key(j_begin * BN + x * kHalf));
        for (int jj = 0; jj < n_tiles && ok; ++jj) {
          const int key0 = (j_begin + jj) * BN;
          int nx[2] = {0, 0};
          if (jj + 1 < n_tiles)
            for (int x = 0; x < 2; ++x) nx[x] = page_at(box_key(key0 + BN + x * kHalf));
          for (int y = 0; y < 4 && ok; ++y) load(y >= 2, key0 + (y & 1) * kHalf, y & 1 ? pg[1] : pg[0]);
          pg[0] = nx[0];
          pg[1] = nx[1];
        }
        if (!ok) {
          mbar_wait(q_full, 0, nullptr, p.err);
          for (int r = max(0, r_issued - NR); r < r_issued; ++r)
            mbar_wait(&raw_full[r % NR], (r / NR) & 1, nullptr, p.err);
        }
      }
    } else if (warp == 9 && n_tiles > 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t fmt = kCodes ? ~((1u << 7) | (1u << 10)) : ~0u;  // f16 operands instead of bf16
      constexpr uint32_t id_qk = idesc_bf16_f32(128, BN, false, false) & fmt;
      constexpr uint32_t id_pv = idesc_bf16_f32(128, D, false, true) & fmt;
      const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dv = sdesc_sw128(smem_u32(sV), BN * 128, 1024);
      bool ok = wait_all(mbar_wait(kCodes ? q_ready : q_full, 0, abort_v, p.err));
      auto qk = [&](int t, int s) {
        const uint64_t a0 = dq + (uint64_t)((t * L::kQBytes) >> 4);
        const uint64_t b0 = dk + (uint64_t)((s * L::kKVBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ao = ((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4;
          const uint32_t bo = ((kk >> 2) * (BN * 128) + (kk & 3) * 32) >> 4;
          mma_ss_w(tbase + t * 128, a0 + ao, b0 + bo, id_qk, kk > 0);
        }
      };
      auto pv = [&](int t, int s, bool first) {
        const uint64_t b0 = dv + (uint64_t)((s * L::kKVBytes) >> 4);
        const uint32_t a_tm = kPSep ? tbase + 384 + t * 64 : tbase + t * 128;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_ts_w(tbase + 256 + t * D, a_tm + kk * 8, b0 + (uint64_t)((kk * 16 * 128) >> 4), id_pv, (!first) || kk > 0);
      };
      auto wait_v = [&](int jj) {
        bool r = wait_all(mbar_wait(&v_full[jj % NS], (jj / NS) & 1, abort_v, p.err));
        if (!kCodes && r && edge_tile(j_begin + jj)) {
          // rows of V that stand for no visible key: 0 x NaN would be NaN.  At
          // most the first and the last tile of a unit, so this warp does it.
          const int key0 = (j_begin + jj) * BN;
          uint8_t* v = sV + (jj % NS) * L::kKVBytes + (lane & 7) * 16;
          for (int x = lane >> 3; x < BN * L::kPanels; x += 4) {
            const int key = key0 + (x & (BN - 1));
            if (key < klo || key >= khi) *reinterpret_cast<uint4*>(v + x * 128) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_shared();
          __syncwarp();
        }
        return r;
      };
      if (ok) ok = wait_all(mbar_wait(&k_full[0], 0, abort_v, p.err));
      if (ok) {
        tc_fence_after();
        qk(0, 0);
        mma_commit_w(&s_full[0]);
        qk(1, 0);
        mma_commit_w(&s_full[1]);
        mma_commit_w(&k_empty[0]);
      }
      for (int jj = 0; jj < n_tiles && ok; ++jj) {
        const int s = jj % NS, s1 = (jj + 1) % NS;
        const bool more = jj + 1 < n_tiles;
        if constexpr (kPSep) {
          if (more) {
            ok = wait_all(mbar_wait(&k_full[s1], ((jj + 1) / NS) & 1, abort_v, p.err));
            if (ok) ok = wait_all(mbar_wait(&s_free[0], jj & 1, abort_v, p.err));
            if (!ok) break;
            tc_fence_after();
            qk(0, s1);
            mma_commit_w(&s_full[0]);
          }
          ok = wait_v(jj);
          if (ok) ok = wait_all(mbar_wait(&p_full[0], jj & 1, abort_v, p.err));
          if (!ok) break;
          tc_fence_after();
          pv(0, s, jj == 0);
          mma_commit_w(&o_ready[0]);
          if (more) {
            ok = wait_all(mbar_wait(&s_free[1], jj & 1, abort_v, p.err));
            if (!ok) break;
            tc_fence_after();
            qk(1, s1);
            mma_commit_w(&s_full[1]);
            mma_commit_w(&k_empty[s1]);
          }
          ok = wait_all(mbar_wait(&p_full[1], jj & 1, abort_v, p.err));
          if (!ok) break;
          tc_fence_after();
          pv(1, s, jj == 0);
          mma_commit_w(&o_ready[1]);
          mma_commit_w(&v_empty[s]);
        } else {
          ok = wait_v(jj);
          if (ok) ok = wait_all(mbar_wait(&p_full[0], jj & 1, abort_v, p.err));
          if (!ok) break;
          tc_fence_after();
          pv(0, s, jj == 0);
          if (more) {
            ok = wait_all(mbar_wait(&k_full[s1], ((jj + 1) / NS) & 1, abort_v, p.err));
            if (!ok) break;
            tc_fence_after();
            qk(0, s1);
            mma_commit_w(&s_full[0]);
          }
          ok = wait_all(mbar_wait(&p_full[1], jj & 1, abort_v, p.err));
          if (!ok) break;
          tc_fence_after();
          pv(1, s, jj == 0);
          mma_commit_w(&v_empty[s]);
          if (more) {
            qk(1, s1);
            mma_commit_w(&s_full[1]);
            mma_commit_w(&k_empty[s1]);
          }
        }
      }
      mma_commit_w(&o_done[0]);
      mma_commit_w(&o_done[1]);
    } else if (kCodes && warp >= 12 && n_tiles > 0) {
      // ------------------------------------------------------------ converters
      // Warp 12 + i has keys 32 i .. of every tile, a key per lane.
      const int part = warp - 12, half = part >> 1;
      bool ok = true;
      int r_next = half;  // raw pieces alternate between the halves
      // The scales of this lane's key: its page number is fetched two tiles
      // ahead, the scales one, so neither load is waited for.
      float ks_n = 0.f, vs_n = 0.f;
      int pg_n = 0;
      auto seen_key = [&](int jj) {
        const int key = (j_begin + jj) * BN + part * 32 + lane;
        return jj < n_tiles && key >= klo && key < khi ? key : -1;
      };
      auto fetch_page = [&](int jj) {
        const int key = seen_key(jj);
        pg_n = key >= 0 ? page_entry(p.s, p.c, u.b, key) : 0;
      };
      auto fetch_scales = [&](int jj) {
        const int key = seen_key(jj);
        ks_n = vs_n = 0.f;  // rows nobody sees become zeros
        if (key >= 0) {
          const long long pg = max(0, good_page(p.c, pg_n, p.err));
          const int off = key - (int)fdiv((uint32_t)key, p.c.fd_page) * p.c.page_size;
          ks_n = ld_prior(p.c.ks + pg * p.c.ksp + u.hk * p.c.ksh + off * p.c.kst);
          vs_n = ld_prior(p.c.vs + pg * p.c.vsp + u.hk * p.c.vsh + off * p.c.vst);
        }
      };
      // The largest finite scale's exponent less 6 (a row with an infinite one
      // becomes NaN whatever it is relative to), and scale 2^-e of a key as the
      // sum of two f16 (the first in the low half).
      auto common = [&](float s) {
        const unsigned top = __reduce_max_sync(0xffffffffu, s < INFINITY ? __float_as_uint(s) : 0u);
        return max(-36, (int)(top >> 23) - 127 - 6);
      };
      auto two_halves = [](float s, int e) {
        const float r = s * __uint_as_float((uint32_t)(127 - e) << 23);
        const __half hi = __float2half_rn(r);
        const __half lo = __float2half_rn(r - __half2float(hi));
        return (uint32_t)__half_as_ushort(hi) | ((uint32_t)__half_as_ushort(lo) << 16);
      };
      constexpr int kPieces = D / 16;        // of a row, 16 codes each
      constexpr int kPass = 32 / kPieces;    // rows of a pass
      const int pc = lane % kPieces, r0 = lane / kPieces;
      fetch_page(0);
      fetch_scales(0);
      fetch_page(1);
      uint32_t v_scale = 0;
      // K(j) and V(j) in turn, in one rolled loop: unrolled twice over, this
      // code and the softmax warps' do not fit the instruction cache together
      // (2048 new tokens behind 6144, e4m3: 519 us, rolled 313)
#pragma unroll 1
      for (int it = 0; it < 2 * n_tiles && ok; ++it) {
        const bool is_v = it & 1;
        const int jj = it >> 1, s = jj % NS, use = jj / NS;
        uint32_t scales = v_scale;
        if (use > 0) ok = wait_all(mbar_wait(is_v ? &v_empty[s] : &k_empty[s], (use - 1) & 1, abort_v, p.err));
        if (!ok) break;
        if (!is_v) {
          const int ek = common(ks_n), ev = common(vs_n);
          scales = two_halves(ks_n, ek);
          v_scale = two_halves(vs_n, ev);
          // The tile that used this slot, jj - SR, is behind every softmax
          // warp: K stage jj % NS being free means S(jj - NS) is complete, and
          // that S is only issued once tile jj - NS - 1's scores (head_dim 64)
          // or P (128) were taken from tensor memory: tiles up to jj - NS - 2
          // (64) or jj - NS - 1 (128) are finished, and SR >= NS + 2.
          if (lane == 0) {
            sSc[(jj % SR) * 4 + part] = make_float4(__uint_as_float((uint32_t)(127 + ek) << 23), (float)ev,
                                                    __uint_as_float((uint32_t)(127 - ev) << 23), 0.f);
            mbar_arrive(&sc_full[jj % SR]);
          }
          fetch_scales(jj + 1);
          fetch_page(jj + 2);
        }
        const int rs = r_next % NR;
        ok = wait_all(mbar_wait(&raw_full[rs], (r_next / NR) & 1, abort_v, p.err));
        if (!ok) break;
        const int key0 = (j_begin + jj) * BN + part * 32;
        const bool all = key0 >= klo && key0 + 32 <= khi;
        const uint8_t* src = sRaw + rs * L::kRaw + ((part & 1) * 32 + r0) * D + pc * 16;
        // codes 16 pc ..: panel pc / 4, 16-byte chunks 2 (pc % 4) and the next, at chunk ^ (row % 8)
        uint8_t* line = (is_v ? sV : sK) + s * L::kKVBytes + (pc >> 2) * BN * 128 + (part * 32 + r0) * 128;
        const int c0 = 2 * (pc & 3);
        constexpr int kBatch = 4;  // pieces loaded together
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += kBatch * kPass) {
          uint4 w[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            w[i] = *reinterpret_cast<const uint4*>(src + (i0 + i * kPass) * D);
            const int key = key0 + i0 + i * kPass + r0;
            if (!all && (key < klo || key >= khi)) w[i] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int first = i0 + i * kPass;  // this warp's row first + r0
            const uint32_t sc = __shfl_sync(0xffffffffu, scales, first + r0);
            const uint32_t hi2 = __byte_perm(sc, 0, 0x1010), lo2 = __byte_perm(sc, 0, 0x3232);
            __half2 shi, slo;
            memcpy(&shi, &hi2, 4);
            memcpy(&slo, &lo2, 4);
            const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t h[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if constexpr (KV == KV_E4M3) {
                e4m3x4_to_half2(ws[q], h[2 * q], h[2 * q + 1]);
              } else {
                const uint32_t y = ws[q] ^ 0x80808080u;
                h[2 * q] = biased_bytes_to_half2(y, 0x4140);
                h[2 * q + 1] = biased_bytes_to_half2(y, 0x4342);
              }
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              __half2 c;
              memcpy(&c, &h[q], 4);
              c = __hfma2(c, shi, __hmul2(c, slo));
              memcpy(&h[q], &c, 4);
            }
            const int sw = (first + r0) & 7;
            *reinterpret_cast<uint4*>(line + first * 128 + ((c0 ^ sw) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(line + first * 128 + (((c0 + 1) ^ sw) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[rs]);
          mbar_arrive(is_v ? &v_full[s] : &k_full[s]);
        }
        r_next += 2;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------ softmax of tile t
    const int t = warp >> 2;
    const int lr = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tbase + lane_off + t * 128;
    const uint32_t o_addr = tbase + lane_off + 256 + t * D;
    const uint32_t p_addr = kPSep ? tbase + lane_off + 384 + t * 64 : s_addr;
    const int tk = (int)fdiv((uint32_t)lr, args.fd_g), g = lr - tk * p.group;
    const int i = u.tok0 + t * args.tok + tk;  // token of the sequence's new ones
    const bool row_valid = tk < args.tok && i < u.s.n;
    const int h = u.hk * p.group + g;
    const int pos = u.s.L - u.s.n + i;
    int lo_i, hi_i;
    seen(p, pos, lo_i, hi_i);
    if (!row_valid) { lo_i = 0; hi_i = 0x7fffffff; }  // its scores are never used: no masking work
    bool ok = true;
    float xs = p.scale * kLog2e;  // accumulator to log2 units (codes: times ks)
    if constexpr (kCodes) {
      if (n_tiles > 0) {
        // this row of Q from bf16 to f16, in place
        ok = wait_all(mbar_wait(q_full, 0, abort_v, p.err));
        uint8_t* row = sQ + t * L::kQBytes + lr * 128;
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(row + (c >> 3) * kRows * 128 + (((c & 7) ^ (lr & 7)) << 4));
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[q] << 16)), fabsf(__uint_as_float(x[q] & 0xffff0000u))));
        }
        const int ex = top > 0.f && top < INFINITY ? min(126, max(-126, 141 - (int)(__float_as_uint(top) >> 23))) : 0;
        const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
        xs *= __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint4* at = reinterpret_cast<uint4*>(row + (c >> 3) * kRows * 128 + (((c & 7) ^ (lr & 7)) << 4));
          const uint4 w = *at;
          uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const __half2 hh = __floats2half2_rn(__uint_as_float(x[q] << 16) * up, __uint_as_float(x[q] & 0xffff0000u) * up);
            memcpy(&x[q], &hh, 4);
          }
          *at = make_uint4(x[0], x[1], x[2], x[3]);
        }
        fence_proxy_async_shared();
        mbar_arrive(q_ready);
      }
    }
    // MOD 0 multiplies masked scores, -inf, by the factor as well: it must not
    // become 0 (below 2^-119 every score is as good as 0 anyway)
    auto at_least = [](float x) { return MOD == 0 ? fmaxf(x, 1.5e-36f) : x; };
    const uint64_t xs2 = f2(at_least(xs), at_least(xs));
    const float slope = MOD && p.slopes && row_valid ? ld_prior(p.slopes + h) * kLog2e : 0.f;
    // of scores in log2 units
    const float cap_in = MOD == 2 ? 2.f / p.softcap : MOD == 3 ? kLn2 / p.softcap : 0.f;
    const float cap_out = p.softcap * kLog2e;
    // groups of keys with an exponent offset of their own: V's scales, the slope's part of a group
    constexpr int NG = kCodes || MOD ? 4 : 1;

    float m_run = -INFINITY, l_run = 0.f;
    for (int jj = 0; jj < n_tiles && ok; ++jj) {
      const int j0 = (j_begin + jj) * BN;
      float goff[NG], gsum[NG];
      uint64_t gx2[NG];
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        goff[y] = MOD ? slope * (float)(j0 - pos + y * (BN / NG)) : 0.f;
        gx2[y] = xs2;
      }
      if constexpr (kCodes) ok = wait_all(mbar_wait(&sc_full[jj % SR], (jj / SR) & 1, abort_v, p.err));
      if (ok) ok = wait_all(mbar_wait(&s_full[t], jj & 1, abort_v, p.err));
      if (!ok) break;
      tc_fence_after();
      uint32_t sr[BN];
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 32) tmem_ld32p(s_addr + c0, sr + c0);
      tmem_wait_ld();
      if constexpr (kPSep) {
        tc_fence_before();
        mbar_arrive(&s_free[t]);
      }
      if constexpr (kCodes) {
#pragma unroll
        for (int y = 0; y < NG; ++y) {
          const float4 e = sSc[(jj % SR) * 4 + y];
          const float gx = at_least(xs * e.x);
          gx2[y] = f2(gx, gx);
          goff[y] += e.y;
          gsum[y] = e.z;
        }
      }
      const bool edge = !(j0 >= lo_i && j0 + BN <= hi_i);
      if constexpr (MOD == 2) {
        if (edge) {  // a masked NaN must not share a visible score's reciprocal
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (j0 + c < lo_i || j0 + c >= hi_i) sr[c] = 0;
        }
      }
      // slopes: (j - pos) slope = a group's first key's, in goff, + 0, slope, 2 slope ..
      // over the group, a running sum (32 steps: the fp32 rounding of the scores)
      uint64_t x2[BN / 2];
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        uint64_t ramp = f2(0.f, slope);
        const uint64_t two = f2(2.f * slope, 2.f * slope);
#pragma unroll
        for (int c = y * BN / 2 / NG; c < (y + 1) * BN / 2 / NG; ++c) {
          const uint64_t s2 = f2u(sr[2 * c], sr[2 * c + 1]);
          if constexpr (MOD == 0) x2[c] = s2;  // scaled in the exponent's fma (the scale is positive)
          if constexpr (MOD == 1) x2[c] = f2_fma(s2, gx2[y], ramp);
          if constexpr (MOD == 2) {
            x2[c] = f2_mul(s2, gx2[y]);
            if (c & 1) {
              cap4(x2[c - 1], x2[c], cap_in, cap_out);
              x2[c - 1] = f2_add(x2[c - 1], ramp);
              ramp = f2_add(ramp, two);
              x2[c] = f2_add(x2[c], ramp);
              ramp = f2_add(ramp, two);
            }
          }
          if constexpr (MOD == 3) {
            float v0, v1;
            f2_split(f2_mul(s2, gx2[y]), v0, v1);
            x2[c] = f2_add(f2(cap_any(v0, cap_out, cap_in), cap_any(v1, cap_out, cap_in)), ramp);
            ramp = f2_add(ramp, two);
          }
          if constexpr (MOD == 1) ramp = f2_add(ramp, two);
        }
      }
      if (edge) {
#pragma unroll
        for (int c = 0; c < BN; ++c)
          if (j0 + c < lo_i || j0 + c >= hi_i) {
            float lo, hi;
            f2_split(x2[c / 2], lo, hi);
            if (c & 1) hi = -INFINITY; else lo = -INFINITY;
            x2[c / 2] = f2(lo, hi);
          }
      }
      float mx = -INFINITY;
      if constexpr (MOD == 0) {
        const float none[1] = {0.f};
#pragma unroll
        for (int y = 0; y < NG; ++y) {
          float gx, unused;
          f2_split(gx2[y], gx, unused);
          mx = fmaxf(mx, fmaf(tile::row_max<1, BN / NG>(x2 + y * (BN / 2 / NG), none), gx, goff[y]));
        }
      } else {
        mx = tile::row_max<NG, BN / NG>(x2, goff);
      }
      const float m_new = fmaxf(m_run, mx);
      const bool need = m_new > m_run + kLag;
      float alpha = 1.f;
      if (need) {
        alpha = ex2_approx(m_run - m_new);
        l_run *= alpha;
        m_run = m_new;
      }
      const float m_use = m_run == -INFINITY ? 0.f : m_run - kOffset;
      uint32_t pk[BN / 2];
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        const float no = goff[y] - m_use;
        const uint64_t no2 = f2(no, no);
        uint64_t sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int c = y * BN / 2 / NG; c < (y + 1) * BN / 2 / NG; ++c) {
          const uint64_t e2 = MOD == 0 ? f2_fma(x2[c], gx2[y], no2) : f2_add(x2[c], no2);
          float lo, hi;
          f2_split(e2, lo, hi);
          lo = ex2_approx(lo);
          hi = ex2_approx(hi);
          sum[c & 1] = f2_add(sum[c & 1], f2(lo, hi));
          if constexpr (kCodes) {
            const __half2 hh = __floats2half2_rn(lo, hi);
            memcpy(&pk[c], &hh, 4);
          } else {
            pk[c] = pack_bf16x2(lo, hi);
          }
        }
        float a0, a1, b0, b1;
        f2_split(sum[0], a0, a1);
        f2_split(sum[1], b0, b1);
        const float total = (a0 + a1) + (b0 + b1);
        l_run = kCodes ? fmaf(total, gsum[y], l_run) : l_run + total;
      }
      if constexpr (kPSep) {
        if (jj > 0) {
          ok = wait_all(mbar_wait(&o_ready[t], (jj - 1) & 1, abort_v, p.err));
          if (!ok) break;
          tc_fence_after();
        }
      }
      if (jj > 0 && __any_sync(0xffffffffu, need)) tile::rescale_o<D>(o_addr, alpha);
      tile::store_p<BN>(p_addr, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[t]);
    }

    if (n_tiles > 0 && ok) {
      ok = wait_all(mbar_wait(kPSep ? &o_ready[t] : &o_done[t], kPSep ? (n_tiles - 1) & 1 : 0, abort_v, p.err));
      tc_fence_after();
    }
    const bool live = n_tiles > 0 && ok;
    const float m_off = m_run - kOffset;  // what P and the sum are relative to
    if (args.n_split == 1) {
      const long long tok = u.s.q0 + i;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + tok * p.ot + (long long)h * p.oh;
      if (live) {
        tile::store_o_row<D>(o_addr, l_run != 0.f ? 1.f / l_run : 0.f, orow, row_valid);
      } else if (row_valid && n_tiles == 0) {
#pragma unroll
        for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(orow + c) = make_uint4(0, 0, 0, 0);
      }
      if (row_valid && p.lse) p.lse[tok * p.Hq + h] = l_run != 0.f ? m_off * kLn2 + logf(l_run) : -INFINITY;
    } else {
      const long long part = (long long)unit * args.n_split + sidx;
      const int row = t * kRows + lr;
      const bool have = live && l_run != 0.f;
      if (live) {
        float4* wo = reinterpret_cast<float4*>(args.ws_o) + part * (D / 4) * 256 + row;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t r[32];
          tmem_ld32(o_addr + c0, r);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            wo[((c0 + c) / 4) * 256] = make_float4(__uint_as_float(r[c]), __uint_as_float(r[c + 1]),
                                                   __uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
        }
      }
      args.ws_ml[part * 256 + row] = make_float2(have ? m_off : -INFINITY, have ? l_run : 0.f);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) {
    if (lane == 0 && n_tiles > 0) {
      mma_commit(fin);
      mbar_wait(fin, 0, nullptr, p.err);
    }
    __syncwarp();
    tmem_dealloc(tbase, 512);
  }
}

// Adds the parts of a unit's rows, O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i:
// a block has 32 rows of a unit, a thread 16 columns of one.
constexpr int kMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) paged_tc_merge_kernel(const __grid_constant__ TcPagedArgs args) {
  const PagedParams& p = args.p;
  grid_dep_wait();
  grid_dep_launch();
  const int unit = blockIdx.x >> 3;
  TcUnit u;
  if (!find_unit<kMergeThreads>(args, unit, u)) return;
  for (int x = threadIdx.x; x < 32 * (D / 16); x += kMergeThreads) {
    const int row = (blockIdx.x & 7) * 32 + (x & 31), c0 = (x >> 5) * 4;  // first of 4 float4 columns
    const int t = row >> 7, lr = row & 127;
    const int tk = (int)fdiv((uint32_t)lr, args.fd_g), g = lr - tk * p.group;
    const int i = u.tok0 + t * args.tok + tk;
    if (tk >= args.tok || i >= u.s.n) continue;
    const long long part0 = (long long)unit * args.n_split;
    float2 ml[kMaxSplit];
    float top = -INFINITY, den = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxSplit; ++k) {
      ml[k] = k < args.n_split ? args.ws_ml[(part0 + k) * 256 + row] : make_float2(-INFINITY, 0.f);
      top = fmaxf(top, ml[k].x);
    }
    float4 acc[4] = {};
#pragma unroll
    for (int k = 0; k < kMaxSplit; ++k) {
      if (ml[k].y == 0.f) continue;  // a part without keys wrote nothing else
      const float w = ex2_approx(ml[k].x - top);
      den = fmaf(w, ml[k].y, den);
      const float4* src = reinterpret_cast<const float4*>(args.ws_o) + ((part0 + k) * (D / 4) + c0) * 256 + row;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 y = src[c * 256];
        acc[c].x = fmaf(w, y.x, acc[c].x); acc[c].y = fmaf(w, y.y, acc[c].y);
        acc[c].z = fmaf(w, y.z, acc[c].z); acc[c].w = fmaf(w, y.w, acc[c].w);
      }
    }
    const float inv = den != 0.f ? 1.f / den : 0.f;
    const long long tok = u.s.q0 + i;
    const int h = u.hk * p.group + g;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + tok * p.ot + (long long)h * p.oh + c0 * 4;
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
      uint4 y;
      y.x = pack_bf16x2(acc[c].x * inv, acc[c].y * inv);
      y.y = pack_bf16x2(acc[c].z * inv, acc[c].w * inv);
      y.z = pack_bf16x2(acc[c + 1].x * inv, acc[c + 1].y * inv);
      y.w = pack_bf16x2(acc[c + 1].z * inv, acc[c + 1].w * inv);
      *reinterpret_cast<uint4*>(dst + c * 4) = y;
    }
    if (c0 == 0 && p.lse) p.lse[tok * p.Hq + h] = den != 0.f ? top * kLn2 + logf(den) : -INFINITY;
  }
}

// ---------------------------------------------------------------- host side
int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// Units a call may have: every sequence with rows for this kernel ends in one
// unfilled block.  One at least where rows are given, however few max_q allows:
// the kernel reports the ranges that break it.
long long unit_bound(const PagedParams& p, int limit) {
  const long long tok2 = 2 * (kRows / p.group);
  const long long least = limit / p.group + 1;  // tokens of a sequence that is not the decode kernel's
  const long long seqs = p.s.total_q / least < p.s.B ? p.s.total_q / least : p.s.B;
  const long long per = p.s.max_q > 0 ? (p.s.max_q + tok2 - 1) / tok2 : 1;
  const long long a = p.s.total_q / tok2 + seqs, b = seqs * per;
  return (a < b ? a : b) * p.c.Hkv;
}

// Parts a unit's keys are cut into: the count that gives the least modelled
// time, waves of CTAs times (key tiles of a part + a fixed cost, and what
// writing and adding the parts costs), in key tiles.  The key range is the
// table's, the only bound the host has.
int split_of(const PagedParams& p, long long units) {
  const long long cap = (long long)p.s.max_pages * p.c.page_size;
  const long long reach = p.window > 0 && p.window + 256 < cap ? p.window + 256 : cap;
  const int nt = (int)((reach + BN - 1) / BN), nsm = num_sms();
  if (units >= nsm || nt < 4) return 1;
  int best = 1;
  double cost = (double)((units + nsm - 1) / nsm) * (nt + 3.0);
  for (int s = 2; s <= kMaxSplit && 2 * s <= nt; ++s) {
    const double c = (double)((units * s + nsm - 1) / nsm) * ((nt + s - 1) / s + 3.0) + 2.0 + 0.15 * s;
    if (c < cost) { cost = c; best = s; }
  }
  return best;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

bool q_map(CUtensorMap* m, const PagedParams& p, int tok) {
  cuuint64_t dims[3] = {(cuuint64_t)p.c.d, (cuuint64_t)p.Hq, (cuuint64_t)p.s.total_q};
  cuuint64_t strides[2] = {(cuuint64_t)p.qh * 2, (cuuint64_t)p.qt * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)tok};
  return encode_cached(m, p.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int KV, int D>
cudaError_t tc_one(const TcPagedArgs& a, int mod, long long units, cudaStream_t stream) {
  using L = TcLayout<KV, D>;
  auto kern = mod == 0   ? paged_tc_kernel<KV, D, 0>
              : mod == 1 ? paged_tc_kernel<KV, D, 1>
              : mod == 2 ? paged_tc_kernel<KV, D, 2>
                         : paged_tc_kernel<KV, D, 3>;
  static std::mutex mu;
  static uint64_t done[4];
  static cudaError_t bad[4];
  {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (!(done[mod] >> (dev & 63) & 1)) {
      bad[mod] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
      // setmaxnreg.inc takes from the registers the CTA was launched with:
      // launch only what was compiled to the count the split assumes
      cudaFuncAttributes fa;
      if (bad[mod] == cudaSuccess) bad[mod] = cudaFuncGetAttributes(&fa, kern);
      if (bad[mod] == cudaSuccess && fa.numRegs != kRegsLaunch<KV>) bad[mod] = cudaErrorInvalidConfiguration;
      if (bad[mod] == cudaSuccess) done[mod] |= 1ull << (dev & 63);
    }
    if (bad[mod] != cudaSuccess) return bad[mod];
  }
  cudaError_t e = launch_serialized(kern, dim3((unsigned)(units * a.n_split)), dim3(kThreadsOf<KV>), (size_t)L::kAlloc, stream, a);
  if (e != cudaSuccess || a.n_split == 1) return e;
  return launch_serialized(paged_tc_merge_kernel<D>, dim3((unsigned)(units * 8)), dim3(kMergeThreads), 0, stream, a);
}

}  // namespace

int paged_tc_check(const PagedParams& p, sdpa_dtype_t dtype) {
  const CacheView& c = p.c;
  if (dtype != SDPA_BF16 || c.dtype == SDPA_CACHE_F32 || c.d == 16) return SDPA_ERR_UNSUPPORTED;
  if (c.page_size % 16 != 0 || p.group > kRows) return SDPA_ERR_UNSUPPORTED;
  const long long es = c.dtype == SDPA_CACHE_BF16 ? 2 : 1;
  const long long bytes[] = {c.kp * es, c.kh * es, c.kt * es, c.vp * es, c.vh * es, c.vt * es, p.qt * 2, p.qh * 2,
                             p.ot * 2, p.oh * 2};
  for (long long x : bytes) {
    if (x % 16 != 0) return SDPA_ERR_MISALIGNED;
    if (x >= (1LL << 40)) return SDPA_ERR_UNSUPPORTED;
  }
  if ((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) | reinterpret_cast<uintptr_t>(p.q) |
       reinterpret_cast<uintptr_t>(p.out)) % 16 != 0)
    return SDPA_ERR_MISALIGNED;
  if (unit_bound(p, 0) * kMaxSplit * 8 > 0x7fffffffLL) return SDPA_ERR_UNSUPPORTED;
  return SDPA_OK;
}

size_t paged_tc_workspace(const PagedParams& p, int limit) {
  const long long units = unit_bound(p, limit);
  const int sp = split_of(p, units);
  if (sp == 1) return 0;
  const size_t parts = (size_t)units * sp;
  return up256(parts * 256 * p.c.d * 4) + up256(parts * 256 * 8);
}

cudaError_t launch_paged_tc(const PagedParams& p, int limit, void* ws, cudaStream_t stream) {
  TcPagedArgs a;
  memset(&a, 0, sizeof(a));
  a.p = p;
  a.tok = kRows / p.group;
  a.limit = limit;
  const long long units = unit_bound(p, limit);
  if (units == 0) return cudaSuccess;
  a.n_split = split_of(p, units);
  a.fd_split = make_fastdiv((uint32_t)a.n_split);
  a.fd_hkv = make_fastdiv((uint32_t)p.c.Hkv);
  a.fd_g = make_fastdiv((uint32_t)p.group);
  const CacheView& c = p.c;
  const bool codes = c.dtype != SDPA_CACHE_BF16;
  const CUtensorMapDataType ty = codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t es = codes ? 1 : 2;
  a.box_rows = gcd(c.page_size, codes ? kHalf : BN);
  const uint32_t bw = codes ? c.d : 64;
  bool ok = q_map(&a.tq, p, a.tok);
  ok = ok && make_tmap_4d(&a.tk, c.k, ty, c.d, c.page_size, c.Hkv, c.num_pages, c.kt * es, c.kh * es, c.kp * es, bw,
                          a.box_rows, codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
  ok = ok && make_tmap_4d(&a.tv, c.v, ty, c.d, c.page_size, c.Hkv, c.num_pages, c.vt * es, c.vh * es, c.vp * es, bw,
                          a.box_rows, codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  if (a.n_split > 1) {
    const size_t parts = (size_t)units * a.n_split;
    a.ws_o = static_cast<float*>(ws);
    a.ws_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + up256(parts * 256 * c.d * 4));
  }
  const int mod = p.softcap > kPlainCap ? 3 : p.softcap > 0.f ? 2 : p.slopes != nullptr || !(p.scale > 0.f) ? 1 : 0;
  const bool wide = c.d == 128;
  switch (c.dtype) {
    case SDPA_CACHE_BF16: return wide ? tc_one<KV_BF16, 128>(a, mod, units, stream) : tc_one<KV_BF16, 64>(a, mod, units, stream);
    case SDPA_CACHE_E4M3: return wide ? tc_one<KV_E4M3, 128>(a, mod, units, stream) : tc_one<KV_E4M3, 64>(a, mod, units, stream);
    case SDPA_CACHE_INT8: return wide ? tc_one<KV_INT8, 128>(a, mod, units, stream) : tc_one<KV_INT8, 64>(a, mod, units, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
