// Attention of chunks of new tokens over a paged cache on the tensor cores:
// TMA + tcgen05/TMEM, online softmax, for sequences whose (token, head) rows
// per kv head are too many for the decode kernel.
//
// A unit is 256 rows of one (sequence, kv head), two tiles of 128: row r of a
// tile is token r / G, query head r % G of the G heads that share the kv head,
// so a tile is full whatever G is, K and V are read once for all G heads, and
// the causal diagonal costs 128 / G tokens.  Q comes as one TMA box
// (64 columns, G heads, 128 / G tokens) per panel.  Roles, 384 threads:
//   warps 0-3, 4-7  softmax of tile A, B (thread = row = TMEM lane)
//   warp  8         producer: K / V pages by TMA, one box per run of tokens
//                   inside a page, page numbers a tile ahead
//   warp  9         TMEM owner, MMA issuer
//   warps 10-11     codes: the converters
// The tile pipeline (S_t = Q_t.K^T, softmax, O_t += P_t.V, stale-max rescale)
// is that of the dense kernel, flash_tc.cu: at head_dim 128 P_t overwrites S_t,
// at 64 it has its own columns and S_t runs a tile ahead.
//
// 8-bit caches: raw pages land in a ring of 64-key pieces; the converters turn
// codes into f16 (exactly) in the K / V stages, in the 128-byte swizzle the
// MMA reads, and put ks, log2 vs and 1 / vs of the tile's keys beside them.
// The softmax warps scale their Q row in place by a power of two into f16 (its
// largest element to [2^14, 2^15)).  Scores are acc * ks_j; V's scale goes into
// the exponent, t_j = x_j log2e + log2 vs_j, p_j = 2^(t_j - m), and out is
// sum p_j code_j / sum p_j (1 / vs_j), as in the decode kernel.
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

constexpr int kThreads = 384;
constexpr int kRows = 128;           // of a tile
constexpr int BN = 128;              // keys of a tile
constexpr int kHalf = 64;            // keys of a raw piece
constexpr int kConv = 64;            // converter threads
constexpr int kMaxSplit = 16;
constexpr int kRegsLaunch = 168;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
  static constexpr int NR = D == 64 ? 4 : 3;        // raw pieces
  static constexpr int SR = D == 64 ? 8 : 4;        // tiles of scales kept: see the softmax loop
  static constexpr int kPanels = D / 64;
  static constexpr int kQBytes = kPanels * kRows * 128;
  static constexpr int kKVBytes = kPanels * BN * 128;
  static constexpr int kRaw = kCodes ? kHalf * D : 0;
  static constexpr int oQ = 0;
  static constexpr int oK = oQ + 2 * kQBytes;
  static constexpr int oV = oK + NS * kKVBytes;
  static constexpr int oRaw = oV + NS * kKVBytes;
  static constexpr int oSc = oRaw + NR * kRaw;       // [SR][3][BN] floats
  static constexpr int oBar = oSc + (kCodes ? SR * 3 * BN * 4 : 0);
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
  if (s.n * a.p.group <= a.limit) return 0;
  return (s.n + 2 * a.tok - 1) / (2 * a.tok);
}

// Unit `unit` of the launch, blocks numbered from the last one down; false past
// the last.  The whole CTA takes part.
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

template <int KV, int D, bool MOD>
__global__ void __launch_bounds__(kThreads, 1) paged_tc_kernel(const __grid_constant__ TcPagedArgs args) {
  using L = TcLayout<KV, D>;
  constexpr bool kCodes = L::kCodes;
  constexpr bool kPSep = D == 64;
  constexpr int NS = L::NS, NR = L::NR, SR = L::SR;
  constexpr float kLag = kCodes ? 3.f : 8.f, kOffset = kCodes ? 12.f : 0.f;
  constexpr int kRegsSoftmax = 216, kRegsOther = 72;
  static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * kRegsLaunch, "register split");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem + L::oQ;
  uint8_t* sK = smem + L::oK;
  uint8_t* sV = smem + L::oV;
  uint8_t* sRaw = smem + L::oRaw;
  float* sSc = reinterpret_cast<float*>(smem + L::oSc);
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
  if (!find_unit(args, unit, u)) return;
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
        mbar_init(&k_full[i], kConv);
        mbar_init(&v_full[i], kConv);
      }
      for (int i = 0; i < NR; ++i) mbar_init(&raw_empty[i], kConv);
      for (int i = 0; i < SR; ++i) mbar_init(&sc_full[i], kConv);
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
        int pg[2], pv[2] = {0, 0};
        for (int x = 0; x < 2; ++x) pg[x] = page_at(box_key(j_begin * BN + x * kHalf));
        for (int jj = 0; jj <= n_tiles && ok; ++jj) {
          const int key0 = (j_begin + jj) * BN;
          int nx[2] = {0, 0};
          if (jj + 1 < n_tiles)
            for (int x = 0; x < 2; ++x) nx[x] = page_at(box_key(key0 + BN + x * kHalf));
          if (jj < n_tiles)
            for (int x = 0; x < 2 && ok; ++x) load(false, key0 + x * kHalf, pg[x]);
          if (jj > 0)
            for (int x = 0; x < 2 && ok; ++x) load(true, key0 - BN + x * kHalf, pv[x]);
          for (int x = 0; x < 2; ++x) { pv[x] = pg[x]; pg[x] = nx[x]; }
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
    } else if (kCodes && warp >= 10 && n_tiles > 0) {
      // ------------------------------------------------------------ converters
      const int ct = tid - 320;  // 0 .. 63
      bool ok = true;
      int r_next = 0;
      // scales of this thread's two keys of a tile: page numbers fetched two
      // tiles ahead, scales one, so neither load is waited for
      float ks_n[2], vs_n[2];
      int pg_n[2];
      auto seen_key = [&](int jj, int x) {
        const int key = (j_begin + jj) * BN + x * kHalf + ct;
        return jj < n_tiles && key >= klo && key < khi ? key : -1;
      };
      auto fetch_pages = [&](int jj) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int key = seen_key(jj, x);
          pg_n[x] = key >= 0 ? page_of(p.s, p.c, u.b, key, p.err) : 0;
        }
      };
      auto fetch_scales = [&](int jj) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int key = seen_key(jj, x);
          ks_n[x] = vs_n[x] = 1.f;
          if (key >= 0) {
            const long long pg = pg_n[x];
            const int off = key - (int)fdiv((uint32_t)key, p.c.fd_page) * p.c.page_size;
            ks_n[x] = __ldg(p.c.ks + pg * p.c.ksp + u.hk * p.c.ksh + off * p.c.kst);
            vs_n[x] = __ldg(p.c.vs + pg * p.c.vsp + u.hk * p.c.vsh + off * p.c.vst);
          }
        }
      };
      auto convert = [&](bool is_v, int jj) {
        const int s = jj % NS, use = jj / NS;
        if (use > 0) ok = wait_all(mbar_wait(is_v ? &v_empty[s] : &k_empty[s], (use - 1) & 1, abort_v, p.err));
        uint8_t* dst = (is_v ? sV : sK) + s * L::kKVBytes;
        for (int x = 0; x < 2 && ok; ++x) {
          const int rs = r_next % NR;
          ok = wait_all(mbar_wait(&raw_full[rs], (r_next / NR) & 1, abort_v, p.err));
          if (!ok) break;
          constexpr int kPieces = D / 16;  // 16 codes each
          constexpr int kPass = kConv / kPieces;
          const int pc = ct % kPieces, r0 = ct / kPieces;
          const uint8_t* src = sRaw + rs * L::kRaw + r0 * D + pc * 16;
          const int key0 = (j_begin + jj) * BN + x * kHalf + r0;
          const bool all = key0 - r0 >= klo && key0 - r0 + kHalf <= khi;
          // codes 16 pc ..: panel pc / 4, 16-byte chunks 2 (pc % 4) and the next, at chunk ^ (row % 8)
          uint8_t* line = dst + (pc >> 2) * BN * 128 + (x * kHalf + r0) * 128;
          const int c0 = 2 * (pc & 3), sw = r0 & 7;
          static_assert(kPass % 8 == 0, "a thread's rows have one swizzle");
          constexpr int kBatch = 4;  // pieces loaded together
#pragma unroll
          for (int i0 = 0; i0 < kHalf / kPass; i0 += kBatch) {
            uint4 w[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              w[i] = *reinterpret_cast<const uint4*>(src + (i0 + i) * kPass * D);
              const int key = key0 + (i0 + i) * kPass;
              if (!all && (key < klo || key >= khi)) w[i] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int row = (i0 + i) * kPass;  // past r0
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
              *reinterpret_cast<uint4*>(line + row * 128 + ((c0 ^ sw) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(line + row * 128 + (((c0 + 1) ^ sw) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
          }
          mbar_arrive(&raw_empty[rs]);
          ++r_next;
        }
        if (!ok) return;
        fence_proxy_async_shared();
        mbar_arrive(is_v ? &v_full[s] : &k_full[s]);
      };
      fetch_pages(0);
      fetch_scales(0);
      fetch_pages(1);
      for (int jj = 0; jj <= n_tiles && ok; ++jj) {
        if (jj < n_tiles) {
          float* sc = sSc + (jj % SR) * 3 * BN;
          // The tile that used this slot, jj - SR, is behind every softmax
          // warp: K stage jj % NS being free means S(jj - NS) is complete, and
          // that S is only issued once tile jj - NS - 1's scores (head_dim 64)
          // or P (128) were taken from tensor memory: tiles up to jj - NS - 2
          // (64) or jj - NS - 1 (128) are finished, and SR >= NS + 2.
          if (jj >= NS) ok = wait_all(mbar_wait(&k_empty[jj % NS], (jj / NS - 1) & 1, abort_v, p.err));
          if (!ok) break;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float lg;
            asm("lg2.approx.f32 %0, %1;" : "=f"(lg) : "f"(vs_n[x]));
            sc[x * kHalf + ct] = ks_n[x];
            sc[BN + x * kHalf + ct] = lg;
            sc[2 * BN + x * kHalf + ct] = rcp_approx(vs_n[x]);
          }
          mbar_arrive(&sc_full[jj % SR]);
          fetch_scales(jj + 1);
          fetch_pages(jj + 2);
          convert(false, jj);
        }
        if (ok && jj > 0) convert(true, jj - 1);
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
    const uint64_t xs2 = f2(xs, xs);
    const float slope = MOD && p.slopes && row_valid ? __ldg(p.slopes + h) * kLog2e : 0.f;
    const float cap_in = MOD && p.softcap > 0.f ? 2.f / p.softcap : 0.f;  // of scores in log2 units
    const float cap_out = p.softcap * kLog2e;
    const float goff[1] = {0.f};

    float m_run = -INFINITY, l_run = 0.f;
    for (int jj = 0; jj < n_tiles && ok; ++jj) {
      const int j0 = (j_begin + jj) * BN;
      const float* sc = sSc + (jj % SR) * 3 * BN;
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
      uint64_t x2[BN / 2];
      if constexpr (kCodes) {
#pragma unroll
        for (int c = 0; c < BN; c += 4) {
          const float4 k4 = *reinterpret_cast<const float4*>(sc + c);
          const float4 v4 = *reinterpret_cast<const float4*>(sc + BN + c);
          const uint64_t a = f2_mul(f2u(sr[c], sr[c + 1]), f2(k4.x, k4.y));
          const uint64_t b = f2_mul(f2u(sr[c + 2], sr[c + 3]), f2(k4.z, k4.w));
          if constexpr (MOD) {
            x2[c / 2] = f2_mul(a, xs2);
            x2[c / 2 + 1] = f2_mul(b, xs2);
          } else {
            x2[c / 2] = f2_fma(a, xs2, f2(v4.x, v4.y));
            x2[c / 2 + 1] = f2_fma(b, xs2, f2(v4.z, v4.w));
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < BN / 2; ++c) x2[c] = f2_mul(f2u(sr[2 * c], sr[2 * c + 1]), xs2);
      }
      if constexpr (MOD) {
        if (p.softcap > 0.f) {  // c tanh(x / c) = c - 2 c / (1 + e^(2 x / c))
#pragma unroll
          for (int c = 0; c < BN / 2; ++c) {
            float lo, hi;
            f2_split(x2[c], lo, hi);
            lo = fmaf(-2.f * cap_out, rcp_approx(1.f + ex2_approx(lo * cap_in)), cap_out);
            hi = fmaf(-2.f * cap_out, rcp_approx(1.f + ex2_approx(hi * cap_in)), cap_out);
            x2[c] = f2(lo, hi);
          }
        }
        const float d0 = (float)(j0 - pos);
        const uint64_t sl2 = f2(slope, slope);
#pragma unroll
        for (int c = 0; c < BN / 2; ++c) x2[c] = f2_fma(f2(d0 + (float)(2 * c), d0 + (float)(2 * c + 1)), sl2, x2[c]);
        if constexpr (kCodes) {
#pragma unroll
          for (int c = 0; c < BN; c += 4) {
            const float4 v4 = *reinterpret_cast<const float4*>(sc + BN + c);
            x2[c / 2] = f2_add(x2[c / 2], f2(v4.x, v4.y));
            x2[c / 2 + 1] = f2_add(x2[c / 2 + 1], f2(v4.z, v4.w));
          }
        }
      }
      if (!(j0 >= lo_i && j0 + BN <= hi_i)) {
#pragma unroll
        for (int c = 0; c < BN; ++c)
          if (j0 + c < lo_i || j0 + c >= hi_i) {
            float lo, hi;
            f2_split(x2[c / 2], lo, hi);
            if (c & 1) hi = -INFINITY; else lo = -INFINITY;
            x2[c / 2] = f2(lo, hi);
          }
      }
      const float mx = tile::row_max<1, BN>(x2, goff);
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
      if constexpr (kCodes) {
        const uint64_t nm = f2(-m_use, -m_use);
        uint64_t sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < BN; c += 4) {
          const float4 i4 = *reinterpret_cast<const float4*>(sc + 2 * BN + c);
          float w[4];
          f2_split(f2_add(x2[c / 2], nm), w[0], w[1]);
          f2_split(f2_add(x2[c / 2 + 1], nm), w[2], w[3]);
#pragma unroll
          for (int q = 0; q < 4; ++q) w[q] = ex2_approx(w[q]);
          sum[0] = f2_fma(f2(w[0], w[1]), f2(i4.x, i4.y), sum[0]);
          sum[1] = f2_fma(f2(w[2], w[3]), f2(i4.z, i4.w), sum[1]);
          const __half2 h0 = __floats2half2_rn(w[0], w[1]), h1 = __floats2half2_rn(w[2], w[3]);
          memcpy(&pk[c / 2], &h0, 4);
          memcpy(&pk[c / 2 + 1], &h1, 4);
        }
        float a0, a1, b0, b1;
        f2_split(sum[0], a0, a1);
        f2_split(sum[1], b0, b1);
        l_run += (a0 + a1) + (b0 + b1);
      } else {
        l_run += tile::exp_pack<BN, BN>(x2, goff, m_use, pk);
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
        tile::store_o_row<D>(o_addr, l_run > 0.f ? 1.f / l_run : 0.f, orow, row_valid);
      } else if (row_valid && n_tiles == 0) {
#pragma unroll
        for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(orow + c) = make_uint4(0, 0, 0, 0);
      }
      if (row_valid && p.lse) p.lse[tok * p.Hq + h] = l_run > 0.f ? m_off * kLn2 + logf(l_run) : -INFINITY;
    } else {
      const long long part = (long long)unit * args.n_split + sidx;
      const int row = t * kRows + lr;
      const bool have = live && l_run > 0.f;
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
template <int D>
__global__ void __launch_bounds__(kThreads) paged_tc_merge_kernel(const __grid_constant__ TcPagedArgs args) {
  const PagedParams& p = args.p;
  grid_dep_wait();
  grid_dep_launch();
  const int unit = blockIdx.x >> 3;
  TcUnit u;
  if (!find_unit(args, unit, u)) return;
  for (int x = threadIdx.x; x < 32 * (D / 16); x += kThreads) {
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
      if (ml[k].x == -INFINITY) continue;  // a part without keys wrote nothing else
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
    const float inv = den > 0.f ? 1.f / den : 0.f;
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
    if (c0 == 0 && p.lse) p.lse[tok * p.Hq + h] = den > 0.f ? top * kLn2 + logf(den) : -INFINITY;
  }
}

// ---------------------------------------------------------------- host side
int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// Units a call may have: every sequence with rows for this kernel ends in one
// unfilled block.
long long unit_bound(const PagedParams& p, int limit) {
  const long long tok2 = 2 * (kRows / p.group);
  const long long least = limit / p.group + 1;  // tokens of a sequence that is not the decode kernel's
  const long long seqs = p.s.total_q / least < p.s.B ? p.s.total_q / least : p.s.B;
  const long long per = (p.s.max_q + tok2 - 1) / tok2;
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
cudaError_t tc_one(const TcPagedArgs& a, bool mod, long long units, cudaStream_t stream) {
  using L = TcLayout<KV, D>;
  auto kern = mod ? paged_tc_kernel<KV, D, true> : paged_tc_kernel<KV, D, false>;
  static std::mutex mu;
  static uint64_t done[2];
  static cudaError_t bad[2];
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
      if (bad[mod] == cudaSuccess && fa.numRegs != kRegsLaunch) bad[mod] = cudaErrorInvalidConfiguration;
      if (bad[mod] == cudaSuccess) done[mod] |= 1ull << (dev & 63);
    }
    if (bad[mod] != cudaSuccess) return bad[mod];
  }
  cudaError_t e = launch_serialized(kern, dim3((unsigned)(units * a.n_split)), dim3(kThreads), (size_t)L::kAlloc, stream, a);
  if (e != cudaSuccess || a.n_split == 1) return e;
  return launch_serialized(paged_tc_merge_kernel<D>, dim3((unsigned)(units * 8)), dim3(kThreads), 0, stream, a);
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
  const bool mod = p.softcap > 0.f || p.slopes != nullptr;
  const bool wide = c.d == 128;
  switch (c.dtype) {
    case SDPA_CACHE_BF16: return wide ? tc_one<KV_BF16, 128>(a, mod, units, stream) : tc_one<KV_BF16, 64>(a, mod, units, stream);
    case SDPA_CACHE_E4M3: return wide ? tc_one<KV_E4M3, 128>(a, mod, units, stream) : tc_one<KV_E4M3, 64>(a, mod, units, stream);
    case SDPA_CACHE_INT8: return wide ? tc_one<KV_INT8, 128>(a, mod, units, stream) : tc_one<KV_INT8, 64>(a, mod, units, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
