// Attention over a paged cache on the CUDA cores: every type, head_dim, page
// size, stride and option, fp32 arithmetic throughout.
//
//   x_j = scale q.k_j,  x_j <- c tanh(x_j / c) (softcap c),  x_j += slope_h (j - pos)
//   out = sum_j 2^(x_j log2e - m) v_j / sum_j 2^(x_j log2e - m)     over the keys seen
//
// One block owns one (query row, head).  A key row is held by G = row bytes /
// 16 neighbouring lanes, 16 bytes each, for K and V alike: a dot product is a
// partial product and log2 G shuffles, the value sum needs none.  Each lane
// group keeps its own online softmax (running max, sum, accumulator) over the
// keys it takes, kAhead of them loaded together; groups and warps are merged
// once at the end.  Latency-bound on short caches (one round trip per kAhead
// keys of a group), else bound by re-reading K and V for every query row: this
// is the fp32 path and the path of layouts the others do not take.
#include <cooperative_groups.h>
#include <math.h>

#include "paged.cuh"
#include "pdl_launch.cuh"

namespace sdpa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kWarps = 8;
constexpr int kAhead = 4;  // keys of a lane group in flight

// kSplit: CTAs of a cluster that share a row's keys; the first adds their sums
// through distributed shared memory.
template <typename T, typename C, int D, int kSplit>
__global__ void __launch_bounds__(kWarps * 32) paged_exact_kernel(const __grid_constant__ PagedParams p, int vec) {
  constexpr int E = 16 / sizeof(C);
  constexpr int G = D / E;  // lanes of a key row
  constexpr int KW = 32 / G;  // key rows of a warp side by side
  __shared__ float s_acc[kWarps][D];
  __shared__ float s_m[kWarps], s_l[kWarps];
  __shared__ float s_num[D], s_top, s_den;
  __shared__ int s_b;
  sm100::grid_dep_launch();
  sm100::grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / kSplit, rank = blockIdx.x % kSplit, h = blockIdx.y;
  int b = t;
  if (p.s.cu_q != nullptr) {
    if (threadIdx.x == 0) {
      int lo = 0, hi = p.s.B;  // largest b with cu[b] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (ld_prior(p.s.cu_q + mid) <= t) lo = mid; else hi = mid;
      }
      s_b = lo;
    }
    __syncthreads();
    b = s_b;
  }
  const Seq q = seq_of(p.s, p.c, b, p.err);
  if (t < q.q0 || t >= q.q0 + q.n) return;  // a row behind the last sequence: left as it is
  if (q.n <= p.skip_rows / p.group) return;
  const int pos = q.L - q.n + (t - q.q0);
  int lo, hi;
  seen(p, pos, lo, hi);

  const int hk = h / p.group;
  const int e0 = (lane % G) * E;
  float qv[E];
  const T* qrow = static_cast<const T*>(p.q) + t * p.qt + h * p.qh + e0;
#pragma unroll
  for (int i = 0; i < E; ++i) qv[i] = to_f32(qrow[i]);
  const C* kb = static_cast<const C*>(p.c.k) + hk * p.c.kh + e0;
  const C* vb = static_cast<const C*>(p.c.v) + hk * p.c.vh + e0;
  const float slope = p.slopes ? ld_prior(p.slopes + h) : 0.f;

  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = 0.f;
  constexpr int kStride = kSplit * kWarps * KW * kAhead;
  const int first = lo + (rank * kWarps + warp) * KW * kAhead;
  int entry[kAhead];  // of the next keys, on their way while the last are worked on
  auto fetch = [&](int j0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u * KW + lane / G;
      entry[u] = j < hi ? page_entry(p.s, p.c, b, j) : 0;
    }
  };
  fetch(first);
  for (int j0 = first; j0 < hi; j0 += kStride) {
    alignas(16) C kr[kAhead][E], vr[kAhead][E];
    float x[kAhead], vscale[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u * KW + lane / G;
      x[u] = -INFINITY;
      vscale[u] = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) kr[u][i] = vr[u][i] = C();
      if (j < hi) {
        const long long page = max(0, good_page(p.c, entry[u], p.err));
        const int off = j - (int)fdiv((uint32_t)j, p.c.fd_page) * p.c.page_size;
        const C* kp = kb + page * p.c.kp + off * p.c.kt;
        const C* vp = vb + page * p.c.vp + off * p.c.vt;
        if (vec) {
          *reinterpret_cast<uint4*>(kr[u]) = *reinterpret_cast<const uint4*>(kp);
          *reinterpret_cast<uint4*>(vr[u]) = *reinterpret_cast<const uint4*>(vp);
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) { kr[u][i] = kp[i]; vr[u][i] = vp[i]; }
        }
        x[u] = p.scale;
        vscale[u] = 1.f;
        if constexpr (is_code<C>::value) {
          x[u] *= p.c.ks[page * p.c.ksp + hk * p.c.ksh + off * p.c.kst];
          vscale[u] = p.c.vs[page * p.c.vsp + hk * p.c.vsh + off * p.c.vst];
        }
      }
    }
    fetch(j0 + kStride);
    float top = m;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u * KW + lane / G;
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) dot = fmaf(qv[i], cache_elem(kr[u][i]), dot);
#pragma unroll
      for (int o = 1; o < G; o *= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (j < hi) {
        float y = dot * x[u];
        if (p.softcap > 0.f) y = p.softcap * tanhf(y / p.softcap);
        x[u] = fmaf(slope, (float)(j - pos), y) * kLog2e;
      }
      top = fmaxf(top, x[u]);
    }
    // the maxima pass over NaN scores, the weights and their sum do not
    const float from = top == -INFINITY ? 0.f : top;
    const float a = exp2f(m - from);
    l *= a;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] *= a;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const float w = exp2f(x[u] - from);
      l += w;
      const float wv = w * vscale[u];
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] = fmaf(wv, cache_elem(vr[u][i]), acc[i]);
    }
    m = top;
  }
  // lane groups of the warp, then the warps
#pragma unroll
  for (int o = G; o < 32; o *= 2) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    const float top = fmaxf(m, m2);
    const float a = top == -INFINITY ? 0.f : exp2f(m - top), a2 = top == -INFINITY ? 0.f : exp2f(m2 - top);
    l = l * a + l2 * a2;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * a + __shfl_xor_sync(0xffffffffu, acc[i], o) * a2;
    m = top;
  }
  if (lane < G) {
#pragma unroll
    for (int i = 0; i < E; ++i) s_acc[warp][e0 + i] = acc[i];
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
  __syncthreads();
  auto finish = [&](float top, float num, float den) {  // column threadIdx.x of the row
    static_cast<T*>(p.out)[t * p.ot + h * p.oh + threadIdx.x] = from_f32<T>(den != 0.f ? num / den : 0.f);
    if (p.lse != nullptr && threadIdx.x == 0)
      p.lse[(long long)t * p.Hq + h] = den != 0.f ? top * kLn2 + logf(den) : -INFINITY;
  };
  if (threadIdx.x < D) {
    float top = -INFINITY, den = 0.f, num = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    for (int w = 0; w < kWarps; ++w) {
      const float a = top == -INFINITY ? 0.f : exp2f(s_m[w] - top);
      den = fmaf(a, s_l[w], den);
      num = fmaf(a, s_acc[w][threadIdx.x], num);
    }
    if constexpr (kSplit > 1) {
      s_num[threadIdx.x] = num;
      if (threadIdx.x == 0) { s_top = top; s_den = den; }
    } else {
      finish(top, num, den);
    }
  }
  if constexpr (kSplit > 1) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (rank == 0 && threadIdx.x < D) {
      float tops[kSplit], top = -INFINITY, den = 0.f, num = 0.f;
#pragma unroll
      for (int r = 0; r < kSplit; ++r) {
        tops[r] = *cluster.map_shared_rank(&s_top, r);
        top = fmaxf(top, tops[r]);
      }
#pragma unroll
      for (int r = 0; r < kSplit; ++r) {
        const float a = top == -INFINITY ? 0.f : exp2f(tops[r] - top);
        den = fmaf(a, *cluster.map_shared_rank(&s_den, r), den);
        num = fmaf(a, cluster.map_shared_rank(s_num, r)[threadIdx.x], num);
      }
      finish(top, num, den);
    }
    cluster.sync();  // the others' shared memory stays until it has been read
  }
}

template <typename T, typename C, int D>
cudaError_t exact_one(const PagedParams& p, cudaStream_t stream) {
  const CacheView& c = p.c;
  const long long es = sizeof(C);
  const bool vec = (reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) | (c.kp * es) | (c.kh * es) |
                    (c.kt * es) | (c.vp * es) | (c.vh * es) | (c.vt * es)) % 16 == 0;
  // Fewer rows than SMs: four CTAs, a cluster, share a row's keys (48 rows of
  // 1024 keys, f32: 12.5 us against 20.6, graph replay).
  if ((long long)p.s.total_q * p.Hq <= num_sms()) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.s.total_q * 4, (unsigned)p.Hq);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 4;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, paged_exact_kernel<T, C, D, 4>, p, (int)vec);
  }
  return launch_serialized(paged_exact_kernel<T, C, D, 1>, dim3((unsigned)p.s.total_q, (unsigned)p.Hq),
                           dim3(kWarps * 32), 0, stream, p, (int)vec);
}
template <typename T, typename C>
cudaError_t exact_d(const PagedParams& p, cudaStream_t stream) {
  switch (p.c.d) {
    case 16: return exact_one<T, C, 16>(p, stream);
    case 64: return exact_one<T, C, 64>(p, stream);
    case 128: return exact_one<T, C, 128>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_exact(const PagedParams& p, sdpa_dtype_t dtype, cudaStream_t stream) {
  const bool f = dtype == SDPA_F32;
  switch (p.c.dtype) {
    case SDPA_CACHE_F32: return exact_d<float, float>(p, stream);
    case SDPA_CACHE_BF16: return exact_d<__nv_bfloat16, __nv_bfloat16>(p, stream);
    case SDPA_CACHE_E4M3: return f ? exact_d<float, __nv_fp8_e4m3>(p, stream) : exact_d<__nv_bfloat16, __nv_fp8_e4m3>(p, stream);
    case SDPA_CACHE_INT8: return f ? exact_d<float, int8_t>(p, stream) : exact_d<__nv_bfloat16, int8_t>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
