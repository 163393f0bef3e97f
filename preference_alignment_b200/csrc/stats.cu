// Token statistics: log-prob of a given token, entropy and the largest logits of each
// position, from one pass over the vocabulary that never stores the logits.
//   k_tc_gemm<EpiStats<K>>  z = Hp . W^T on tcgen05; the epilogue keeps, per position and
//                    vocabulary tile, the running maximum m, S = sum e^(z-m),
//                    T = sum e^(z-m) (z-m), the target logit and the tile's K largest logits
//   k_stats_f32<K>   the same partials on the fp32 SIMT route
//   k_stats_finish<K>  one warp per position: joins the tiles
//
// Entropy: -sum p log p = log S - T / S. Both terms are >= 0 (T <= 0), so the sum does not
// cancel, and T rescales with the maximum like S does: moving from m to m' multiplies both
// by f = e^(m-m') after T has taken S (m - m').
#include <cmath>

#include "internal.h"
#include "gemm_launch.cuh"

namespace dpo {

constexpr float kLog2eS = 1.4426950408889634f;
constexpr float kLn2S = 0.6931471805599453f;
// Logits at or below this count as -inf: they add nothing and are no alternative.
constexpr float kFloor = -1e30f;

// Order-preserving map of floats to unsigned integers; 0 is below every float's image.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);           // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  if (o == 0) return -INFINITY;
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// x[j] with j known only at run time: five rounds of selects, so x stays in registers.
__device__ __forceinline__ float pick32(const float (&x)[32], int j) {
  float a[16], b[8], c[4], d[2];
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = (j & 16) ? x[i + 16] : x[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = (j & 8) ? a[i + 8] : a[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = (j & 4) ? b[i + 4] : b[i];
#pragma unroll
  for (int i = 0; i < 2; ++i) d[i] = (j & 2) ? c[i + 2] : c[i];
  return (j & 1) ? d[1] : d[0];
}

// Per-tile lists of the K largest logits: a list is worth writing only if it can still
// matter. Each position has a threshold in global memory, the largest K-th value any of its
// finished tiles has published (atomicMax; the maximum does not depend on the order), a lower
// bound of the position's K-th largest logit. A tile takes a logit only if it reaches the
// threshold, and the finish reads a tile's list only if the tile's maximum reaches the final
// threshold: such a tile did write it, because the threshold it saw was no higher.
template <int K>
struct EpiStats {
  static constexpr bool kStaging = false;
  static constexpr bool kSystemFence = false;
  struct Params {
    const int* y;        // given token of each position, or nullptr
    float2* part;        // [S, ldp] (m, S)
    float* tsum;         // [S, ldp] T
    float* zy;           // [ldp] target logit
    uint32_t* tau;       // [ldp] thresholds, zeroed before the launch
    float2* list;        // [S, K, ldp] (logit, id), falling, fillers (<= kFloor, -)
    int n, V, ldp;
  };
  static constexpr int kList = K > 0 ? K : 1;
  int tok, nt, yl, vlim;
  bool valid;
  float mx, ref, s, t, zyv, tauv;
  float val[kList];
  int id[kList];

  __device__ __forceinline__ void begin(const Params& p, int m_row, int nt_, int, const EpiCtx&) {
    nt = nt_;
    tok = m_row;
    valid = tok < p.n;
    const int vbase = nt * kBN;
    vlim = p.V - vbase;
    yl = valid && p.y != nullptr ? __ldg(p.y + tok) : -1;
    yl = yl >= 0 ? yl - vbase : -1;
    mx = kFloor;
    ref = kFloor * kLog2eS;
    s = 0.f;
    t = 0.f;
    zyv = 0.f;
    if (K > 0) {
      tauv = valid ? from_ordered(__ldcg(p.tau + tok)) : INFINITY;   // padding rows take nothing
#pragma unroll
      for (int j = 0; j < kList; ++j) {
        val[j] = kFloor;
        id[j] = 0;
      }
    }
  }

  // Sorted insert; among equal logits the earlier column stays in front.
  __device__ __forceinline__ void insert(float x, int col) {
#pragma unroll
    for (int j = kList - 1; j > 0; --j) {
      const bool here = x > val[j], above = x > val[j - 1];
      id[j] = above ? id[j - 1] : (here ? col : id[j]);
      val[j] = above ? val[j - 1] : (here ? x : val[j]);
    }
    if (x > val[0]) {
      val[0] = x;
      id[0] = col;
    }
  }

  __device__ __forceinline__ void chunk(const Params&, int c, const uint32_t (&v)[32]) {
    float x[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]);
    if (vlim < kBN) {                      // last vocab tile: columns >= V are padding
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c * 32 + j >= vlim) x[j] = -INFINITY;
    }
    float cm = x[0];
#pragma unroll
    for (int j = 1; j < 32; ++j) cm = fmaxf(cm, x[j]);
    const float nm = fmaxf(mx, cm);
    const float nref = nm * kLog2eS;                 // the sums' reference, in powers of two
    const float back = ref - nref;                   // <= 0; exactly 0 while the maximum stands
    const float f = ex2_approx(back);
    t = f * fmaf(s, back, t);
    s *= f;
    ref = nref;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float a = fmaf(x[j], kLog2eS, -nref);
      const float e = ex2_approx(a);
      s += e;
      t = fmaf(e, fmaxf(a, -1e30f), t);              // the bound keeps 0 * -inf out of T
    }
    mx = nm;
    const int jj = yl - c * 32;
    if (static_cast<unsigned>(jj) < 32u) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j == jj) zyv = x[j];
    }
    if (K > 0) {
      const bool any = cm >= tauv && cm > val[kList - 1];
      if (__any_sync(0xffffffffu, any)) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          m |= (x[j] >= tauv && x[j] > val[kList - 1] ? 1u : 0u) << j;
        while (__any_sync(0xffffffffu, m != 0)) {
          const int j = m ? __ffs(m) - 1 : 0;
          const float xv = pick32(x, j);
          if (m != 0) insert(xv, c * 32 + j);
          m &= m - 1;
        }
      }
    }
  }

  __device__ __forceinline__ void end(const Params& p) {
    if (!valid) return;
    const long long at = static_cast<long long>(nt) * p.ldp + tok;
    // ref is mx * log2(e) rounded: move the sums by the residue to mx itself
    const float r = fmaf(-mx, kLog2eS, ref);
    p.part[at] = make_float2(mx, fmaf(s, r * kLn2S, s));
    p.tsum[at] = fmaf(s, r, t) * kLn2S;
    if (yl >= 0 && yl < kBN && yl < vlim) p.zy[tok] = zyv;
    if (K > 0 && val[0] > kFloor) {
      float2* l = p.list + static_cast<long long>(nt) * K * p.ldp + tok;
#pragma unroll
      for (int j = 0; j < kList; ++j)
        l[static_cast<long long>(j) * p.ldp] = make_float2(val[j], __int_as_float(nt * kBN + id[j]));
      if (val[kList - 1] > fmaxf(tauv, kFloor)) atomicMax(p.tau + tok, ordered(val[kList - 1]));
    }
  }
};

// ------------------------------------------------------------------ lists across a warp
// A falling list of 32 (logit, id) entries, entry j in lane j.
struct Entry {
  float v;
  int id;
};

__device__ __forceinline__ bool ahead(const Entry& a, const Entry& b) {
  return a.v > b.v || (a.v == b.v && a.id < b.id);
}

// The 32 best of two falling lists: entry j against entry 31 - j of the other leaves the best
// 32 in an order that falls and then rises (or the reverse), which five exchange rounds sort.
__device__ __forceinline__ void merge_lists(Entry& a, Entry b, int lane) {
  b.v = __shfl_sync(0xffffffffu, b.v, 31 - lane);
  b.id = __shfl_sync(0xffffffffu, b.id, 31 - lane);
  if (ahead(b, a)) a = b;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const Entry o{__shfl_xor_sync(0xffffffffu, a.v, w), __shfl_xor_sync(0xffffffffu, a.id, w)};
    if (((lane & w) == 0) == ahead(o, a)) a = o;
  }
}

// ------------------------------------------------------------------ finish
struct StatsOut {
  float *logp, *entropy, *lse, *top_logp;
  int* top_ids;
  int n_top;
};

// One warp per position. Lane l joins tiles l, l + 32, ... (S and T in fp64, so that a
// vocabulary of millions loses nothing), then the lanes join by a fixed tree; tiles whose
// maximum reaches the threshold bring their lists in, in rising tile order.
template <int K>
__global__ void __launch_bounds__(256) k_stats_finish(const float2* __restrict__ part,
                                                      const float* __restrict__ tsum,
                                                      const float2* __restrict__ list,
                                                      const uint32_t* __restrict__ tau,
                                                      const float* __restrict__ zy,
                                                      const int* __restrict__ y, int n, int S,
                                                      int V, int ldp, StatsOut out, DevCtl ctl) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= n) return;
  float M = -INFINITY;
  double s = 0.0, t = 0.0;
  Entry best{-INFINITY, -1};
  const float tauv = K > 0 && tau != nullptr ? from_ordered(__ldg(tau + i)) : -INFINITY;
  auto join = [&](float m, double s2, double t2) {
    if (m == -INFINITY) return;
    if (m > M) {
      if (M != -INFINITY) {
        const double f = expf(M - m), back = M - m;
        t = f * (t + s * back) + t2;
        s = f * s + s2;
      } else {
        s = s2;
        t = t2;
      }
      M = m;
    } else {
      const double f = expf(m - M), back = m - M;
      t += f * (t2 + s2 * back);
      s += f * s2;
    }
  };
  for (int base = 0; base < S; base += 128) {
    float2 q[4];
    float tq[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = base + u * 32 + lane;
      q[u] = make_float2(-INFINITY, 0.f);
      tq[u] = 0.f;
      if (k < S) {
        q[u] = __ldg(part + static_cast<long long>(k) * ldp + i);
        tq[u] = __ldg(tsum + static_cast<long long>(k) * ldp + i);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) join(q[u].x, q[u].y, tq[u]);
    if (K > 0) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t hit = __ballot_sync(0xffffffffu, q[u].x > kFloor && q[u].x >= tauv);
        while (hit) {
          const int k = base + u * 32 + __ffs(hit) - 1;
          hit &= hit - 1;
          Entry e{-INFINITY, -1};
          if (lane < K) {
            const float2 r = __ldg(list + (static_cast<long long>(k) * K + lane) * ldp + i);
            if (r.x > kFloor) e = Entry{r.x, __float_as_int(r.y)};
          }
          // a later tile's equal logit has the higher id: only a larger one can enter a full list
          const float first = __shfl_sync(0xffffffffu, e.v, 0);
          const float last = __shfl_sync(0xffffffffu, best.v, K - 1);
          if (first > last) merge_lists(best, e, lane);
        }
      }
    }
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const float m2 = __shfl_down_sync(0xffffffffu, M, w);
    const double s2 = __shfl_down_sync(0xffffffffu, s, w);
    const double t2 = __shfl_down_sync(0xffffffffu, t, w);
    join(m2, s2, t2);
  }
  const double ls = log(s);
  const float lse = static_cast<float>(M + ls);
  if (lane == 0) {
    if (out.lse != nullptr) out.lse[i] = lse;
    if (out.entropy != nullptr) out.entropy[i] = static_cast<float>(ls - t / s);
    if (y != nullptr) {
      const int yi = __ldg(y + i);
      const bool ok = yi >= 0 && yi < V;
      if (!ok) record_status(ctl, kStatusBadTarget);
      // against M before log S: z_y - lse would round away what large logits leave
      if (out.logp != nullptr)
        out.logp[i] = ok ? static_cast<float>((static_cast<double>(__ldg(zy + i)) - M) - ls) : 0.f;
    }
  }
  const double m0 = __shfl_sync(0xffffffffu, M, 0), l0 = __shfl_sync(0xffffffffu, ls, 0);
  if (K > 0 && lane < out.n_top) {
    const long long at = static_cast<long long>(i) * out.n_top + lane;
    out.top_ids[at] = best.id;
    out.top_logp[at] = best.id >= 0 ? static_cast<float>((best.v - m0) - l0) : -INFINITY;
  }
}

// ------------------------------------------------------------------ fp32 route
// Each warp takes 32 vocabulary rows (one tile of partials) for kPos positions: W rows are
// read once per kPos positions, lanes stride over d, and after the 32 dot products lane l
// holds z of row l.
constexpr int kPos = 4;

template <int K>
__global__ void __launch_bounds__(256) k_stats_f32(const float* __restrict__ H,
                                                   const int* __restrict__ at, long long h_stride,
                                                   const float* __restrict__ W,
                                                   const int* __restrict__ y, int n, int d, int V,
                                                   int ldp, float2* __restrict__ part,
                                                   float* __restrict__ tsum,
                                                   float* __restrict__ zy,
                                                   float2* __restrict__ list) {
  const int lane = threadIdx.x & 31;
  const int nt = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int v0 = nt * 32;
  if (v0 >= V) return;
  const int i0 = blockIdx.y * kPos;
  const float* h[kPos];
#pragma unroll
  for (int q = 0; q < kPos; ++q) {
    const int i = min(i0 + q, n - 1);
    h[q] = H + (at != nullptr ? at[i] : i) * h_stride;
  }
  float z[kPos];
#pragma unroll
  for (int q = 0; q < kPos; ++q) z[q] = -INFINITY;
  for (int r = 0; r < 32 && v0 + r < V; ++r) {
    const float* w = W + static_cast<long long>(v0 + r) * d;
    float a[kPos] = {};
    for (int k = lane; k < d; k += 32) {
      const float wk = __ldg(w + k);
#pragma unroll
      for (int q = 0; q < kPos; ++q) a[q] = fmaf(__ldg(h[q] + k), wk, a[q]);
    }
#pragma unroll
    for (int q = 0; q < kPos; ++q) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a[q] += __shfl_xor_sync(0xffffffffu, a[q], o);
      if (lane == r) z[q] = a[q];
    }
  }
#pragma unroll
  for (int q = 0; q < kPos; ++q) {
    const int i = i0 + q;
    if (i >= n) break;
    const float x = z[q];
    float m = fmaxf(x, kFloor);                 // padding rows hold -inf; a NaN gives the floor
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float e = expf(x - m);
    float s = e, t = e > 0.f ? e * (x - m) : (e == 0.f ? 0.f : e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    const long long to = static_cast<long long>(nt) * ldp + i;
    if (lane == 0) {
      part[to] = make_float2(m, s);
      tsum[to] = t;
    }
    if (y != nullptr && __ldg(y + i) == v0 + lane && v0 + lane < V) zy[i] = x;
    if (K > 0) {
      Entry best{-INFINITY, -1};
      for (int r = 0; r < 32; ++r) {            // insertion across the lanes, in rising id
        const float xr = __shfl_sync(0xffffffffu, x, r);
        const bool take = xr > kFloor;          // false for NaN
        const int at_lane = __popc(__ballot_sync(0xffffffffu, best.v >= xr));
        const Entry up{__shfl_up_sync(0xffffffffu, best.v, 1),
                       __shfl_up_sync(0xffffffffu, best.id, 1)};
        if (take) best = lane < at_lane ? best : (lane == at_lane ? Entry{xr, v0 + r} : up);
      }
      if (lane < K)
        list[(static_cast<long long>(nt) * K + lane) * ldp + i] =
            make_float2(best.v, __int_as_float(best.id));
    }
  }
}

// ------------------------------------------------------------------ launches
int stats_list_len(int n_top) { return n_top == 0 ? 0 : n_top == 1 ? 1 : n_top <= 8 ? 8 : 32; }

int stats_tiles(bool bf16, int V) { return (V + (bf16 ? kBN : 32) - 1) / (bf16 ? kBN : 32); }

namespace {

template <int K>
cudaError_t stats_bf16(const CUtensorMap& mapA, const CUtensorMap& mapB, const StatsBuf& b, int n,
                       int V, int d, const int* y, int sms, int* sync, const DevCtl& ctl,
                       cudaStream_t st) {
  if (K > 0) {
    const cudaError_t e = cudaMemsetAsync(b.tau, 0, sizeof(uint32_t) * n, st);
    if (e != cudaSuccess) return e;
  }
  typename EpiStats<K>::Params p{y, b.part, b.tsum, b.zy, b.tau, b.list, n, V, b.ldp};
  return launch_gemm<false, false, EpiStats<K>>(mapA, mapB, mapA, n, V, d, 2, p, sms, ctl, st,
                                                kGemmForward, token_group(d), sync);
}

template <int K>
cudaError_t stats_finish(const StatsBuf& b, bool with_tau, int n, int S, int V, const int* y,
                         const StatsOut& out, const DevCtl& ctl, cudaStream_t st) {
  k_stats_finish<K><<<(n + 7) / 8, 256, 0, st>>>(b.part, b.tsum, b.list, with_tau ? b.tau : nullptr,
                                                 b.zy, y, n, S, V, b.ldp, out, ctl);
  return cudaGetLastError();
}

}  // namespace

#define DPO_BY_LIST(K, call)                       \
  ((K) == 0   ? call<0>                            \
   : (K) == 1 ? call<1>                            \
   : (K) == 8 ? call<8>                            \
              : call<32>)

cudaError_t launch_stats_bf16(const CUtensorMap& mapA, const CUtensorMap& mapB, const StatsBuf& b,
                              int n_top, int n, int V, int d, const int* y, int sms, int* sync,
                              const DevCtl& ctl, cudaStream_t st) {
  return DPO_BY_LIST(stats_list_len(n_top), stats_bf16)(mapA, mapB, b, n, V, d, y, sms, sync, ctl,
                                                        st);
}

cudaError_t launch_stats_f32(const float* H, const int* at, long long h_stride, const float* W,
                             const StatsBuf& b, int n_top, int n, int V, int d, const int* y,
                             cudaStream_t st) {
  const int K = stats_list_len(n_top);
  const dim3 grid((stats_tiles(false, V) + 7) / 8, (n + kPos - 1) / kPos);
  auto kern = K == 0   ? k_stats_f32<0>
              : K == 1 ? k_stats_f32<1>
              : K == 8 ? k_stats_f32<8>
                       : k_stats_f32<32>;
  kern<<<grid, 256, 0, st>>>(H, at, h_stride, W, y, n, d, V, b.ldp, b.part, b.tsum, b.zy, b.list);
  return cudaGetLastError();
}

cudaError_t launch_stats_finish(const StatsBuf& b, bool bf16, int n_top, int n, int V, const int* y,
                                float* logp, float* entropy, float* lse, int* top_ids,
                                float* top_logp, const DevCtl& ctl, cudaStream_t st) {
  const StatsOut out{logp, entropy, lse, top_logp, top_ids, n_top};
  return DPO_BY_LIST(stats_list_len(n_top), stats_finish)(b, bf16, n, stats_tiles(bf16, V), V, y,
                                                          out, ctl, st);
}

}  // namespace dpo
