// Token statistics: log-prob of a given token, entropy and the largest logits of each
// position, from one pass over the vocabulary that never stores the logits.
//   k_tc_gemm<EpiStats<K>>  z = Hp . W^T on tcgen05; the epilogue keeps, per position and
//                    vocabulary tile, the running maximum m, S = sum e^(z-m),
//                    T = sum e^(z-m) (z-m), the target logit and the tile's K largest logits
//   k_stats_f32<K>   the same partials on the fp32 SIMT route
//   k_stats_join<K>  joins the tiles, a block per position (stats_join.cuh), or
//   k_stats_finish<K>  a warp per position: many positions, or very many tiles
// Up to 64 bf16 positions stream W instead (stats_stream.cu).
//
// Entropy: -sum p log p = log S - T / S. Both terms are >= 0 (T <= 0), so the sum does not
// cancel, and T rescales with the maximum like S does: moving from m to m' multiplies both
// by f = e^(m-m') after T has taken S (m - m').
#include <cmath>

#include "internal.h"
#include "gemm_launch.cuh"
#include "stats.cuh"
#include "stats_join.cuh"

namespace dpo {

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
// matter. The tiles fall into K groups (tile mod K); each position has a threshold per group in
// global memory, the largest logit any finished tile of the group has bid (atomicMax; the maximum
// does not depend on the order). K groups stand for K different logits, so the smallest of them is
// a lower bound of the position's K-th largest logit, and a close one: about K log K logits reach
// it. A tile takes a logit only if it reaches the bound, and the finish looks at a tile only if
// the tile's maximum reaches the final bound: such a tile did write its list, because the bound it
// saw was no higher. (With the largest K-th logit of any one tile as the bound, 4 logits of every
// tile reached it at K = 8.)
template <int K>
struct EpiStats {
  static constexpr bool kStaging = false;
  static constexpr bool kSystemFence = false;
  struct Params {
    const int* y;        // given token of each position, or nullptr
    float2* part;        // [S, ldp] (m, S)
    float* tsum;         // [S, ldp] T
    float* zy;           // [ldp] target logit
    uint32_t* tau;       // [K, ldp] thresholds, zeroed before the launch
    float2* list;        // [S, K, ldp] (logit, id), falling, fillers (<= kFloor, -)
    int n, V, ldp;
  };
  static constexpr int kList = K > 0 ? K : 1;
  int tok, nt, yl, vlim;
  bool valid;
  float mx, ref, s, t, zyv, tauv;
  float val[kList];
  int id[kList];
  uint32_t bid;          // the highest bid of this tile's group so far

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
      uint32_t th = 0xffffffffu;
      bid = 0;
#pragma unroll
      for (int g = 0; g < kList; ++g) {
        const uint32_t o = valid ? __ldcg(p.tau + static_cast<long long>(g) * p.ldp + tok) : 0u;
        th = min(th, o);
        if (g == nt % kList) bid = o;
      }
      tauv = valid ? from_ordered(th) : INFINITY;                // padding rows take nothing
#pragma unroll
      for (int j = 0; j < kList; ++j) {
        val[j] = kFloor;
        id[j] = 0;
      }
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
    // the sums' reference in powers of two: the rounded product, not a fused one
    const float nref = __fmul_rn(nm, kLog2eS);
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
          if (m != 0) insert_sorted<kList>(val, id, xv, c * 32 + j);
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
      if (ordered(val[0]) > bid)
        atomicMax(p.tau + static_cast<long long>(nt % kList) * p.ldp + tok, ordered(val[0]));
    }
  }
};

// ------------------------------------------------------------------ finish
// Tiles in id order: the GEMM's or the SIMT route's partials, as the join reads them.
template <int K>
struct TileSets {
  const float2* part;
  const float* tsum;
  const float2* list;
  const uint32_t* tau;       // or nullptr
  int S, ldp;
  static constexpr int kFrom = 0;
  __device__ __forceinline__ int sums() const { return S; }
  __device__ __forceinline__ float4 sum(int p, int k) const {
    const long long at = static_cast<long long>(k) * ldp + p;
    const float2 q = __ldcg(part + at);
    return make_float4(q.x, q.y, __ldcg(tsum + at), 0.f);
  }
  __device__ __forceinline__ int sets() const { return S; }
  __device__ __forceinline__ uint32_t floor_of(int p, int lane) const {
    if (tau == nullptr) return 0;
    return __reduce_min_sync(
        0xffffffffu, lane < K ? __ldcg(tau + static_cast<long long>(lane) * ldp + p) : 0xffffffffu);
  }
  __device__ __forceinline__ unsigned long long key(int p, int k, uint32_t floor) const {
    const float m = __ldcg(part + static_cast<long long>(k) * ldp + p).x;
    return ordered(m) >= floor ? entry_key(make_float2(m, __int_as_float(k))) : 0;
  }
  template <int KK>
  __device__ __forceinline__ int group(int k) const {
    return k % KK;
  }
  template <int KK>
  __device__ __forceinline__ float2 entry(int p, unsigned long long key, int j) const {
    return __ldcg(list + (static_cast<long long>(key_id(key)) * KK + j) * ldp + p);
  }
};

// The join of many positions, or of more tiles than stats_join.cuh's has room for: one warp per
// position. Lane l joins tiles l, l + 32, ..., then the lanes join in a fixed order (S and T in
// fp64, so that a vocabulary of millions loses nothing).
//
// Alternatives. The K largest logits lie in the K first tiles by (maximum falling, id rising): a
// logit of any other tile has the maxima of those K ahead of it. So the warp keeps the K first
// tiles while it reads the partials; their maxima are then a sorted list of logits already, and
// the tiles' second, third, ... entries go in until none is ahead of the list's last. (Joining
// every tile's list instead, in one chain of dependent loads, took 230 us of the 435 us of a
// single token at V = 128,256.)
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
  after_previous();
  // what the kernel before wrote is read past L1 (__ldcg): this one may have started before it
  constexpr int U = 4;
  uint32_t th = 0;
  if (K > 0 && tau != nullptr)
    th = lane < K ? __ldcg(tau + static_cast<long long>(lane) * ldp + i) : 0xffffffffu;
  Sums a;
  Entry best{-INFINITY, -1};              // tiles by their maximum
  float tauv = 0.f;
  for (int base = 0; base < S; base += 32 * U) {
    float2 q[U];
    float tq[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = base + u * 32 + lane;
      q[u] = make_float2(-INFINITY, 0.f);
      tq[u] = 0.f;
      if (k < S) {
        q[u] = __ldcg(part + static_cast<long long>(k) * ldp + i);
        tq[u] = __ldcg(tsum + static_cast<long long>(k) * ldp + i);
      }
    }
    if (K > 0 && base == 0) tauv = from_ordered(__reduce_min_sync(0xffffffffu, th));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      a.join(q[u].x, q[u].y, tq[u]);
      if (K > 0) {
        // tiles come in rising order: an equal maximum is behind the ones held
        const float m = q[u].x > kFloor && q[u].x >= tauv ? q[u].x : -INFINITY;
        uint32_t hit = __ballot_sync(0xffffffffu, m > __shfl_sync(0xffffffffu, best.v, K - 1));
        while (hit) {
          const int src = __ffs(hit) - 1;
          insert_entry(best, Entry{__shfl_sync(0xffffffffu, m, src),
                                   base + u * 32 + src}, lane);
          hit &= hit - 1;
          hit &= __ballot_sync(0xffffffffu, m > __shfl_sync(0xffffffffu, best.v, K - 1));
        }
      }
    }
  }
  warp_join(a.M, a.s, a.t);
  const double ls = log(a.s);
  if (lane == 0) {
    if (out.lse != nullptr) out.lse[i] = static_cast<float>(a.M + ls);
    if (out.entropy != nullptr) out.entropy[i] = entropy_of(static_cast<float>(ls - a.t / a.s));
    if (y != nullptr) {
      const int yi = __ldcg(y + i);
      const bool ok = yi >= 0 && yi < V;
      if (!ok) record_status(ctl, kStatusBadTarget);
      // against M before log S: z_y - lse would round away what large logits leave
      if (out.logp != nullptr)
        out.logp[i] = ok ? static_cast<float>((static_cast<double>(__ldcg(zy + i)) - a.M) - ls) : 0.f;
    }
  }
  if (K > 0) {
    const double m0 = a.M, l0 = ls;       // every lane has them
    bool more = lane < K && best.id >= 0;
    const float2* mine = list + static_cast<long long>(best.id) * K * ldp + i;   // lane j: tile j
    Entry top{-INFINITY, -1};
    if (more) {
      const float2 r = __ldcg(mine);
      top = Entry{r.x, __float_as_int(r.y)};
    }
    for (int j = 1; j < K; ++j) {
      Entry e{-INFINITY, -1};
      if (more) {
        const float2 r = __ldcg(mine + static_cast<long long>(j) * ldp);
        if (r.x > kFloor) e = Entry{r.x, __float_as_int(r.y)};
      }
      more = take_entries<K>(top, e, lane);   // a tile's entries fall: no later one can go in either
      if (!__any_sync(0xffffffffu, more)) break;
    }
    if (lane < out.n_top) {
      const long long at = static_cast<long long>(i) * out.n_top + lane;
      out.top_ids[at] = top.id;
      out.top_logp[at] = top.id >= 0 ? static_cast<float>((top.v - m0) - l0) : -INFINITY;
    }
  }
}

// ------------------------------------------------------------------ fp32 route
// A block takes 32 vocabulary rows (one tile of partials) and 32 positions, a warp 4 of them, a
// lane one vocabulary row: z = h . w is summed in the lane, over d in pieces that both operands
// pass through shared memory, and no exchange between lanes is needed before the statistics. W is
// read once per 32 positions. (With lanes along d, a warp per vocabulary row and five exchanges
// per logit it took 37 us at 65 positions, V = 1000, d = 64.)
constexpr int kPos = 4;                  // positions per warp
constexpr int kF32Rows = 32;             // vocabulary rows per tile
constexpr int kF32Pos = 8 * kPos;        // positions per block
constexpr int kF32K = 32;                // values of d per piece

template <int K>
__global__ void __launch_bounds__(256) k_stats_f32(const float* __restrict__ H,
                                                   const int* __restrict__ at, long long h_stride,
                                                   const float* __restrict__ W,
                                                   const int* __restrict__ y, int n, int d, int V,
                                                   int ldp, float2* __restrict__ part,
                                                   float* __restrict__ tsum,
                                                   float* __restrict__ zy,
                                                   float2* __restrict__ list) {
  // rows of 9 groups of 4 values: lanes 8 rows apart start 8 banks apart
  __shared__ float4 sw[kF32Rows][kF32K / 4 + 1], sh[kF32Pos][kF32K / 4 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nt = blockIdx.x, v0 = nt * kF32Rows;
  const int base = blockIdx.y * kF32Pos, i0 = base + warp * kPos;
  // this thread copies 4 values of one row of each operand per piece
  const int cr = threadIdx.x >> 3, ck = threadIdx.x & 7;
  const float* w = W + static_cast<long long>(min(v0 + cr, V - 1)) * d;
  const int hi = min(base + cr, n - 1);
  const float* h = H + (at != nullptr ? at[hi] : hi) * h_stride;
  float z[kPos] = {};
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 cw = none, ch = none;
  if (ck * 4 < d) {                        // d is a multiple of 8: 4 values are all in or all out
    cw = __ldg(reinterpret_cast<const float4*>(w) + ck);
    ch = __ldg(reinterpret_cast<const float4*>(h) + ck);
  }
  for (int k0 = 0; k0 < d; k0 += kF32K) {
    __syncthreads();
    sw[cr][ck] = cw;
    sh[cr][ck] = ch;
    __syncthreads();
    const int k = k0 + kF32K + ck * 4;     // the next piece while this one is worked on
    cw = k < d ? __ldg(reinterpret_cast<const float4*>(w + k)) : none;
    ch = k < d ? __ldg(reinterpret_cast<const float4*>(h + k)) : none;
#pragma unroll
    for (int c = 0; c < kF32K / 4; ++c) {
      const float4 a = sw[lane][c];
#pragma unroll
      for (int q = 0; q < kPos; ++q) {
        const float4 b = sh[warp * kPos + q][c];
        z[q] = fmaf(a.x, b.x, z[q]);
        z[q] = fmaf(a.y, b.y, z[q]);
        z[q] = fmaf(a.z, b.z, z[q]);
        z[q] = fmaf(a.w, b.w, z[q]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kPos; ++q) {
    const int i = i0 + q;
    if (i >= n) break;
    const float x = v0 + lane < V ? z[q] : -INFINITY;
    const float m = from_ordered(__reduce_max_sync(0xffffffffu, ordered(fmaxf(x, kFloor))));
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
      // the lane's rank is the number of rows ahead of it
      const uint32_t mine = x > kFloor ? ordered(x) : 0u;      // 0: none (NaN included)
      int rank = 0;
      for (int r = 0; r < 32; ++r) {
        const uint32_t other = __shfl_sync(0xffffffffu, mine, r);
        rank += other > mine || (other == mine && r < lane) ? 1 : 0;
      }
      if (rank < K)
        list[(static_cast<long long>(nt) * K + rank) * ldp + i] =
            mine != 0 ? make_float2(x, __int_as_float(v0 + lane)) : make_float2(kFloor, 0.f);
    }
  }
}

// ------------------------------------------------------------------ launches
// List lengths compiled: the upkeep grows with K (48 positions over V = 151,936, d = 2,048: 103 us
// without alternatives, 106, 110 and 121 us at K = 1, 8 and 32; 8,000 over V = 32,000, d = 512, where the
// upkeep is most of the time: 235, 274, 446 and 1131 us), so one length for all would cost short lists.
int stats_list_len(int n_top) { return n_top == 0 ? 0 : n_top == 1 ? 1 : n_top <= 8 ? 8 : 32; }

int stats_tiles(bool bf16, int V) {
  const int rows = bf16 ? kBN : kF32Rows;
  return (V + rows - 1) / rows;
}

namespace {

// Calls of up to this many positions join each one's tiles by a block, larger ones by a warp. In all, at
// V = 32,000, d = 512, with 0 / 8 / 20 alternatives: 300 positions 25.6 / 57 / 120 us by blocks and
// 27.5 / 59 / 128 us by warps, 1,000 44 / 89 / 206 and 44 / 89 / 208, 2,000 75 / 145 / 359 and
// 73 / 139 / 349, 8,000 243 / 477 / 1189 and 235 / 446 / 1131.
constexpr int kBlockJoin = 1024;

template <int K>
cudaError_t stats_bf16(const CUtensorMap& mapA, const CUtensorMap& mapB, const StatsBuf& b, int n,
                       int V, int d, const int* y, int sms, int* sync, const DevCtl& ctl,
                       cudaStream_t st) {
  if (K > 0) {
    const cudaError_t e =
        cudaMemsetAsync(b.tau, 0, sizeof(uint32_t) * static_cast<size_t>(K) * b.ldp, st);
    if (e != cudaSuccess) return e;
  }
  typename EpiStats<K>::Params p{y, b.part, b.tsum, b.zy, b.tau, b.list, n, V, b.ldp};
  return launch_gemm<false, false, EpiStats<K>>(mapA, mapB, mapA, n, V, d, 2, p, sms, ctl, st,
                                                kGemmForward, token_group(d), sync);
}

template <int K>
cudaError_t stats_finish(const StatsBuf& b, bool with_tau, int n, long long n_call, int S, int V,
                         const int* y, const StatsOut& out, const DevCtl& ctl, cudaStream_t st) {
  const uint32_t* tau = with_tau ? b.tau : nullptr;
  if (n_call <= kBlockJoin && S <= kJoinSets)
    return launch_join<K>(TileSets<K>{b.part, b.tsum, b.list, tau, S, b.ldp}, y, b.zy, n, V, out, ctl,
                          st);
  return launch_after(k_stats_finish<K>, dim3((n + 7) / 8), 256, st, b.part, b.tsum, b.list, tau, b.zy,
                      y, n, S, V, b.ldp, out, ctl);
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
  const dim3 grid(stats_tiles(false, V), (n + kF32Pos - 1) / kF32Pos);
  auto kern = K == 0   ? k_stats_f32<0>
              : K == 1 ? k_stats_f32<1>
              : K == 8 ? k_stats_f32<8>
                       : k_stats_f32<32>;
  kern<<<grid, 256, 0, st>>>(H, at, h_stride, W, y, n, d, V, b.ldp, b.part, b.tsum, b.zy, b.list);
  return cudaGetLastError();
}

cudaError_t launch_stats_finish(const StatsBuf& b, bool thresholds, int S, int n, long long n_call,
                                int V, const int* y, const StatsOut& out, const DevCtl& ctl,
                                cudaStream_t st) {
  return DPO_BY_LIST(stats_list_len(out.n_top), stats_finish)(b, thresholds, n, n_call, S, V, y, out,
                                                              ctl, st);
}

}  // namespace dpo
