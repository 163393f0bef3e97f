// The norm's backward (see norm.cu for the formulas): x and dy are read once and dx written once,
// so HBM bounds it; the weight gradients gather on chip and leave one partial row per block, which
// k_norm_dw_sum adds up in a fixed order. 16,384 rows of 4,096, bf16 x, fp32 dy, both weight
// gradients: 82 us (6.5 TB/s), 85 us in calls one after another; bf16 dy 70 us.
// By the row's length d (times with the weight gradients, bf16 x, fp32 dy):
//   d <= 128   a few lanes per row, one group of 8 values per lane (262,144 rows of 128: 58 us, a
//              warp per row 73 us; of 256: 113 us and 90 us)
//   d <= 8192  groups of 1 to 8 warps per row (8,192 rows of 8,192: 95 us; as below 168 us)
//   above      a block per row that reads it twice, and a column sum that reads it again: the weight
//              gradients of a row of 16,384 no longer fit the registers and shared memory of one SM
//              beside two rows (4,096 rows of 16,384: 158 us, half the rate). A row split over a
//              cluster of two would; it is not built.
#include "chain.cuh"
#include "norm.cuh"

namespace dpo {

namespace {

struct BwdArgs {
  int rows, d, wbf16;
  const void* weight;
  const float *mean, *rstd;     // mean NULL: rms
  float *pw, *pb;               // [parts, d] partial weight gradients, or NULL
};

// One row's terms: xh in place of x (f), g in place of dy (e), the weight gradients' and the row
// sums' additions.
template <bool kMean>
__device__ __forceinline__ void grad_terms(float2 (&f)[4], float2 (&e)[4], float mu, float r,
                                           const float2 (&w)[4], float2 (&aw)[4], float2 (&ab)[4],
                                           float& c1, float& c2) {
  float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = __fmul2_rn(kMean ? __fadd2_rn(f[j], both(-mu)) : f[j], both(r));
    aw[j] = __ffma2_rn(e[j], f[j], aw[j]);
    ab[j] = __fadd2_rn(ab[j], e[j]);
    e[j] = __fmul2_rn(e[j], w[j]);
    if (kMean) s1 = __fadd2_rn(s1, e[j]);
    s2 = __ffma2_rn(e[j], f[j], s2);
  }
  c1 = s1.x + s1.y;
  c2 = s2.x + s2.y;
}
// dx = r (g - c1 - xh c2), into xh's place
template <bool kMean>
__device__ __forceinline__ void grad_x(float2 (&f)[4], const float2 (&g)[4], float r, float c1,
                                       float c2) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 t = __ffma2_rn(f[j], both(-c2), g[j]);
    f[j] = __fmul2_rn(kMean ? __fadd2_rn(t, both(-c1)) : t, both(r));
  }
}

constexpr int kShortThreads = 256;

// Short rows: G lanes per row; the block's rows leave one partial weight gradient.
template <class X, class Dy, class Dx, int G>
__global__ void __launch_bounds__(kShortThreads) k_norm_bwd_short(X x, Dy dy, Dx dx, BwdArgs a) {
  constexpr int kRows = kShortThreads / G;      // rows at a time
  __shared__ float red[kRows][G * 8 + 1];
  const int lane = threadIdx.x & (G - 1), sub = threadIdx.x / G, col = lane * 8;
  const bool in = col < a.d;
  const float inv_d = 1.f / static_cast<float>(a.d);
  float2 w[4], aw[4], ab[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = aw[j] = ab[j] = both(0.f);
  if (in) load_vec(a.weight, a.wbf16, col, 1.f, w);
  // every thread of a warp makes the same number of rounds: the exchanges need them all
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  const long long first = static_cast<long long>(blockIdx.x) * kRows;
  for (long long r0 = first; r0 < a.rows; r0 += 2 * step) {
    typename X::Raw rx[2];
    typename Dy::Raw rd[2];
    float mu[2], rs[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const long long row = r0 + q * step + sub;
      mu[q] = rs[q] = 0.f;
      if (in && row < a.rows) {
        rx[q] = x.load(row, col);
        rd[q] = dy.load(row, col);
        if (a.mean != nullptr) mu[q] = __ldg(a.mean + row);
        rs[q] = __ldg(a.rstd + row);
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const long long row = r0 + q * step + sub;
      const bool ok = in && row < a.rows;
      float2 f[4], e[4];
      float c1 = 0.f, c2 = 0.f;
      if (ok) {
        X::widen(rx[q], f);
        Dy::widen(rd[q], e);
        grad_terms<true>(f, e, mu[q], rs[q], w, aw, ab, c1, c2);
      }
      c1 = a.mean != nullptr ? lanes_total<G>(c1) * inv_d : 0.f;
      c2 = lanes_total<G>(c2) * inv_d;
      if (ok && dx.p != nullptr) {
        grad_x<true>(f, e, rs[q], c1, c2);
        dx.store(row, col, f);
      }
    }
  }
  for (int which = 0; which < 2; ++which) {
    float* out = which == 0 ? a.pw : a.pb;
    if (out == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[sub][col + 2 * j] = which == 0 ? aw[j].x : ab[j].x;
      red[sub][col + 2 * j + 1] = which == 0 ? aw[j].y : ab[j].y;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += kShortThreads) {
      float s = 0.f;
      for (int k = 0; k < kRows; ++k) s += red[k][c];
      out[static_cast<long long>(blockIdx.x) * a.d + c] = s;
    }
  }
}

// Groups of WG warps per row, NV groups of 8 values per lane (see the forward): a lane's columns
// stay the same from row to row, so the weight gradients gather in its registers; the block's
// groups add theirs up at the end and leave one partial gradient. Two slots per group: while a
// row is worked on, the next two are on their way. More than 2 groups a lane leave no registers
// for g, more than 3 none for xh either: those are formed again from the slot, which is then
// refilled a little later. (8,192 rows of 8,192: 95 us; with xh kept 116 us, with both and 384
// threads 115 us.)
constexpr int kSlots = 2;
constexpr bool holds_g(int nv) { return nv <= 2; }
constexpr bool holds_xh(int nv) { return nv <= 3; }

template <class X, class Dy, class Dx, int NV, int WG, int kThreads, bool kMean>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_rows(X x, Dy dy, Dx dx, BwdArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];   // weight [d] fp32; the groups' slots
  __shared__ float red[2][2][kThreads / 32];
  constexpr int kLanes = WG * 32;
  constexpr uint32_t kSlotDy = NV * kLanes * Dy::kSlot, kSlot = kSlotDy + NV * kLanes * X::kSlot;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / WG, wg = warp % WG, groups = (blockDim.x >> 5) / WG;
  const int gl = wg * 32 + lane;
  const int vecs = a.d / 8;
  const Planes sw{reinterpret_cast<float4*>(smem_raw), vecs};
  const uint32_t ring = smem_u32(sw.p + 2 * vecs) + group * kSlots * kSlot;
  const long long step = static_cast<long long>(gridDim.x) * groups;
  long long row = static_cast<long long>(blockIdx.x) * groups + group;
  auto fetch = [&](long long r, uint32_t slot) {
    if (r < a.rows) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        dy.fetch(slot, u * kLanes + gl, vecs, r);
        x.fetch(slot + kSlotDy, u * kLanes + gl, vecs, r);
      }
    }
    cp_async_commit();
  };
  fetch(row, ring);
  fetch(row + step, ring + kSlot);
  // the next row's statistics and scales are asked for while this one is worked on
  auto stat = [&](const float* p, long long r) {
    return p != nullptr && r < a.rows ? __ldg(p + r) : 0.f;
  };
  float mu = kMean ? stat(a.mean, row) : 0.f, rs = stat(a.rstd, row);
  typename X::Side side[NV];
  auto sides = [&](long long r) {
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (r < a.rows && u * kLanes + gl < vecs) side[u] = x.side(r, u * kLanes + gl);
  };
  sides(row);
  for (int k = threadIdx.x; k < vecs; k += blockDim.x) {
    float2 f[4];
    load_vec(a.weight, a.wbf16, k * 8, 1.f, f);
    sw.store(k, f);
  }
  __syncthreads();
  const float inv_d = 1.f / static_cast<float>(a.d);
  float2 aw[NV][4], ab[NV][4];
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j) aw[u][j] = ab[u][j] = both(0.f);
  int turn = 0;
  for (; row < a.rows; row += step) {
    const uint32_t slot = ring + turn * kSlot;
    cp_async_wait<kSlots - 1>();
    __syncwarp();
    const float mu2 = kMean ? stat(a.mean, row + step) : 0.f, rs2 = stat(a.rstd, row + step);
    constexpr bool kHold = holds_g(NV);
    constexpr bool kHoldX = holds_xh(NV);
    float2 f[kHoldX ? NV : 1][4], e[kHold ? NV : 1][4];
    float c1 = 0.f, c2 = 0.f;
    auto terms = [&](int u, int k, float2 (&dyv)[4]) {
      float2 w[4];
      sw.load(k, w);
      float p1, p2;
      grad_terms<kMean>(f[kHoldX ? u : 0], dyv, mu, rs, w, aw[u], ab[u], p1, p2);
      c1 += p1;
      c2 += p2;
    };
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int k = u * kLanes + gl;
      if (k < vecs) {
        float2 (&dyv)[4] = e[kHold ? u : 0];
        Dy::widen(Dy::take(slot, k, {}), dyv);
        X::widen(X::take(slot + kSlotDy, k, side[u]), f[kHoldX ? u : 0]);
        if (!kHold) terms(u, k, dyv);
      }
    }
    if (kHold) {
      __syncwarp();
      fetch(row + 2 * step, slot);                      // the slot is read: refill it
    }
    if (kHoldX) sides(row + step);
    if (kHold) {
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (u * kLanes + gl < vecs) terms(u, u * kLanes + gl, e[kHold ? u : 0]);
    }
    c1 = kMean ? lanes_total(c1) : 0.f;
    c2 = lanes_total(c2);
    if constexpr (WG > 1) {
      float* b1 = &red[turn][0][group * WG];
      float* b2 = &red[turn][1][group * WG];
      if (lane == 0) {
        if (kMean) b1[wg] = c1;
        b2[wg] = c2;
      }
      group_sync(group, kLanes);
      c1 = c2 = 0.f;
#pragma unroll
      for (int k = 0; k < WG; ++k) {
        if (kMean) c1 += b1[k];
        c2 += b2[k];
      }
    }
    if (dx.p != nullptr) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int k = u * kLanes + gl;
        if (k < vecs) {
          float2 (&g)[4] = e[kHold ? u : 0];
          if (!kHold) {
            float2 w[4];
            sw.load(k, w);
            Dy::widen(Dy::take(slot, k, {}), g);
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = __fmul2_rn(g[j], w[j]);
          }
          float2 (&xh)[4] = f[kHoldX ? u : 0];
          if (!kHoldX) {
            X::widen(X::take(slot + kSlotDy, k, side[u]), xh);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              xh[j] = __fmul2_rn(kMean ? __fadd2_rn(xh[j], both(-mu)) : xh[j], both(rs));
          }
          grad_x<kMean>(xh, g, rs, c1 * inv_d, c2 * inv_d);
          dx.store(row, k * 8, xh);
        }
      }
    }
    if (!kHold) {
      __syncwarp();
      fetch(row + 2 * step, slot);
    }
    if (!kHoldX) sides(row + step);
    mu = mu2;
    rs = rs2;
    turn ^= 1;
  }
  // the groups' gradients meet where the slots were, and are added in group order
  cp_async_wait<0>();
  float* meet = reinterpret_cast<float*>(sw.p + 2 * vecs);      // [groups][d]
  for (int which = 0; which < 2; ++which) {
    float* out = which == 0 ? a.pw : a.pb;
    if (out == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int k = u * kLanes + gl;
      if (k < vecs) OutF32{meet, a.d}.store(group, k * 8, which == 0 ? aw[u] : ab[u]);
    }
    __syncthreads();
    for (int c = threadIdx.x * 4; c < a.d; c += blockDim.x * 4) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int g = 0; g < groups; ++g) {
        const float4 v = *reinterpret_cast<const float4*>(meet + static_cast<long long>(g) * a.d + c);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      *reinterpret_cast<float4*>(out + static_cast<long long>(blockIdx.x) * a.d + c) = s;
    }
  }
}

// Long rows: dx with one block per row and two readings of it, and the weight gradients over
// slabs of 256 columns and splits of the rows.
template <class X, class Dy, class Dx>
__global__ void __launch_bounds__(kWideThreads) k_norm_dx_wide(X x, Dy dy, Dx dx, BwdArgs a) {
  __shared__ float buf[32];
  const long long row = blockIdx.x;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const float mu = a.mean != nullptr ? __ldg(a.mean + row) : 0.f, r = __ldg(a.rstd + row);
  float c1 = 0.f, c2 = 0.f;
  float2 f[4], e[4], w[4], unused[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) unused[j] = both(0.f);
  for (int col = threadIdx.x * 8; col < a.d; col += kWideThreads * 8) {
    X::widen(x.load(row, col), f);
    Dy::widen(dy.load(row, col), e);
    load_vec(a.weight, a.wbf16, col, 1.f, w);
    float p1, p2;
    grad_terms<true>(f, e, mu, r, w, unused, unused, p1, p2);
    c1 += p1;
    c2 += p2;
  }
  c1 = block_total(c1, buf) * inv_d;
  c2 = block_total(c2, buf) * inv_d;
  if (a.mean == nullptr) c1 = 0.f;
  for (int col = threadIdx.x * 8; col < a.d; col += kWideThreads * 8) {
    X::widen(x.load(row, col), f);
    Dy::widen(dy.load(row, col), e);
    load_vec(a.weight, a.wbf16, col, 1.f, w);
    float p1, p2;
    grad_terms<true>(f, e, mu, r, w, unused, unused, p1, p2);
    grad_x<true>(f, e, r, c1, c2);
    dx.store(row, col, f);
  }
}

// Partial weight gradients of a slab of 256 columns (blockIdx.x) and a split of the rows
// (blockIdx.y): warp w takes rows w, w + 8, ... of the split, its lanes 8 columns each.
template <class X, class Dy>
__global__ void __launch_bounds__(256) k_norm_dw_wide(X x, Dy dy, BwdArgs a) {
  __shared__ float red[8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 256 + lane * 8;
  const long long r0 = static_cast<long long>(a.rows) * blockIdx.y / gridDim.y;
  const long long r1 = static_cast<long long>(a.rows) * (blockIdx.y + 1) / gridDim.y;
  float2 aw[4], ab[4], w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = aw[j] = ab[j] = both(0.f);
  if (col < a.d) {
    for (long long row = r0 + warp; row < r1; row += 8) {
      float2 f[4], e[4];
      X::widen(x.load(row, col), f);
      Dy::widen(dy.load(row, col), e);
      float p1, p2;
      grad_terms<true>(f, e, a.mean != nullptr ? __ldg(a.mean + row) : 0.f, __ldg(a.rstd + row), w, aw,
                 ab, p1, p2);
    }
  }
  for (int which = 0; which < 2; ++which) {
    float* out = which == 0 ? a.pw : a.pb;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[warp][lane * 8 + 2 * j] = which == 0 ? aw[j].x : ab[j].x;
      red[warp][lane * 8 + 2 * j + 1] = which == 0 ? aw[j].y : ab[j].y;
    }
    __syncthreads();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (out != nullptr && c < a.d) {
      float s = 0.f;
      for (int k = 0; k < 8; ++k) s += red[k][threadIdx.x];
      out[static_cast<long long>(blockIdx.y) * a.d + c] = s;
    }
  }
}

// out (+)= sum over the n partial rows: a block takes 32 columns, 8 threads of 4 columns each by
// 32 groups of rows (group g: rows g, g + 32, ...), then the groups in order; blockIdx.y picks
// the weight's or the bias' gradient. d is a multiple of 8.
__global__ void __launch_bounds__(256) k_norm_dw_sum(const float* pw, const float* pb, int n, int d,
                                                     float* dweight, float* dbias, int accumulate) {
  __shared__ float4 red[32][8];
  after_previous();
  const float* p = blockIdx.y == 0 ? pw : pb;
  float* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const int c4 = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + c4 * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < d) {
#pragma unroll 8
    for (int k = g; k < n; k += 32) {
      // past L1: this kernel may have started before the partials were written
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p + static_cast<long long>(k) * d + col));
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  red[g][c4] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int c = blockIdx.x * 32 + threadIdx.x;
    if (c < d) {
      const float* q = reinterpret_cast<const float*>(&red[0][0]) + threadIdx.x;
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < 32; ++k) t += q[k * 32];
      out[c] = accumulate ? out[c] + t : t;
    }
  }
}

constexpr int kMaxShort = 128;
constexpr int kWideSplits = 32;
constexpr int kMaxBwd = 8192;           // longest row of the groups: 8 warps of 4 groups a lane

// The weight gradients take 16 registers per group of a lane: 2 groups, on as many warps as the row
// needs up to 8 (with 4 groups on half the warps 94 us instead of 82 us for 16,384 rows of 4,096,
// 50 us instead of 45 us at 2,048), then 3 and 4 groups, so that two rows are worked on at a time
// (16 warps of 2 groups, one row at a time: 181 us instead of 103 us for 16,384 rows of 5,120). One
// group needs few registers: 1,024 threads (262,144 rows of 256: 90 us, with 512 123 us).
template <class X, class Dy, class Dx, int NV, int WG, bool kMean>
cudaError_t bwd_rows(const X& x, const Dy& dy, const Dx& dx, const BwdArgs& a, int* parts, int sms,
                     cudaStream_t st) {
  constexpr int kThreads = NV == 1 ? 1024 : 512;
  auto kern = k_norm_bwd_rows<X, Dy, Dx, NV, WG, kThreads, kMean>;
  const size_t vec = sizeof(float) * static_cast<size_t>(a.d);
  const size_t slots = static_cast<size_t>(kSlots) * NV * WG * 32 * (X::kSlot + Dy::kSlot);
  const int per_sm = blocks_of(a.rows, sms);
  int groups = std::min<int>(kThreads / (WG * 32), (kSmemBytes - vec) / slots);
  groups = std::max(1, std::min(groups, per_sm));
  const size_t smem = vec + groups * std::max(slots, vec);   // the gradients meet in the slots
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  *parts = std::min(std::min(sms, norm_parts(a.d)), blocks_of(a.rows, groups));
  kern<<<*parts, groups * WG * 32, smem, st>>>(x, dy, dx, a);
  return cudaGetLastError();
}

template <class X, class Dy, class Dx, bool kMean>
cudaError_t bwd_by_length(const X& x, const Dy& dy, const Dx& dx, const BwdArgs& a, int* parts,
                          int sms, cudaStream_t st) {
  if (a.d <= 256) return bwd_rows<X, Dy, Dx, 1, 1, kMean>(x, dy, dx, a, parts, sms, st);
  if (a.d <= 512) return bwd_rows<X, Dy, Dx, 2, 1, kMean>(x, dy, dx, a, parts, sms, st);
  if (a.d <= 1024) return bwd_rows<X, Dy, Dx, 2, 2, kMean>(x, dy, dx, a, parts, sms, st);
  if (a.d <= 2048) return bwd_rows<X, Dy, Dx, 2, 4, kMean>(x, dy, dx, a, parts, sms, st);
  if (a.d <= 4096) return bwd_rows<X, Dy, Dx, 2, 8, kMean>(x, dy, dx, a, parts, sms, st);
  if (a.d <= 6144) return bwd_rows<X, Dy, Dx, 3, 8, kMean>(x, dy, dx, a, parts, sms, st);
  return bwd_rows<X, Dy, Dx, 4, 8, kMean>(x, dy, dx, a, parts, sms, st);
}

template <class X, class Dy, class Dx>
cudaError_t bwd_short(const X& x, const Dy& dy, const Dx& dx, const BwdArgs& a, int parts,
                      cudaStream_t st) {
  static_assert(kMaxShort <= 16 * 8, "rows of 16 lanes at most");
  switch (short_lanes(a.d)) {
    case 1: k_norm_bwd_short<X, Dy, Dx, 1><<<parts, kShortThreads, 0, st>>>(x, dy, dx, a); break;
    case 2: k_norm_bwd_short<X, Dy, Dx, 2><<<parts, kShortThreads, 0, st>>>(x, dy, dx, a); break;
    case 4: k_norm_bwd_short<X, Dy, Dx, 4><<<parts, kShortThreads, 0, st>>>(x, dy, dx, a); break;
    case 8: k_norm_bwd_short<X, Dy, Dx, 8><<<parts, kShortThreads, 0, st>>>(x, dy, dx, a); break;
    default: k_norm_bwd_short<X, Dy, Dx, 16><<<parts, kShortThreads, 0, st>>>(x, dy, dx, a); break;
  }
  return cudaGetLastError();
}

template <class X, class Dy, class Dx>
cudaError_t norm_bwd(const X& x, const Dy& dy, const Dx& dx, BwdArgs a, float* ws, float* dweight,
                     float* dbias, int accumulate, int sms, cudaStream_t st) {
  a.pw = dweight != nullptr ? ws : nullptr;
  a.pb = dbias != nullptr ? ws + static_cast<size_t>(norm_parts(a.d)) * a.d : nullptr;
  int parts;
  cudaError_t e;
  if (a.d > kMaxBwd) {
    parts = std::min(kWideSplits, a.rows);
    // the weight gradients first: dx may take dy's place
    if (a.pw != nullptr || a.pb != nullptr)
      k_norm_dw_wide<<<dim3((a.d + 255) / 256, parts), 256, 0, st>>>(x, dy, a);
    if (dx.p != nullptr) k_norm_dx_wide<<<a.rows, kWideThreads, 0, st>>>(x, dy, dx, a);
    e = cudaGetLastError();
  } else if (a.d <= kMaxShort) {
    const int rows_at_once = kShortThreads / short_lanes(a.d);
    parts = std::min(std::min(4 * sms, norm_parts(a.d)), blocks_of(a.rows, rows_at_once));
    e = bwd_short(x, dy, dx, a, parts, st);
  } else if (a.mean != nullptr) {
    e = bwd_by_length<X, Dy, Dx, true>(x, dy, dx, a, &parts, sms, st);
  } else {
    e = bwd_by_length<X, Dy, Dx, false>(x, dy, dx, a, &parts, sms, st);
  }
  if (e != cudaSuccess || (dweight == nullptr && dbias == nullptr)) return e;
  return launch_after(k_norm_dw_sum, dim3((a.d + 31) / 32, 2), 256, st, a.pw, a.pb, parts, a.d,
                      dweight, dbias, accumulate);
}

template <class X, class Dx>
cudaError_t norm_bwd_dy(const X& x, const NormGradBuf& g, const Dx& dx, const BwdArgs& a, int sms,
                        cudaStream_t st) {
  if (g.dy_bf16)
    return norm_bwd(x, RowsBf16{static_cast<const uint16_t*>(g.dy), g.dy_stride}, dx, a, g.ws,
                    g.dweight, g.dbias, g.accumulate, sms, st);
  return norm_bwd(x, RowsF32{static_cast<const float*>(g.dy), g.dy_stride}, dx, a, g.ws, g.dweight,
                  g.dbias, g.accumulate, sms, st);
}

}  // namespace

// One partial per SM; short rows take several blocks of 256 threads per SM.
int norm_parts(int d) { return d > kMaxBwd ? kWideSplits : d <= kMaxShort ? 4 * kPlanSms : kPlanSms; }

cudaError_t launch_norm_bwd(const NormIn& n, const NormGradBuf& g, int sms, cudaStream_t st) {
  const BwdArgs a{n.rows, n.d, n.wbf16, n.weight, g.mean, g.rstd, nullptr, nullptr};
  const OutBf16 db{static_cast<uint16_t*>(g.dx), g.dx_stride};
  const OutF32 df{static_cast<float*>(g.dx), g.dx_stride};
  if (n.codes != nullptr)
    return n.bf16 ? norm_bwd_dy(held_rows(n), g, db, a, sms, st)
                  : norm_bwd_dy(held_rows(n), g, df, a, sms, st);
  if (n.bf16)
    return norm_bwd_dy(RowsBf16{static_cast<const uint16_t*>(n.x), n.x_stride}, g, db, a, sms, st);
  return norm_bwd_dy(RowsF32{static_cast<const float*>(n.x), n.x_stride}, g, df, a, sms, st);
}

}  // namespace dpo
