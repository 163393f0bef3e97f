// The norm before the head, forward and backward (layer norm, and its rms form without the
// mean). Both only move bytes: the forward reads and writes each value once, the backward
// reads x and dy once and writes dx once, so HBM bounds them.
//
//   mu = mean x (rms: 0), r = 1 / sqrt(mean (x - mu)^2 + eps), xh = (x - mu) r
//   y  = xh w + b
//   dx = r (g - c1 - xh c2), g = dy w, c1 = mean g (rms: 0), c2 = mean(g xh)
//   dw = sum over rows of dy xh, db = sum over rows of dy
//
// The forward: 16,384 rows of 4,096 in bf16 take 45.7 us (5.9 TB/s; 48 to 50 in calls one after
// another), 65 us when they are held in 8 bits too. No unit is full (issue slots 49 % and the shared-memory pipe 66 % of the time, ncu): four warps
// per scheduler, all that its registers leave, do not cover the waits for shared memory (the slot, the
// weight and bias in fp32, the exchanges of the row sums), 2.9 of 8.1 cycles per instruction.
//
// Forms by the row's length d, each row read once except in the last:
//   d <= 256     a few lanes per row, one group of 8 values per lane (16,384 rows of 256: 5.1 us, a
//                warp per row 6.5 us; 262,144 rows: 68 us and 65 us)
//   d <= 16384   groups of 1 to 8 warps per row, the row in registers (4,096 rows of 16,384: 48 us)
//   above        a block per row that reads it again (from L2) instead of holding it (61 us there)
// The backward is in norm_bwd.cu.
#include "norm.cuh"

namespace dpo {

namespace {

struct FwdArgs {
  int rows, d, blocks, rms, wbf16;
  float eps;
  const void *weight, *bias;
  float *mean, *rstd;
  int8_t* codes;      // checkpoint to write, or NULL
  uint8_t* scales;
};

// f = f r w + b, f centred
__device__ __forceinline__ void normed(float2 (&f)[4], float r, const float2 (&w)[4],
                                       const float2 (&b)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = __ffma2_rn(__fmul2_rn(f[j], both(r)), w[j], b[j]);
}

// 1 / sqrt(v), v = spread / d + eps: the hardware's estimate (a few units off in the last place)
// and one Newton step, a sixth of the instructions of a rounded square root and division. The
// estimate stands where the step has no number to give (v = 0 or infinite).
__device__ __forceinline__ float rstd_of(float spread, float inv_d, float eps) {
  const float v = fmaf(spread, inv_d, eps);
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.f);
  return v > 1e-37f && v < 1e37f ? fmaf(0.5f * r, e, r) : r;
}

// ------------------------------------------------------------------ forward, short rows
// G lanes (a power of two) per row, 32 / G rows per warp.
template <class Src, class Out, int G>
__global__ void __launch_bounds__(256) k_norm_fwd_short(Src x, Out y, FwdArgs a) {
  const int lane = threadIdx.x & (G - 1);
  const long long row = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / G;
  const int col = lane * 8;
  const bool in = row < a.rows && col < a.d;
  float2 f[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
  if (in) Src::widen(x.load(row, col), f);
  if (a.codes != nullptr)
    hold8(f, Held(a.codes, a.scales, row, col, a.d, a.blocks), in, G < 4 ? G : 4);
  const float inv_d = 1.f / static_cast<float>(a.d);
  const float mu = a.rms ? 0.f : lanes_total<G>(sum8(f)) * inv_d;
  const float r = rstd_of(lanes_total<G>(in ? center8(f, mu) : 0.f), inv_d, a.eps);
  if (lane == 0 && in) {
    if (a.mean != nullptr) a.mean[row] = mu;
    if (a.rstd != nullptr) a.rstd[row] = r;
  }
  if (in) {
    float2 w[4], b[4];
    load_vec(a.weight, a.wbf16, col, 1.f, w);
    load_vec(a.bias, a.wbf16, col, 0.f, b);
    normed(f, r, w, b);
    y.store(row, col, f);
  }
}

// ------------------------------------------------------------------ forward, groups of warps
// WG warps per row (a group), NV groups of 8 values per lane, kept in registers as fp32 from the
// row's arrival to its output; weight and bias are widened once per block into shared memory.
// Groups walk over rows blockIdx.x * groups + group, + gridDim.x * groups, ...: while a row is
// worked on, the next one is on its way into the group's slot (cp.async), so the bytes in flight
// do not depend on how many warps the registers leave room for.
template <class Src, class Out, int NV, int WG, int kThreads>
__global__ void __launch_bounds__(kThreads) k_norm_fwd_rows(Src x, Out y, FwdArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];   // weight, bias [d] fp32; a slot per group
  __shared__ float red[2][kThreads / 32];
  constexpr int kLanes = WG * 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / WG, wg = warp % WG, groups = (blockDim.x >> 5) / WG;
  const int gl = wg * 32 + lane;                        // lane within the group
  const int vecs = a.d / 8;
  const Planes sw{reinterpret_cast<float4*>(smem_raw), vecs};
  const Planes sb{sw.p + 2 * vecs, vecs};
  const uint32_t slot = smem_u32(sb.p + 2 * vecs) + group * (NV * kLanes * Src::kSlot);
  const long long step = static_cast<long long>(gridDim.x) * groups;
  long long row = static_cast<long long>(blockIdx.x) * groups + group;
  typename Src::Side side[NV];
  auto fetch = [&](long long r) {
    if (r < a.rows) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        x.fetch(slot, u * kLanes + gl, vecs, r);
        if (u * kLanes + gl < vecs) side[u] = x.side(r, u * kLanes + gl);
      }
    }
    cp_async_commit();
  };
  fetch(row);
  for (int k = threadIdx.x; k < vecs; k += blockDim.x) {
    float2 f[4];
    load_vec(a.weight, a.wbf16, k * 8, 1.f, f);
    sw.store(k, f);
    load_vec(a.bias, a.wbf16, k * 8, 0.f, f);
    sb.store(k, f);
  }
  __syncthreads();
  const float inv_d = 1.f / static_cast<float>(a.d);
  int turn = 0;
  for (; row < a.rows; row += step) {
    cp_async_wait<0>();
    __syncwarp();
    float2 f[NV][4];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[u][j] = both(0.f);
      if (u * kLanes + gl < vecs) Src::widen(Src::take(slot, u * kLanes + gl, side[u]), f[u]);
    }
    __syncwarp();
    fetch(row + step);                                  // the slot is read: refill it
    if (a.codes != nullptr) {
      const Held to(a.codes, a.scales, row, gl * 8, a.d, a.blocks);
#pragma unroll
      for (int u = 0; u < NV; ++u)
        hold8(f[u], to.right(u * kLanes * 8), u * kLanes + gl < vecs);
    }
    float mu = 0.f;
    if (!a.rms) {
      float s = 0.f;
#pragma unroll
      for (int u = 0; u < NV; ++u) s += sum8(f[u]);
      mu = group_total<WG>(s, &red[turn][group * WG], group, wg, lane) * inv_d;
      turn ^= 1;
    }
    float q = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (u * kLanes + gl < vecs) q += center8(f[u], mu);
    const float r = rstd_of(group_total<WG>(q, &red[turn][group * WG], group, wg, lane), inv_d,
                            a.eps);
    turn ^= 1;
    if (gl == 0) {
      if (a.mean != nullptr) a.mean[row] = mu;
      if (a.rstd != nullptr) a.rstd[row] = r;
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int col = (u * kLanes + gl) * 8;
      if (col < a.d) {
        float2 w[4], b[4];
        sw.load(u * kLanes + gl, w);
        sb.load(u * kLanes + gl, b);
        normed(f[u], r, w, b);
        y.store(row, col, f[u]);
      }
    }
  }
}

// ------------------------------------------------------------------ forward, long rows
template <class Src, class Out>
__global__ void __launch_bounds__(kWideThreads) k_norm_fwd_wide(Src x, Out y, FwdArgs a) {
  __shared__ float buf[32];
  const long long row = blockIdx.x;
  const float inv_d = 1.f / static_cast<float>(a.d);
  float mu = 0.f;
  if (!a.rms) {
    float s = 0.f;
    for (int col = threadIdx.x * 8; col < a.d; col += kWideThreads * 8) {
      float2 f[4];
      Src::widen(x.load(row, col), f);
      s += sum8(f);
    }
    mu = block_total(s, buf) * inv_d;
  }
  float q = 0.f;
  for (int col = threadIdx.x * 8; col < a.d; col += kWideThreads * 8) {
    float2 f[4];
    Src::widen(x.load(row, col), f);
    q += center8(f, mu);
  }
  const float r = rstd_of(block_total(q, buf), inv_d, a.eps);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mu;
    if (a.rstd != nullptr) a.rstd[row] = r;
  }
  // whole warps take part in hold8's exchanges, also past the row's end
  for (int c0 = 0; c0 < a.d; c0 += kWideThreads * 8) {
    const int col = c0 + threadIdx.x * 8;
    const bool in = col < a.d;
    float2 f[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
    if (in) Src::widen(x.load(row, col), f);
    if (a.codes != nullptr) hold8(f, Held(a.codes, a.scales, row, col, a.d, a.blocks), in);
    if (in) {
      float2 w[4], b[4];
      load_vec(a.weight, a.wbf16, col, 1.f, w);
      load_vec(a.bias, a.wbf16, col, 0.f, b);
      center8(f, mu);
      normed(f, r, w, b);
      y.store(row, col, f);
    }
  }
}

constexpr int kMaxShortFwd = 256;       // longest row of the short form
constexpr int kMaxFwd = 16384;          // longest row of the groups: 8 warps of 8 groups a lane

// As many warps as registers allow (about 8 NV + 60 a thread), in one block per SM so that the
// weights are widened once; fewer where the rows do not fill them.
template <class Src, class Out, int NV, int WG>
cudaError_t fwd_rows(const Src& x, const Out& y, const FwdArgs& a, int sms, cudaStream_t st) {
  constexpr int kThreads = NV > 4 ? 512 : 768;
  auto kern = k_norm_fwd_rows<Src, Out, NV, WG, kThreads>;
  const size_t vec = 2 * sizeof(float) * static_cast<size_t>(a.d);
  const size_t slot = static_cast<size_t>(NV) * WG * 32 * Src::kSlot;
  const int per_sm = blocks_of(a.rows, sms);
  int groups = std::min<int>(kThreads / (WG * 32), (kSmemBytes - vec) / slot);
  groups = std::max(1, std::min(groups, per_sm));
  const size_t smem = vec + groups * slot;
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(sms, blocks_of(a.rows, groups));
  kern<<<grid, groups * WG * 32, smem, st>>>(x, y, a);
  return cudaGetLastError();
}

// Rows of more than kMin values. (2 and 8 warps take rows that 1 and 4 cannot hold: 5 groups a lane at
// least.)
template <class Src, class Out, int WG, int kMin>
cudaError_t fwd_by_length(const Src& x, const Out& y, const FwdArgs& a, int sms, cudaStream_t st) {
  const int nv = (a.d + WG * 256 - 1) / (WG * 256);
  if constexpr (kMin < 2 * WG * 256)
    if (nv <= 2) return fwd_rows<Src, Out, 2, WG>(x, y, a, sms, st);
  if constexpr (kMin < 4 * WG * 256)
    if (nv <= 4) return fwd_rows<Src, Out, 4, WG>(x, y, a, sms, st);
  if (nv <= 6) return fwd_rows<Src, Out, 6, WG>(x, y, a, sms, st);
  return fwd_rows<Src, Out, 8, WG>(x, y, a, sms, st);
}

template <class Src, class Out>
cudaError_t norm_fwd(const Src& x, const Out& y, const FwdArgs& a, int sms, cudaStream_t st) {
  if (a.d <= kMaxShortFwd) {
    const int g = short_lanes(a.d);
    const int grid = static_cast<int>((static_cast<long long>(a.rows) * g + 255) / 256);
    switch (g) {
      case 1: k_norm_fwd_short<Src, Out, 1><<<grid, 256, 0, st>>>(x, y, a); break;
      case 2: k_norm_fwd_short<Src, Out, 2><<<grid, 256, 0, st>>>(x, y, a); break;
      case 4: k_norm_fwd_short<Src, Out, 4><<<grid, 256, 0, st>>>(x, y, a); break;
      case 8: k_norm_fwd_short<Src, Out, 8><<<grid, 256, 0, st>>>(x, y, a); break;
      case 16: k_norm_fwd_short<Src, Out, 16><<<grid, 256, 0, st>>>(x, y, a); break;
      default: k_norm_fwd_short<Src, Out, 32><<<grid, 256, 0, st>>>(x, y, a); break;
    }
    return cudaGetLastError();
  }
  if (a.d > kMaxFwd) {
    k_norm_fwd_wide<<<a.rows, kWideThreads, 0, st>>>(x, y, a);
    return cudaGetLastError();
  }
  // the fewest warps per row that leave a lane 8 groups (a row of 4,096 on one warp of 16 groups a
  // lane: 51 us instead of 47 us for 16,384 rows, on four warps of 4: 47.5 us; at 2,048 one warp 27
  // us, four 31 us); 4 where there are fewer rows than SMs, so that a row's latency is spread
  if (a.d > 8192) return fwd_by_length<Src, Out, 8, 8192>(x, y, a, sms, st);
  if (a.d > 4096 || a.rows <= sms) return fwd_by_length<Src, Out, 4, kMaxShortFwd>(x, y, a, sms, st);
  if (a.d > 2048) return fwd_by_length<Src, Out, 2, 2048>(x, y, a, sms, st);
  return fwd_by_length<Src, Out, 1, kMaxShortFwd>(x, y, a, sms, st);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormIn& n, void* y, long long y_stride, float* mean, float* rstd,
                            int8_t* codes, uint8_t* scales, int sms, cudaStream_t st) {
  const FwdArgs a{n.rows, n.d, q_blocks(n.d), n.rms, n.wbf16, n.eps, n.weight, n.bias,
                  mean, rstd, codes, scales};
  const OutBf16 yb{static_cast<uint16_t*>(y), y_stride};
  const OutF32 yf{static_cast<float*>(y), y_stride};
  if (n.codes != nullptr)
    return n.bf16 ? norm_fwd(held_rows(n), yb, a, sms, st) : norm_fwd(held_rows(n), yf, a, sms, st);
  if (n.bf16)
    return norm_fwd(RowsBf16{static_cast<const uint16_t*>(n.x), n.x_stride}, yb, a, sms, st);
  return norm_fwd(RowsF32{static_cast<const float*>(n.x), n.x_stride}, yf, a, sms, st);
}

}  // namespace dpo
