// The norm before the head, forward and backward (layer norm, and its rms form without the
// mean). Both only move bytes: the forward reads and writes each value once, the backward
// reads x and dy once and writes dx once, so HBM bounds them.
//
//   mu = mean x (rms: 0), r = 1 / sqrt(mean (x - mu)^2 + eps), xh = (x - mu) r
//   y  = xh w + b
//   dx = r (g - c1 - xh c2), g = dy w, c1 = mean g (rms: 0), c2 = mean(g xh)
//   dw = sum over rows of dy xh, db = sum over rows of dy
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "rows8.cuh"

namespace dpo {

namespace {

__device__ __forceinline__ float warp_total(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// 8 values of the weight or bias (`none` when the pointer is NULL).
__device__ __forceinline__ void load_vec(const void* p, bool bf16, int col, float none,
                                         float (&f)[8]) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = none;
  } else if (bf16) {
    widen_bf16(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + col)), f);
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + col);
    const float4 a = __ldg(q), b = __ldg(q + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

struct FwdArgs {
  int rows, d, blocks, rms, wbf16;
  float eps;
  const void *weight, *bias;
  float *mean, *rstd;
  int8_t* codes;      // checkpoint to write, or NULL
  uint8_t* scales;
};

// ------------------------------------------------------------------ forward
// One warp per row, the row in registers (NV groups of 8 per lane): one read of x, both
// reductions by shuffles, no barrier.
template <class Src, class Out, int NV>
__global__ void __launch_bounds__(256) k_norm_fwd(Src x, Out y, FwdArgs a) {
  const int lane = threadIdx.x & 31;
  const long long row =
      static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  typename Src::Raw raw[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int col = (u * 32 + lane) * 8;
    if (col < a.d) raw[u] = x.load(row, col);
  }
  const float inv_d = 1.f / static_cast<float>(a.d);
  float mu = 0.f;
  if (!a.rms) {
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if ((u * 32 + lane) * 8 < a.d) {
        float f[8];
        Src::widen(raw[u], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) s += f[j];
      }
    }
    mu = warp_total(s) * inv_d;
  }
  float q = 0.f;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    if ((u * 32 + lane) * 8 < a.d) {
      float f[8];
      Src::widen(raw[u], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) q = fmaf(f[j] - mu, f[j] - mu, q);
    }
  }
  const float r = 1.f / sqrtf(warp_total(q) * inv_d + a.eps);
  if (lane == 0) {
    if (a.mean != nullptr) a.mean[row] = mu;
    if (a.rstd != nullptr) a.rstd[row] = r;
  }
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int col = (u * 32 + lane) * 8;
    const bool in = col < a.d;
    float f[8] = {};
    if (in) Src::widen(raw[u], f);
    if (a.codes != nullptr) hold8(f, a.codes, a.scales, row, col, a.d, a.blocks, in);
    if (in) {
      float w[8], b[8];
      load_vec(a.weight, a.wbf16, col, 1.f, w);
      load_vec(a.bias, a.wbf16, col, 0.f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf((f[j] - mu) * r, w[j], b[j]);
      y.store(row, col, f);
    }
  }
}

// Sum over a block of up to 32 warps; every thread gets it. `buf` holds 32 floats and is free
// again after the next barrier.
__device__ __forceinline__ float block_total(float x, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  x = warp_total(x);
  __syncthreads();
  if (lane == 0) buf[warp] = x;
  __syncthreads();
  return warp_total(lane < warps ? buf[lane] : 0.f);
}

// Rows too long for a warp's registers: one block per row reads it three times (the second
// and third from L2).
constexpr int kWideThreads = 512;

template <class Src, class Out>
__global__ void __launch_bounds__(kWideThreads) k_norm_fwd_wide(Src x, Out y, FwdArgs a) {
  __shared__ float buf[32];
  const long long row = blockIdx.x;
  const float inv_d = 1.f / static_cast<float>(a.d);
  float mu = 0.f;
  if (!a.rms) {
    float s = 0.f;
    for (int col = threadIdx.x * 8; col < a.d; col += kWideThreads * 8) {
      float f[8];
      Src::widen(x.load(row, col), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += f[j];
    }
    mu = block_total(s, buf) * inv_d;
  }
  float q = 0.f;
  for (int col = threadIdx.x * 8; col < a.d; col += kWideThreads * 8) {
    float f[8];
    Src::widen(x.load(row, col), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) q = fmaf(f[j] - mu, f[j] - mu, q);
  }
  const float r = 1.f / sqrtf(block_total(q, buf) * inv_d + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mu;
    if (a.rstd != nullptr) a.rstd[row] = r;
  }
  // whole warps take part in hold8's shuffles, also past the row's end
  for (int c0 = 0; c0 < a.d; c0 += kWideThreads * 8) {
    const int col = c0 + threadIdx.x * 8;
    const bool in = col < a.d;
    float f[8] = {};
    if (in) Src::widen(x.load(row, col), f);
    if (a.codes != nullptr) hold8(f, a.codes, a.scales, row, col, a.d, a.blocks, in);
    if (in) {
      float w[8], b[8];
      load_vec(a.weight, a.wbf16, col, 1.f, w);
      load_vec(a.bias, a.wbf16, col, 0.f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf((f[j] - mu) * r, w[j], b[j]);
      y.store(row, col, f);
    }
  }
}

template <class Src, class Out>
cudaError_t norm_fwd(const Src& x, const Out& y, const FwdArgs& a, cudaStream_t st) {
  // a row's raw groups have to leave room in a thread's 255 registers: 16 groups of fp32 (128
  // registers), 32 of the narrower forms
  constexpr int kMaxNV = sizeof(typename Src::Raw) > 16 ? 16 : 32;
  const int groups = (a.d / 8 + 31) / 32;
  if (groups > kMaxNV) {
    k_norm_fwd_wide<<<a.rows, kWideThreads, 0, st>>>(x, y, a);
    return cudaGetLastError();
  }
  const int warps = 4;
  const int grid = (a.rows + warps - 1) / warps;
  if (groups <= 1)
    k_norm_fwd<Src, Out, 1><<<grid, warps * 32, 0, st>>>(x, y, a);
  else if (groups <= 2)
    k_norm_fwd<Src, Out, 2><<<grid, warps * 32, 0, st>>>(x, y, a);
  else if (groups <= 4)
    k_norm_fwd<Src, Out, 4><<<grid, warps * 32, 0, st>>>(x, y, a);
  else if (groups <= 8)
    k_norm_fwd<Src, Out, 8><<<grid, warps * 32, 0, st>>>(x, y, a);
  else if (groups <= 16)
    k_norm_fwd<Src, Out, 16><<<grid, warps * 32, 0, st>>>(x, y, a);
  else
    k_norm_fwd<Src, Out, kMaxNV><<<grid, warps * 32, 0, st>>>(x, y, a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ backward
struct BwdArgs {
  int rows, d, wbf16;
  const void* weight;
  const float *mean, *rstd;     // mean NULL: rms
  float *pw, *pb;               // [gridDim.x, d] partial weight gradients, or NULL
};

// A block takes rows blockIdx.x, blockIdx.x + gridDim.x, ... and thread t the columns of its
// NV groups in every one of them, so the weight gradients gather in registers; the next row's
// loads are issued before the current row's sums are joined.
template <class X, class Dy, class Dx, int NV, int kThreads>
__global__ void __launch_bounds__(kThreads) k_norm_bwd(X x, Dy dy, Dx dx, BwdArgs a) {
  __shared__ float2 red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const float inv_d = 1.f / static_cast<float>(a.d);
  float w[NV][8], aw[NV][8], ab[NV][8];
  int col[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    col[u] = (u * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[u][j] = aw[u][j] = ab[u][j] = 0.f;
    if (col[u] < a.d) load_vec(a.weight, a.wbf16, col[u], 1.f, w[u]);
  }
  typename X::Raw rx[NV];
  typename Dy::Raw rd[NV];
  float mu = 0.f, r = 0.f;
  auto fetch = [&](long long row) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (col[u] < a.d) {
        rx[u] = x.load(row, col[u]);
        rd[u] = dy.load(row, col[u]);
      }
    }
    mu = a.mean != nullptr ? __ldg(a.mean + row) : 0.f;
    r = __ldg(a.rstd + row);
  };
  int it = 0;
  if (static_cast<int>(blockIdx.x) < a.rows) fetch(blockIdx.x);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, ++it) {
    float g[NV][8], xh[NV][8];
    float c1 = 0.f, c2 = 0.f;
    const float rr = r;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[u][j] = xh[u][j] = 0.f;
      if (col[u] < a.d) {
        X::widen(rx[u], xh[u]);
        Dy::widen(rd[u], g[u]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float h = (xh[u][j] - mu) * r, e = g[u][j];
          xh[u][j] = h;
          aw[u][j] = fmaf(e, h, aw[u][j]);
          ab[u][j] += e;
          g[u][j] = e * w[u][j];
          c1 += g[u][j];
          c2 = fmaf(g[u][j], h, c2);
        }
      }
    }
    if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
    c1 = warp_total(c1);
    c2 = warp_total(c2);
    // two buffers: a warp may write the next row's sums while another still reads this row's
    float2* b = red[it & 1];
    if (lane == 0) b[warp] = make_float2(c1, c2);
    __syncthreads();
    const float2 q = lane < warps ? b[lane] : make_float2(0.f, 0.f);
    c1 = a.mean != nullptr ? warp_total(q.x) * inv_d : 0.f;
    c2 = warp_total(q.y) * inv_d;
    if (dx.p != nullptr) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        if (col[u] < a.d) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = rr * (g[u][j] - c1 - xh[u][j] * c2);
          dx.store(row, col[u], f);
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    if (col[u] < a.d) {
      if (a.pw != nullptr) OutF32{a.pw, a.d}.store(blockIdx.x, col[u], aw[u]);
      if (a.pb != nullptr) OutF32{a.pb, a.d}.store(blockIdx.x, col[u], ab[u]);
    }
  }
}

// Rows too long for the above: dx with one block per row and two readings of it, and the
// weight gradients over slabs of 256 columns and splits of the rows.
template <class X, class Dy, class Dx>
__global__ void __launch_bounds__(kWideThreads) k_norm_dx_wide(X x, Dy dy, Dx dx, BwdArgs a) {
  __shared__ float buf[32];
  const long long row = blockIdx.x;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const float mu = a.mean != nullptr ? __ldg(a.mean + row) : 0.f, r = __ldg(a.rstd + row);
  float c1 = 0.f, c2 = 0.f;
  for (int col = threadIdx.x * 8; col < a.d; col += kWideThreads * 8) {
    float f[8], e[8], w[8];
    X::widen(x.load(row, col), f);
    Dy::widen(dy.load(row, col), e);
    load_vec(a.weight, a.wbf16, col, 1.f, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c1 = fmaf(e[j], w[j], c1);
      c2 = fmaf(e[j] * w[j], (f[j] - mu) * r, c2);
    }
  }
  c1 = block_total(c1, buf) * inv_d;
  c2 = block_total(c2, buf) * inv_d;
  if (a.mean == nullptr) c1 = 0.f;
  for (int col = threadIdx.x * 8; col < a.d; col += kWideThreads * 8) {
    float f[8], e[8], w[8];
    X::widen(x.load(row, col), f);
    Dy::widen(dy.load(row, col), e);
    load_vec(a.weight, a.wbf16, col, 1.f, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = r * (e[j] * w[j] - c1 - (f[j] - mu) * r * c2);
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
  float aw[8] = {}, ab[8] = {};
  if (col < a.d) {
    for (long long row = r0 + warp; row < r1; row += 8) {
      float f[8], e[8];
      X::widen(x.load(row, col), f);
      Dy::widen(dy.load(row, col), e);
      const float mu = a.mean != nullptr ? __ldg(a.mean + row) : 0.f, r = __ldg(a.rstd + row);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        aw[j] = fmaf(e[j], (f[j] - mu) * r, aw[j]);
        ab[j] += e[j];
      }
    }
  }
  for (int which = 0; which < 2; ++which) {
    float* out = which == 0 ? a.pw : a.pb;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) red[warp][lane * 8 + j] = which == 0 ? aw[j] : ab[j];
    __syncthreads();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (out != nullptr && c < a.d) {
      float s = 0.f;
      for (int k = 0; k < 8; ++k) s += red[k][threadIdx.x];
      out[static_cast<long long>(blockIdx.y) * a.d + c] = s;
    }
  }
}

// out (+)= sum over the n partial rows: a block takes 32 columns, warp w rows w, w + 8, ...;
// blockIdx.y picks the weight's or the bias' gradient.
__global__ void __launch_bounds__(256) k_norm_dw_sum(const float* pw, const float* pb, int n, int d,
                                                     float* dweight, float* dbias, int accumulate) {
  __shared__ float red[8][32];
  const float* p = blockIdx.y == 0 ? pw : pb;
  float* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d)
    for (int k = warp; k < n; k += 8) s += __ldg(p + static_cast<long long>(k) * d + c);
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < d) {
    for (int k = 1; k < 8; ++k) s += red[k][lane];
    out[c] = accumulate ? out[c] + s : s;
  }
}

constexpr int kMaxBwdThreads = 1024;
constexpr int kWideSplits = 32;

template <class X, class Dy, class Dx>
cudaError_t norm_bwd(const X& x, const Dy& dy, const Dx& dx, BwdArgs a, float* ws, float* dweight,
                     float* dbias, int accumulate, int sms, cudaStream_t st) {
  const int groups = a.d / 8;
  const bool wide = groups > kMaxBwdThreads;
  const int parts = wide ? std::min(a.rows, kWideSplits) : std::min(a.rows, std::min(2 * sms, kNormParts));
  a.pw = dweight != nullptr ? ws : nullptr;
  a.pb = dbias != nullptr ? ws + static_cast<size_t>(kNormParts) * a.d : nullptr;
  if (wide) {
    // the weight gradients first: dx may take dy's place
    if (a.pw != nullptr || a.pb != nullptr)
      k_norm_dw_wide<<<dim3((a.d + 255) / 256, parts), 256, 0, st>>>(x, dy, a);
    if (dx.p != nullptr) k_norm_dx_wide<<<a.rows, kWideThreads, 0, st>>>(x, dy, dx, a);
  } else {
    const int threads = (groups + 31) / 32 * 32;
    if (threads <= 512)
      k_norm_bwd<X, Dy, Dx, 1, 512><<<parts, threads, 0, st>>>(x, dy, dx, a);
    else
      k_norm_bwd<X, Dy, Dx, 1, 1024><<<parts, threads, 0, st>>>(x, dy, dx, a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (dweight == nullptr && dbias == nullptr)) return e;
  k_norm_dw_sum<<<dim3((a.d + 31) / 32, 2), 256, 0, st>>>(a.pw, a.pb, parts, a.d, dweight, dbias,
                                                          accumulate);
  return cudaGetLastError();
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

cudaError_t launch_norm_fwd(const NormIn& n, void* y, long long y_stride, float* mean, float* rstd,
                            int8_t* codes, uint8_t* scales, cudaStream_t st) {
  const FwdArgs a{n.rows, n.d, q_blocks(n.d), n.rms, n.wbf16, n.eps, n.weight, n.bias,
                  mean, rstd, codes, scales};
  const OutBf16 yb{static_cast<uint16_t*>(y), y_stride};
  const OutF32 yf{static_cast<float*>(y), y_stride};
  if (n.codes != nullptr) {
    const RowsQ8 x{n.codes, n.scales, n.d, q_blocks(n.d)};
    return n.bf16 ? norm_fwd(x, yb, a, st) : norm_fwd(x, yf, a, st);
  }
  if (n.bf16) return norm_fwd(RowsBf16{static_cast<const uint16_t*>(n.x), n.x_stride}, yb, a, st);
  return norm_fwd(RowsF32{static_cast<const float*>(n.x), n.x_stride}, yf, a, st);
}

cudaError_t launch_norm_bwd(const NormIn& n, const NormGradBuf& g, int sms, cudaStream_t st) {
  const BwdArgs a{n.rows, n.d, n.wbf16, n.weight, g.mean, g.rstd, nullptr, nullptr};
  const OutBf16 db{static_cast<uint16_t*>(g.dx), g.dx_stride};
  const OutF32 df{static_cast<float*>(g.dx), g.dx_stride};
  if (n.codes != nullptr) {
    const RowsQ8 x{n.codes, n.scales, n.d, q_blocks(n.d)};
    return n.bf16 ? norm_bwd_dy(x, g, db, a, sms, st) : norm_bwd_dy(x, g, df, a, sms, st);
  }
  if (n.bf16)
    return norm_bwd_dy(RowsBf16{static_cast<const uint16_t*>(n.x), n.x_stride}, g, db, a, sms, st);
  return norm_bwd_dy(RowsF32{static_cast<const float*>(n.x), n.x_stride}, g, df, a, sms, st);
}

}  // namespace dpo
