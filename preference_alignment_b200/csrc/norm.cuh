// Shared by the norm's forward and backward kernels: row sums, weights, launch helpers.
#pragma once

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "rows8.cuh"

namespace dpo {

template <int kLanes = 32>
__device__ __forceinline__ float lanes_total(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float sum8(const float2 (&f)[4]) {
  const float2 s = __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3]));
  return s.x + s.y;
}
// f -= mu, and the sum of its squares
__device__ __forceinline__ float center8(float2 (&f)[4], float mu) {
  float2 q = both(0.f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = __fadd2_rn(f[j], both(-mu));
    q = __ffma2_rn(f[j], f[j], q);
  }
  return q.x + q.y;
}

// 8 values of the weight or bias (`none` when the pointer is NULL).
__device__ __forceinline__ void load_vec(const void* p, bool bf16, int col, float none,
                                         float2 (&f)[4]) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = both(none);
  } else if (bf16) {
    widen_bf16(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + col)), f);
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + col);
    RowsF32::widen(RowsF32::Raw{__ldg(q), __ldg(q + 1)}, f);
  }
}

// 8 fp32 values that stay in shared memory, in two planes of 16 bytes per group: lanes read
// neighbouring 16 bytes, so all banks serve them.
struct Planes {
  float4* p;       // [2][n]
  int n;           // groups
  __device__ __forceinline__ void store(int k, const float2 (&f)[4]) const {
    p[k] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    p[n + k] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
  __device__ __forceinline__ void load(int k, float2 (&f)[4]) const {
    RowsF32::widen(RowsF32::Raw{p[k], p[n + k]}, f);
  }
};

// ------------------------------------------------------------------ groups of warps
// Barrier of one group of the block's warps.
__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// Total over a group of WG warps, to every lane; `buf`: WG floats of the group, in turn.
template <int WG>
__device__ __forceinline__ float group_total(float x, float* buf, int group, int wg, int lane) {
  x = lanes_total(x);
  if constexpr (WG > 1) {
    if (lane == 0) buf[wg] = x;
    group_sync(group, WG * 32);
    x = buf[0];
#pragma unroll
    for (int k = 1; k < WG; ++k) x += buf[k];
  }
  return x;
}

// Sum over a block of up to 32 warps; every thread gets it. `buf` holds 32 floats and is free
// again after the next barrier.
__device__ __forceinline__ float block_total(float x, float* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  x = lanes_total(x);
  __syncthreads();
  if (lane == 0) buf[warp] = x;
  __syncthreads();
  return lanes_total(lane < warps ? buf[lane] : 0.f);
}

constexpr int kWideThreads = 512;
constexpr int kSmemBytes = 226 * 1024;    // dynamic shared memory a block may ask for

// Blocks of `each` rows (rows up to 2^31 - 1: the sum takes 64 bits).
inline int blocks_of(int rows, int each) {
  return static_cast<int>((static_cast<long long>(rows) + each - 1) / each);
}

inline int short_lanes(int d) {
  int g = 1;
  while (g * 8 < d) g *= 2;
  return g;
}

// Lets a kernel ask for `bytes` of dynamic shared memory. The limit is the kernel's, not the launch's: it
// is set to the most any length takes, so that a call of another thread in between cannot leave it
// below this launch's.
template <class Kern>
cudaError_t allow_smem(Kern kern, size_t bytes) {
  // 48 KiB without asking, static shared memory included
  return bytes > 40 * 1024
             ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)
             : cudaSuccess;
}

inline RowsQ8 held_rows(const NormIn& n) { return RowsQ8{n.codes, n.scales, n.d, q_blocks(n.d)}; }

}  // namespace dpo
