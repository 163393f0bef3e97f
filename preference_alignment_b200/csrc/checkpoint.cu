// 8-bit activation checkpoints: pack and unpack. Both only move bytes (pack reads 2 or 4
// bytes a value and writes 1 + 1/32; unpack the reverse), so HBM bounds them. A warp takes a
// row's 32 groups of 8 values at a time, several such steps in flight.
#include "internal.h"
#include "rows8.cuh"

namespace dpo {

namespace {

constexpr int kCkWarps = 8;
constexpr int kCkSteps = 4;     // groups in flight per lane

template <class Src>
__global__ void __launch_bounds__(kCkWarps * 32) k_ckpt_pack(Src x, int rows, int d, int blocks,
                                                             int8_t* codes, uint8_t* scales) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kCkWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  for (int c0 = 0; c0 < d; c0 += kCkSteps * 256) {
    typename Src::Raw raw[kCkSteps];
#pragma unroll
    for (int u = 0; u < kCkSteps; ++u) {
      const int col = c0 + (u * 32 + lane) * 8;
      if (col < d) raw[u] = x.load(row, col);
    }
#pragma unroll
    for (int u = 0; u < kCkSteps; ++u) {
      const int col = c0 + (u * 32 + lane) * 8;
      float2 f[4] = {};
      if (col < d) Src::widen(raw[u], f);
      hold8(f, codes, scales, row, col, d, blocks, col < d);
    }
  }
}

template <class Out>
__global__ void __launch_bounds__(kCkWarps * 32) k_ckpt_unpack(RowsQ8 x, int rows, int d, Out y) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kCkWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  for (int c0 = 0; c0 < d; c0 += kCkSteps * 256) {
    RowsQ8::Raw raw[kCkSteps];
#pragma unroll
    for (int u = 0; u < kCkSteps; ++u) {
      const int col = c0 + (u * 32 + lane) * 8;
      if (col < d) raw[u] = x.load(row, col);
    }
#pragma unroll
    for (int u = 0; u < kCkSteps; ++u) {
      const int col = c0 + (u * 32 + lane) * 8;
      if (col < d) {
        float2 f[4];
        RowsQ8::widen(raw[u], f);
        y.store(row, col, f);
      }
    }
  }
}

}  // namespace

cudaError_t launch_ckpt_pack(bool bf16, int rows, int d, const void* x, long long stride,
                             int8_t* codes, uint8_t* scales, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int grid = (rows + kCkWarps - 1) / kCkWarps, nb = q_blocks(d);
  if (bf16)
    k_ckpt_pack<<<grid, kCkWarps * 32, 0, st>>>(
        RowsBf16{static_cast<const uint16_t*>(x), stride}, rows, d, nb, codes, scales);
  else
    k_ckpt_pack<<<grid, kCkWarps * 32, 0, st>>>(RowsF32{static_cast<const float*>(x), stride},
                                                rows, d, nb, codes, scales);
  return cudaGetLastError();
}

cudaError_t launch_ckpt_unpack(bool bf16, int rows, int d, const int8_t* codes,
                               const uint8_t* scales, void* y, long long stride,
                               cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int grid = (rows + kCkWarps - 1) / kCkWarps;
  const RowsQ8 x{codes, scales, d, q_blocks(d)};
  if (bf16)
    k_ckpt_unpack<<<grid, kCkWarps * 32, 0, st>>>(x, rows, d,
                                                  OutBf16{static_cast<uint16_t*>(y), stride});
  else
    k_ckpt_unpack<<<grid, kCkWarps * 32, 0, st>>>(x, rows, d,
                                                  OutF32{static_cast<float*>(y), stride});
  return cudaGetLastError();
}

}  // namespace dpo
