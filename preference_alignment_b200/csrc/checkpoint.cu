// 8-bit activation checkpoints: pack and unpack. Both only move bytes (pack reads 2 or 4
// bytes a value and writes 1 + 1/32; unpack the reverse), so HBM bounds them: 131,072 x 4,096 in
// bf16 is packed in 249 us and unpacked in 243 us (6.5 and 6.7 TB/s).
//
// A lane takes kPlaces groups of 8 values, all their loads under way at once; the scale of a
// block of 32 is found among 4 neighbouring lanes. How the groups are dealt out:
//   long rows   a warp takes `span` values of one row, 1,024 at a time
//   short rows  the rows are one line of places, 4 per block of 32 (a row's last block may leave
//               some empty), and a thread block takes its next kPlaces * kThreads: every lane has
//               work, at the price of two divisions per group (70 % of the copy rate)
// Pack of 262,144 rows of 256: 44 us in the line, 84 us by rows; of 512: 86 us and 112 us; 100,000
// rows of 1,000: 64 us and 58 us.
#include <climits>

#include "internal.h"
#include "rows8.cuh"

namespace dpo {

namespace {

constexpr int kThreads = 256;
constexpr int kPlaces = 4;      // per lane

constexpr int kWarps = kThreads / 32, kStep = kPlaces * 256;

// ------------------------------------------------------------------ long rows
// A block's warps take the same `span` columns of kWarps rows.
struct Span {
  long long row;
  int first, last;      // columns
  __device__ __forceinline__ Span(int d, int span) {
    const unsigned per_row = (d + span - 1) / span, b = blockIdx.x / per_row;
    row = static_cast<long long>(b) * kWarps + (threadIdx.x >> 5);
    first = static_cast<int>(blockIdx.x - b * per_row) * span;
    last = min(first + span, d);
  }
};

template <class Src>
__global__ void __launch_bounds__(kThreads) k_pack_rows(Src x, int rows, int d, int span,
                                                        int8_t* codes, uint8_t* scales) {
  const int lane = threadIdx.x & 31, blocks = q_blocks(d);
  const Span s(d, span);
  if (s.row >= rows) return;
  Held to(codes, scales, s.row, s.first + lane * 8, d, blocks);
  for (int c0 = s.first; c0 < s.last; c0 += kStep, to = to.right(kStep)) {
    typename Src::Raw raw[kPlaces];
#pragma unroll
    for (int u = 0; u < kPlaces; ++u) {
      const int col = c0 + (u * 32 + lane) * 8;
      if (col < s.last) raw[u] = x.load(s.row, col);
    }
#pragma unroll
    for (int u = 0; u < kPlaces; ++u) {
      const int col = c0 + (u * 32 + lane) * 8;
      float2 f[4] = {};
      if (col < s.last) Src::widen(raw[u], f);
      hold8(f, to.right(u * 256), col < s.last);
    }
  }
}

template <class Out>
__global__ void __launch_bounds__(kThreads) k_unpack_rows(RowsQ8 x, int rows, int d, int span, Out y) {
  const int lane = threadIdx.x & 31;
  const Span s(d, span);
  if (s.row >= rows) return;
  for (int c0 = s.first; c0 < s.last; c0 += kStep) {
    RowsQ8::Raw raw[kPlaces];
#pragma unroll
    for (int u = 0; u < kPlaces; ++u) {
      const int col = c0 + (u * 32 + lane) * 8;
      if (col < s.last) raw[u] = x.load(s.row, col);
    }
#pragma unroll
    for (int u = 0; u < kPlaces; ++u) {
      const int col = c0 + (u * 32 + lane) * 8;
      if (col < s.last) {
        float2 f[4];
        RowsQ8::widen(raw[u], f);
        y.store(s.row, col, f);
      }
    }
  }
}

// ------------------------------------------------------------------ short rows
struct Places {
  int rows, d, per_row;         // places of a row
  long long row0;
  uint32_t k0;
  __device__ __forceinline__ Places(int rows_, int d_) : rows(rows_), d(d_), per_row(4 * q_blocks(d_)) {
    const long long first = static_cast<long long>(blockIdx.x) * (kPlaces * kThreads);
    row0 = first / per_row;
    k0 = static_cast<uint32_t>(first - row0 * per_row) + threadIdx.x;
  }
  // The lane's u-th place; false where there is nothing.
  __device__ __forceinline__ bool at(int u, long long& row, int& col) const {
    const uint32_t k = k0 + u * kThreads, down = k / static_cast<uint32_t>(per_row);
    row = row0 + down;
    col = static_cast<int>(k - down * per_row) * 8;
    return row < rows && col < d;
  }
};

template <class Src>
__global__ void __launch_bounds__(kThreads) k_pack_line(Src x, int rows, int d, int8_t* codes,
                                                        uint8_t* scales) {
  const Places at(rows, d);
  const int blocks = q_blocks(d);
  typename Src::Raw raw[kPlaces];
  long long row;
  int col;
#pragma unroll
  for (int u = 0; u < kPlaces; ++u)
    if (at.at(u, row, col)) raw[u] = x.load(row, col);
#pragma unroll
  for (int u = 0; u < kPlaces; ++u) {
    const bool in = at.at(u, row, col);
    float2 f[4] = {};
    if (in) Src::widen(raw[u], f);
    hold8(f, Held(codes, scales, row, col, d, blocks), in);
  }
}

template <class Out>
__global__ void __launch_bounds__(kThreads) k_unpack_line(RowsQ8 x, int rows, int d, Out y) {
  const Places at(rows, d);
  RowsQ8::Raw raw[kPlaces];
  long long row;
  int col;
#pragma unroll
  for (int u = 0; u < kPlaces; ++u)
    if (at.at(u, row, col)) raw[u] = x.load(row, col);
#pragma unroll
  for (int u = 0; u < kPlaces; ++u) {
    if (at.at(u, row, col)) {
      float2 f[4];
      RowsQ8::widen(raw[u], f);
      y.store(row, col, f);
    }
  }
}

// ------------------------------------------------------------------ launches
constexpr int kLine = 512;                   // longest of the short rows
constexpr int kManyWarps = 148 * 32;         // warps that hide the loads' latency

struct Grid {
  long long blocks;
  int span;                                  // 0: short rows
};

Grid grid_of(int rows, int d) {
  if (d <= kLine) {
    const long long places = 4ll * q_blocks(d) * rows;
    return {(places + kPlaces * kThreads - 1) / (kPlaces * kThreads), 0};
  }
  // few rows: a warp takes less of one (512 x 16,384: 6.1 us, with whole rows 14.5 us)
  int span = 4 * kStep;
  while (span > kStep && static_cast<long long>(rows) * ((d + span - 1) / span) < kManyWarps)
    span -= kStep;
  return {static_cast<long long>((d + span - 1) / span) * ((static_cast<long long>(rows) + kWarps - 1) / kWarps), span};
}

template <class Src>
cudaError_t pack(const Src& x, int rows, int d, int8_t* codes, uint8_t* scales, cudaStream_t st) {
  const Grid g = grid_of(rows, d);
  if (g.blocks > INT_MAX) return cudaErrorInvalidValue;     // far more than memory holds
  const unsigned blocks = static_cast<unsigned>(g.blocks);
  if (g.span > 0)
    k_pack_rows<<<blocks, kThreads, 0, st>>>(x, rows, d, g.span, codes, scales);
  else
    k_pack_line<<<blocks, kThreads, 0, st>>>(x, rows, d, codes, scales);
  return cudaGetLastError();
}

template <class Out>
cudaError_t unpack(const RowsQ8& x, int rows, int d, const Out& y, cudaStream_t st) {
  const Grid g = grid_of(rows, d);
  if (g.blocks > INT_MAX) return cudaErrorInvalidValue;
  const unsigned blocks = static_cast<unsigned>(g.blocks);
  if (g.span > 0)
    k_unpack_rows<<<blocks, kThreads, 0, st>>>(x, rows, d, g.span, y);
  else
    k_unpack_line<<<blocks, kThreads, 0, st>>>(x, rows, d, y);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ckpt_pack(bool bf16, int rows, int d, const void* x, long long stride,
                             int8_t* codes, uint8_t* scales, cudaStream_t st) {
  if (bf16)
    return pack(RowsBf16{static_cast<const uint16_t*>(x), stride}, rows, d, codes, scales, st);
  return pack(RowsF32{static_cast<const float*>(x), stride}, rows, d, codes, scales, st);
}

cudaError_t launch_ckpt_unpack(bool bf16, int rows, int d, const int8_t* codes,
                               const uint8_t* scales, void* y, long long stride,
                               cudaStream_t st) {
  const RowsQ8 x{codes, scales, d, q_blocks(d)};
  if (bf16) return unpack(x, rows, d, OutBf16{static_cast<uint16_t*>(y), stride}, st);
  return unpack(x, rows, d, OutF32{static_cast<float*>(y), stride}, st);
}

}  // namespace dpo
