// Rows of activations in groups of 8 values, as the norm and checkpoint kernels read and
// write them: bf16 (16 bytes), fp32 (32 bytes), or an 8-bit checkpoint (8 codes and the scale
// byte of their block of 32). A group is loaded raw, so that several loads can be in flight,
// and widened to fp32 when it is used.
#pragma once

#include <cstdint>

#include "ptx_sm100.cuh"

namespace dpo {

constexpr int kQBlock = 32;                     // values that share a scale (DPO_CHECKPOINT_BLOCK)

__host__ __device__ constexpr int q_blocks(int d) { return (d + kQBlock - 1) / kQBlock; }

// bf16 -> fp32 moves the bits up 16 places.
__device__ __forceinline__ void widen_bf16(const uint4& r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}

// A scale byte as the power of two it stands for (255: NaN). Bytes are >= 1, so the power is
// a normal number.
__device__ __forceinline__ float q_scale(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(s << 23);
}

// Sources and destinations. `row` is the row's index, `col` the first of the group's columns.
struct RowsBf16 {
  const uint16_t* p;
  long long stride;
  struct Raw {
    uint4 v;
  };
  __device__ __forceinline__ Raw load(long long row, int col) const {
    return Raw{*reinterpret_cast<const uint4*>(p + row * stride + col)};
  }
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[8]) { widen_bf16(r.v, f); }
};

struct RowsF32 {
  const float* p;
  long long stride;
  struct Raw {
    float4 a, b;
  };
  __device__ __forceinline__ Raw load(long long row, int col) const {
    const float4* q = reinterpret_cast<const float4*>(p + row * stride + col);
    return Raw{q[0], q[1]};
  }
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[8]) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
  }
};

struct RowsQ8 {
  const int8_t* codes;
  const uint8_t* scales;
  int d, blocks;
  struct Raw {
    uint2 v;
    uint32_t s;
  };
  __device__ __forceinline__ Raw load(long long row, int col) const {
    return Raw{*reinterpret_cast<const uint2*>(codes + row * d + col),
               scales[row * blocks + col / kQBlock]};
  }
  static __device__ __forceinline__ void widen(const Raw& r, float (&f)[8]) {
    const float s = q_scale(r.s);
    const uint32_t w[2] = {r.v.x, r.v.y};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      f[j] = static_cast<float>(static_cast<int8_t>(w[j / 4] >> (8 * (j % 4)))) * s;
  }
};

struct OutBf16 {
  uint16_t* p;
  long long stride;
  __device__ __forceinline__ void store(long long row, int col, const float (&f)[8]) const {
    *reinterpret_cast<uint4*>(p + row * stride + col) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
};

struct OutF32 {
  float* p;
  long long stride;
  __device__ __forceinline__ void store(long long row, int col, const float (&f)[8]) const {
    float4* q = reinterpret_cast<float4*>(p + row * stride + col);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// Holds 8 values of a block of 32 that 4 neighbouring lanes share (every lane of the warp
// calls; lanes past the row's end pass zeros and `in` = false). The block's exponent comes
// from the largest magnitude's bits, so every step but the rounding of x * 2^-E is exact:
// max <= 127 * 2^E = 1.984375 * 2^(E + 6) holds for E = e - 6 when max = 1.f * 2^e with 1.f
// <= 1.984375, else for E = e - 5. NaN and infinity have the largest bits and mark the block.
__device__ __forceinline__ void hold8(const float (&f)[8], int8_t* codes, uint8_t* scales,
                                      long long row, int col, int d, int blocks, bool in) {
  uint32_t u = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) u = max(u, __float_as_uint(f[j]) & 0x7fffffffu);
  u = max(u, __shfl_xor_sync(0xffffffffu, u, 1));
  u = max(u, __shfl_xor_sync(0xffffffffu, u, 2));
  if (!in) return;
  const int e = static_cast<int>(u >> 23);
  int s = e - ((u & 0x7fffffu) <= 0x7e0000u ? 6 : 5);      // E + 127
  s = min(max(s, 1), 248);                                  // 248: 127 * 2^E stays finite
  const bool bad = u >= 0x7f800000u;
  const float down = __uint_as_float(static_cast<uint32_t>(254 - s) << 23);   // 2^-E
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = bad ? 0 : min(max(__float2int_rn(f[j] * down), -127), 127);
    w[j / 4] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (j % 4));
  }
  *reinterpret_cast<uint2*>(codes + row * d + col) = make_uint2(w[0], w[1]);
  if (col % kQBlock == 0) scales[row * blocks + col / kQBlock] = bad ? 255 : s;
}

}  // namespace dpo
