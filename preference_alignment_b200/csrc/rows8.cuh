// Rows of activations in groups of 8 values, as the norm and checkpoint kernels read and
// write them: bf16 (16 bytes), fp32 (32 bytes), or an 8-bit checkpoint (8 codes and the scale
// byte of their block of 32). A group is loaded raw, so that several loads can be in flight,
// and widened to fp32 (four pairs, for the packed fp32 instructions) when it is used.
//
// A source can also be fetched asynchronously (cp.async) into a slot of shared memory, kSlot
// bytes per group, so that the bytes in flight cost no registers. Group k of a row is taken by
// lane k mod 32 of the warp that fetched groups k - k mod 32 .. + 31; lanes copy for one another,
// so the warp synchronises between a copy's arrival and the takes, and between the takes and the
// next fetch into the slot. Every lane of the warp calls, with the row's number of groups.
#pragma once

#include <cstdint>

#include "ptx_sm100.cuh"

namespace dpo {

constexpr int kQBlock = 32;                     // values that share a scale (DPO_CHECKPOINT_BLOCK)

__host__ __device__ constexpr int q_blocks(int d) { return (d + kQBlock - 1) / kQBlock; }
// The block of a column (never negative: a shift).
__host__ __device__ constexpr int q_block_of(int col) {
  return static_cast<int>(static_cast<unsigned>(col) / kQBlock);
}

// ------------------------------------------------------------------ asynchronous copies
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Wait until at most N of this thread's committed groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// ------------------------------------------------------------------ widening
// bf16 -> fp32 moves the bits up 16 places.
__device__ __forceinline__ void widen_bf16(const uint4& r, float2 (&f)[4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    f[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}

// A scale byte as the power of two it stands for (255: NaN). Bytes are >= 1, so the power is
// a normal number.
__device__ __forceinline__ float q_scale(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(s << 23);
}

// Codes of -127..127 to fp32 without an integer conversion (a quarter-rate instruction): a code
// plus 128 put into the low mantissa bits of 2^23 reads 2^23 + 128 + code, exactly.
__device__ __forceinline__ void widen_codes(const uint2& r, float scale, float2 (&f)[4]) {
  const uint32_t w[2] = {r.x ^ 0x80808080u, r.y ^ 0x80808080u};
  const float2 off = make_float2(-8388736.f, -8388736.f), sc = make_float2(scale, scale);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t q = w[j / 2], k = 2 * (j % 2);
    const float2 u = make_float2(__uint_as_float(__byte_perm(q, 0x4b000000u, 0x7650u + k)),
                                 __uint_as_float(__byte_perm(q, 0x4b000000u, 0x7650u + k + 1)));
    f[j] = __fmul2_rn(__fadd2_rn(u, off), sc);
  }
}

// ------------------------------------------------------------------ sources
// `row` is the row's index, `col` the first of the group's columns.
struct RowsBf16 {
  const uint16_t* p;
  long long stride;
  static constexpr int kSlot = 16;
  struct Raw {
    uint4 v;
  };
  struct Side {};
  __device__ __forceinline__ Raw load(long long row, int col) const {
    return Raw{*reinterpret_cast<const uint4*>(p + row * stride + col)};
  }
  __device__ __forceinline__ void fetch(uint32_t slot, int k, int groups, long long row) const {
    if (k < groups) cp_async16(slot + k * 16, p + row * stride + k * 8);
  }
  __device__ __forceinline__ Side side(long long, int) const { return Side{}; }
  static __device__ __forceinline__ Raw take(uint32_t slot, int k, Side) {
    return Raw{ld_shared_v4(slot + k * 16)};
  }
  static __device__ __forceinline__ void widen(const Raw& r, float2 (&f)[4]) { widen_bf16(r.v, f); }
};

struct RowsF32 {
  const float* p;
  long long stride;
  static constexpr int kSlot = 32;
  struct Raw {
    float4 a, b;
  };
  struct Side {};
  __device__ __forceinline__ Raw load(long long row, int col) const {
    const float4* q = reinterpret_cast<const float4*>(p + row * stride + col);
    return Raw{q[0], q[1]};
  }
  // A warp's 32 groups are 64 chunks of 16 bytes. A copy of two chunks per lane side by side
  // would touch every 32-byte sector twice, half of it each time, and read twice the bytes from
  // L2 (129 us instead of 83 us for a backward of 16384 x 4096): lane l copies chunks l and 32 + l.
  // Chunk c lies at place c ^ (c / 8 mod 2), so that the takes of chunks 2 l and 2 l + 1 use all
  // banks.
  static __device__ __forceinline__ int place(int c) { return c ^ ((c >> 3) & 1); }
  __device__ __forceinline__ void fetch(uint32_t slot, int k, int groups, long long row) const {
    const int lane = k & 31, first = k - lane;
    const float* q = p + row * stride + first * 8;
    const int chunks = (groups - first) * 2;
    if (lane < chunks) cp_async16(slot + first * 32 + place(lane) * 16, q + lane * 4);
    if (lane + 32 < chunks)
      cp_async16(slot + first * 32 + place(lane + 32) * 16, q + (lane + 32) * 4);
  }
  __device__ __forceinline__ Side side(long long, int) const { return Side{}; }
  static __device__ __forceinline__ Raw take(uint32_t slot, int k, Side) {
    const int lane = k & 31;
    const uint32_t base = slot + (k - lane) * 32;
    const uint4 a = ld_shared_v4(base + place(2 * lane) * 16);
    const uint4 b = ld_shared_v4(base + place(2 * lane + 1) * 16);
    return Raw{make_float4(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z),
                           __uint_as_float(a.w)),
               make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z),
                           __uint_as_float(b.w))};
  }
  static __device__ __forceinline__ void widen(const Raw& r, float2 (&f)[4]) {
    f[0] = make_float2(r.a.x, r.a.y);
    f[1] = make_float2(r.a.z, r.a.w);
    f[2] = make_float2(r.b.x, r.b.y);
    f[3] = make_float2(r.b.z, r.b.w);
  }
};

struct RowsQ8 {
  const int8_t* codes;
  const uint8_t* scales;
  int d, blocks;
  static constexpr int kSlot = 8;
  struct Raw {
    uint2 v;
    uint32_t s;
  };
  using Side = uint32_t;                    // the scale byte, asked for ahead into a register
  __device__ __forceinline__ Raw load(long long row, int col) const {
    return Raw{*reinterpret_cast<const uint2*>(codes + row * d + col),
               scales[row * blocks + q_block_of(col)]};
  }
  __device__ __forceinline__ void fetch(uint32_t slot, int k, int groups, long long row) const {
    if (k < groups) cp_async8(slot + k * 8, codes + row * d + k * 8);
  }
  __device__ __forceinline__ Side side(long long row, int k) const {
    return __ldg(scales + row * blocks + q_block_of(k * 8));
  }
  static __device__ __forceinline__ Raw take(uint32_t slot, int k, Side s) {
    return Raw{ld_shared_v2(slot + k * 8), s};
  }
  static __device__ __forceinline__ void widen(const Raw& r, float2 (&f)[4]) {
    widen_codes(r.v, q_scale(r.s), f);
  }
};

struct OutBf16 {
  uint16_t* p;
  long long stride;
  __device__ __forceinline__ void store(long long row, int col, const float2 (&f)[4]) const {
    *reinterpret_cast<uint4*>(p + row * stride + col) =
        make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                   pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
  }
};

struct OutF32 {
  float* p;
  long long stride;
  __device__ __forceinline__ void store(long long row, int col, const float2 (&f)[4]) const {
    float4* q = reinterpret_cast<float4*>(p + row * stride + col);
    q[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    q[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
};

// Where a group of 8 goes in a checkpoint. Groups of one row that are a multiple of 32 columns
// apart are so many bytes apart: the addresses are worked out once (pack of 131,072 x 4,096: 246 us;
// worked out for each group 299 us).
struct Held {
  int8_t* code;
  uint8_t* scale;
  bool first;           // of its block: the one that writes the scale
  __device__ __forceinline__ Held(int8_t* codes, uint8_t* scales, long long row, int col, int d,
                                  int blocks)
      : code(codes + row * d + col),
        scale(scales + row * blocks + q_block_of(col)),
        first((col & (kQBlock - 1)) == 0) {}
  __device__ __forceinline__ Held(int8_t* c, uint8_t* s, bool f) : code(c), scale(s), first(f) {}
  // `cols` further on, a multiple of 32
  __device__ __forceinline__ Held right(int cols) const {
    return Held(code + cols, scale + cols / kQBlock, first);
  }
};

// Holds 8 values of a block of 32 that `share` (1, 2 or 4) neighbouring lanes have (every lane of
// the warp calls; lanes past the row's end pass zeros and `in` = false). The block's exponent
// comes from the largest magnitude's bits, so every step but the rounding of x * 2^-E is exact:
// max <= 127 * 2^E = 1.984375 * 2^(E + 6) holds for E = e - 6 when max = 1.f * 2^e with 1.f
// <= 1.984375, else for E = e - 5. NaN and infinity have the largest bits and mark the block.
// The rounding is the addition of 1.5 * 2^23: what is left of the sum's mantissa is the integer
// nearest to x * 2^-E, half to even, and its low byte the code.
__device__ __forceinline__ void hold8(const float2 (&f)[4], const Held& to, bool in,
                                      int share = 4) {
  uint32_t u = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    u = max(u, __float_as_uint(f[j].x) & 0x7fffffffu);
    u = max(u, __float_as_uint(f[j].y) & 0x7fffffffu);
  }
  if (share > 1) u = max(u, __shfl_xor_sync(0xffffffffu, u, 1));
  if (share > 2) u = max(u, __shfl_xor_sync(0xffffffffu, u, 2));
  if (!in) return;
  const int e = static_cast<int>(u >> 23);
  int s = e - ((u & 0x7fffffu) <= 0x7e0000u ? 6 : 5);      // E + 127
  s = min(max(s, 1), 248);                                  // 248: 127 * 2^E stays finite
  const bool bad = u >= 0x7f800000u;
  const float down = __uint_as_float(static_cast<uint32_t>(254 - s) << 23);   // 2^-E
  const float2 d2 = make_float2(down, down), magic = make_float2(12582912.f, 12582912.f);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 a = __fmul2_rn(f[2 * h], d2), b = __fmul2_rn(f[2 * h + 1], d2);
    if (s == 248) {                                         // only here can a value pass 127.5
      a.x = fminf(fmaxf(a.x, -127.f), 127.f);
      a.y = fminf(fmaxf(a.y, -127.f), 127.f);
      b.x = fminf(fmaxf(b.x, -127.f), 127.f);
      b.y = fminf(fmaxf(b.y, -127.f), 127.f);
    }
    a = __fadd2_rn(a, magic);
    b = __fadd2_rn(b, magic);
    const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    w[h] = bad ? 0u : __byte_perm(lo, hi, 0x5410);
  }
  *reinterpret_cast<uint2*>(to.code) = make_uint2(w[0], w[1]);
  if (to.first) *to.scale = bad ? 255 : s;
}

}  // namespace dpo
