// Shared by the token statistics kernels: joining sums of tiles, and lists of the largest logits
// spread over a warp.
#pragma once

#include <cmath>
#include <cstdint>

#include "internal.h"

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

// Rounding can leave an entropy of 0 a little below it (NaN stays NaN).
__device__ __forceinline__ float entropy_of(float e) { return e < 0.f ? 0.f : e; }

// ------------------------------------------------------------------ lists across a warp
// A falling list of 32 (logit, id) entries, entry j in lane j.
struct Entry {
  float v;
  int id;
};

__device__ __forceinline__ bool ahead(const Entry& a, const Entry& b) {
  return a.v > b.v || (a.v == b.v && a.id < b.id);
}

// Puts x into a falling list (entry j in lane j), behind every entry ahead of it.
__device__ __forceinline__ void insert_entry(Entry& list, const Entry& x, int lane) {
  const int at = __popc(__ballot_sync(0xffffffffu, ahead(list, x)));
  const Entry up{__shfl_up_sync(0xffffffffu, list.v, 1), __shfl_up_sync(0xffffffffu, list.id, 1)};
  if (lane == at) list = x;
  else if (lane > at) list = up;
}

// Joins (M, S, T) of the lanes: every lane gets the warp's.
__device__ __forceinline__ void warp_join(float& M, double& s, double& t) {
  float top = M;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (M == -INFINITY) {
    s = t = 0.0;
  } else if (M != top) {
    const double f = expf(M - top);
    t = f * (t + s * static_cast<double>(M - top));
    s *= f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  M = top;
}

// Puts every lane's e (id >= 0) into a falling list of which the first K count, as far as it is
// ahead of the K-th. Returns whether this lane's was when the call began.
template <int K>
__device__ __forceinline__ bool take_entries(Entry& list, const Entry& e, int lane) {
  auto fits = [&] {
    const Entry last{__shfl_sync(0xffffffffu, list.v, K - 1),
                     __shfl_sync(0xffffffffu, list.id, K - 1)};
    return e.id >= 0 && (last.id < 0 || ahead(e, last));
  };
  const bool first = fits();
  uint32_t hit = __ballot_sync(0xffffffffu, first);
  while (hit) {
    const int src = __ffs(hit) - 1;
    insert_entry(list, Entry{__shfl_sync(0xffffffffu, e.v, src),
                             __shfl_sync(0xffffffffu, e.id, src)}, lane);
    hit &= hit - 1;
    hit &= __ballot_sync(0xffffffffu, fits());
  }
  return first;
}

// Running maximum, S and T of a set of tiles (S and T in fp64, so that a vocabulary of millions
// loses nothing).
struct Sums {
  float M = -INFINITY;
  double s = 0.0, t = 0.0;
  __device__ __forceinline__ void join(float m, double s2, double t2) {
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
  }
};

// Sorted insert into a thread's own falling list; among equal logits the earlier one stays in
// front.
template <int K>
__device__ __forceinline__ void insert_sorted(float (&val)[K], int (&id)[K], float x, int xi) {
#pragma unroll
  for (int j = K - 1; j > 0; --j) {
    const bool here = x > val[j], above = x > val[j - 1];
    id[j] = above ? id[j - 1] : (here ? xi : id[j]);
    val[j] = above ? val[j - 1] : (here ? x : val[j]);
  }
  if (x > val[0]) {
    val[0] = x;
    id[0] = xi;
  }
}

// ------------------------------------------------------------------ the streaming form's split
constexpr int kSRows = kStreamRows;    // rows a tile has room for: the accumulator's lanes
constexpr int kSWarps = 8;             // warps that take positions
constexpr int kSSegs = kStreamLists;   // threads per position, and a thread's rows of a tile
constexpr int kSegRows = kSRows / kSSegs;

// Tile t of `rows` vocabulary rows goes to CTA t mod ctas; rows is what makes all CTAs' tiles
// equal (stats_stream_rows).
struct StreamSplit {
  int V, ctas, rows;
  __host__ __device__ __forceinline__ int tiles(int cta) const {
    const int all = (V + rows - 1) / rows;
    return cta < all ? (all - cta + ctas - 1) / ctas : 0;
  }
  __host__ __device__ __forceinline__ int first(int cta, int t) const { return (t * ctas + cta) * rows; }
  // The list of vocabulary row v: its CTA's, of the segment its row of the tile falls into. In unsigned
  // arithmetic any v names one of the ctas * kSSegs lists: after a wait that ran out a CTA has
  // left its lists unwritten, and the join looks up ids that an earlier use of the workspace left.
  __host__ __device__ __forceinline__ int list_of(int v) const {
    const unsigned u = static_cast<unsigned>(v), r = static_cast<unsigned>(rows);
    return static_cast<int>(u / r % static_cast<unsigned>(ctas) * kSSegs + u % r / kSegRows);
  }
};

}  // namespace dpo
