// The join of token statistics: one block per position joins the sums that its tiles or CTAs left
// and finds the alternatives in their lists.
//
// The kernel before has just run W through L2 and pushed this one's instructions out, so its time
// is the number of instruction lines it fetches from HBM as much as anything: loops are rolled,
// sums are fp32 (a few terms a thread), one piece of code joins lanes and warps, and a list entry
// is compared as one number. (Unrolled, in fp64 and with two comparisons per entry it took 12 us
// instead of 5 us for 48 positions at K = 8, and 30 us at K = 32.)
//
// Alternatives, all without a chain of insertions: (1) the sets' largest logits, dealt out over K
// groups, give K different logits, the groups' maxima, so the smallest of those is a lower bound of
// the K-th largest of them, which about K log K reach; (2) each of these counts how many are ahead
// of it, its rank: a logit of any set but the K first has K others ahead of it; (3) the entries of
// those K sets' lists that are not behind the K-th largest logit are ranked again: the answer.
#pragma once

#include "chain.cuh"
#include "internal.h"
#include "stats.cuh"

namespace dpo {

constexpr int kJoin = 256;           // threads: a block per position
constexpr int kJoinSets = 1024;      // sets at most

// A list entry (logit, id) as one number: greater is ahead (the larger logit, then the lower id);
// 0 stands for none.
__device__ __forceinline__ unsigned long long entry_key(const float2& r) {
  return r.x > kFloor ? static_cast<unsigned long long>(ordered(r.x)) << 32 |
                            static_cast<uint32_t>(~__float_as_int(r.y))
                      : 0ull;
}
__device__ __forceinline__ int key_id(unsigned long long k) {
  return ~static_cast<int>(static_cast<uint32_t>(k));
}

// List entries that the join looks at together, one per thread for each of the K lists.
template <int K, class Sets>
__host__ __device__ constexpr int join_batch() {
  return K == 0 ? 0 : K * (K - Sets::kFrom) <= kJoin ? K - Sets::kFrom : kJoin / K;
}

// Sets: where the results lie.
//   sums(), sum(p, k)        sets of sums (m, S, T, -) of position p
//   sets(), key(p, k, floor) sets with a list; the largest logit's key (its id, or with kFrom = 0
//                            the set's index, which orders equal ones alike), 0 if there is no list
//   floor_of(p, lane)        what key() leaves out: an ordered logit, the same in every lane
//   group<K>(k)              the set's group of K
//   entry<K>(p, key, j)      entry j of the list whose key this is, j >= kFrom
template <int K, class Sets>
__global__ void __launch_bounds__(kJoin) k_stats_join(Sets sets, const int* y, const float* zy, int V,
                                                      StatsOut out, DevCtl ctl) {
  constexpr int kList = K > 0 ? K : 1;
  constexpr int kMost = kJoinSets > kList * kList ? kJoinSets : kList * kList;
  __shared__ float4 sums[kJoin / 32];
  __shared__ uint32_t group[kList];
  __shared__ int count[2];
  __shared__ unsigned long long tops[K > 0 ? kJoinSets : 1], cand[K > 0 ? kMost : 1], first[kList];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int p = blockIdx.x;
  if (K > 0) {
    if (t < kList) {
      group[t] = 0;
      first[t] = 0;
    }
    if (t < 2) count[t] = 0;
    __syncthreads();
  }
  after_previous();
  // what the kernel before wrote is read past L1 (__ldcg): this one may have started before it
  float4 q = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  // moves the sums to a new reference; what was never set stays nothing, and equal references
  // (also infinite ones) change nothing
  auto refer = [](float4& v, float top) {
    if (v.x != top) {
      const float back = v.x - top, f = ex2_approx(back * kLog2eS);
      v.z = v.x == -INFINITY ? 0.f : f * fmaf(v.y, back, v.z);
      v.y = v.x == -INFINITY ? 0.f : f * v.y;
      v.x = top;
    }
  };
#pragma unroll 1
  for (int k = t; k < sets.sums(); k += kJoin) {
    float4 v = sets.sum(p, k);
    const float top = fmaxf(q.x, v.x);
    refer(q, top);
    refer(v, top);
    q.y += v.y;
    q.z += v.z;
  }
  if (K > 0) {
    const uint32_t floor = sets.floor_of(p, lane);
#pragma unroll 1
    for (int k = t; k < sets.sets(); k += kJoin) {
      const unsigned long long e = sets.key(p, k, floor);
      tops[k] = e;
      if (e != 0) atomicMax(&group[sets.template group<kList>(k)], static_cast<uint32_t>(e >> 32));
    }
  }
  // lanes, then warps: the same code twice
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    refer(q, from_ordered(__reduce_max_sync(0xffffffffu, ordered(q.x))));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      q.y += __shfl_xor_sync(0xffffffffu, q.y, o);
      q.z += __shfl_xor_sync(0xffffffffu, q.z, o);
    }
    if (round == 0) {
      if (lane == 0) sums[warp] = q;
      __syncthreads();
      q = lane < kJoin / 32 ? sums[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    }
  }
  const float ls = logf(q.y);
  if (t == 0) {
    if (out.lse != nullptr) out.lse[p] = q.x + ls;
    if (out.entropy != nullptr) out.entropy[p] = entropy_of(ls - __fdividef(q.z, q.y));
    if (y != nullptr) {
      const int yp = __ldcg(y + p);
      const bool ok = yp >= 0 && yp < V;
      if (!ok) record_status(ctl, kStatusBadTarget);
      // against M before log S: z_y - lse would round away what large logits leave
      if (out.logp != nullptr) out.logp[p] = ok ? (__ldcg(zy + p) - q.x) - ls : 0.f;
    }
  }
  if (K > 0) {
    const unsigned long long bound =
        static_cast<unsigned long long>(
            __reduce_min_sync(0xffffffffu, lane < kList ? group[lane] : 0xffffffffu)) << 32;
#pragma unroll 1
    for (int k = t; k < sets.sets(); k += kJoin) {
      const unsigned long long e = tops[k];
      if (e != 0 && e >= bound) cand[atomicAdd(&count[0], 1)] = e;
    }
    constexpr int kFrom = Sets::kFrom, kBatch = join_batch<kList, Sets>();
    // ranks twice: of the sets, then of all entries that can be among the K largest
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
      __syncthreads();
      const int n = count[round];
#pragma unroll 1
      for (int k = t; k < n; k += kJoin) {
        const unsigned long long x = cand[k];
        int r = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) r += cand[j] > x ? 1 : 0;
        if (r < kList) first[r] = x;
      }
      __syncthreads();
      if (round == 0) {
        // cand from here on: entries not behind the K-th set's largest; several per list at a
        // time, until no list's last one looked at is
        const unsigned long long f =
            kBatch > 0 && t < kList * kBatch ? first[t / (kBatch > 0 ? kBatch : 1)] : 0;
        const unsigned long long last =
            kFrom > 0 ? first[kList - 1] + 1 : first[kList - 1] >> 32 << 32;
        if (kFrom > 0 && t < kList && first[t] != 0) cand[atomicAdd(&count[1], 1)] = first[t];
        bool open = f != 0, more = kBatch > 0;
#pragma unroll 1
        for (int j0 = kFrom; j0 < kList && more; j0 += kBatch) {
          const int j = j0 + t % (kBatch > 0 ? kBatch : 1);
          bool take = false;
          if (open && j < kList) {
            const unsigned long long x = entry_key(sets.template entry<kList>(p, f, j));
            take = x != 0 && x >= last;
            if (take) cand[atomicAdd(&count[1], 1)] = x;
          }
          if constexpr (kList - kFrom > kBatch) {
            // each list by itself: behind a batch that is not full nothing was written
            static_assert(kBatch > 0 && 32 % kBatch == 0, "a list's threads are in one warp");
            open = (__ballot_sync(0xffffffffu, take) >> (lane | (kBatch - 1)) & 1) != 0;
            more = __syncthreads_or(open) != 0;
          }
        }
      }
    }
    // `first` now holds the answer; where there are fewer logits than asked for, the rest is empty
    if (t < out.n_top) {
      const unsigned long long x = t < count[1] ? first[t] : 0;
      out.top_ids[static_cast<long long>(p) * out.n_top + t] = x != 0 ? key_id(x) : -1;
      out.top_logp[static_cast<long long>(p) * out.n_top + t] =
          x != 0 ? (from_ordered(static_cast<uint32_t>(x >> 32)) - q.x) - ls : -INFINITY;
    }
  }
}

template <int K, class Sets>
cudaError_t launch_join(const Sets& sets, const int* y, const float* zy, int n, int V,
                        const StatsOut& out, const DevCtl& ctl, cudaStream_t st) {
  // the same split of the SMs' memory as the kernel before: another split would wait for the SMs
  // to drain and change over (140 us instead of 132 us for 48 positions with 20 alternatives)
  const cudaError_t e =
      cudaFuncSetAttribute(k_stats_join<K, Sets>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  return launch_after(k_stats_join<K, Sets>, dim3(n), kJoin, st, sets, y, zy, V, out, ctl);
}

}  // namespace dpo
