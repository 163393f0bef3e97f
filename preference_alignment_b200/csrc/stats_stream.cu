// Token statistics of a few positions (a serving step): the head's weight is read once and that
// is the time, so the kernel is a stream of W through the tensor cores.
//
// Orientation: W rows are the accumulator's 128 lanes and the NT positions its columns, z^T = W .
// Hp^T, so a pipeline stage is 16 KiB of W and only NT * 128 bytes of hidden rows (the other
// orientation pads a few positions to 128 rows, 16 KiB a stage). The CTAs walk W side by side,
// tile t going to CTA t mod gridDim, in tiles of at most 128 rows so many that every CTA gets the
// same number (V = 151,936: 9 tiles of 115 rows on each of 148 CTAs; with 128 rows, 3 tiles would
// make a ninth wave). (One contiguous range per CTA reads 148 places of W at a time instead of
// one: 187 us instead of 164 us at V = 128,256, d = 4096.) Every running value stays on chip until
// the CTA is done, so a position leaves one set of sums per CTA, not one per tile.
//
// HBM bounds it: one position at V = 128,256, d = 4096 takes 158 us (6.6 TB/s), with 8 alternatives
// and the join 168 us; 48 positions at V = 151,936, d = 2048 take 103 us, 110 us with 8
// alternatives, 121 us with 20 (the lists' upkeep, see kBidGroups).
//
// Roles (320 threads): warp 0 issues the TMA loads, warp 1 owns TMEM and issues the MMAs, warps
// 2-9 turn the accumulator around through shared memory (z[position][vocabulary row]); then each
// thread has one position and one segment of a tile's rows, keeps the running maximum, S, T and
// its K largest logits in registers.
#include <algorithm>

#include "internal.h"
#include "stats.cuh"
#include "stats_join.cuh"

namespace dpo {

namespace {

constexpr int kSWBytes = kSRows * kBK * 2;     // 16 KiB of W per stage
constexpr int kSThreads = (2 + kSWarps) * 32;

template <int NT>
struct StreamShape {
  static constexpr int kStages = NT == 64 ? 7 : NT == 32 ? 10 : 11;
  static constexpr int kHBytes = NT * kBK * 2;
  static constexpr int kStage = kSWBytes + kHBytes;
  static constexpr int kPitch = kSRows + 1;                // of z: odd, so columns spread over banks
  static constexpr int kZ = NT * kPitch * 4;               // z[position][row], later the sums
  static constexpr int kSmem =
      kStages * kStage + kZ + NT * 4 + 3 * kSSegs * NT * 4 + (2 * kStages + 5) * 8 + 16 + 1024;
  static constexpr int kTmem = 2 * NT < 32 ? 32 : 2 * NT;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

// 8, 16 or 32 consecutive fp32 columns of this warp's 32 TMEM lanes.
template <int N>
__device__ __forceinline__ void tmem_cols(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 32) {
    tmem_ld32(addr, r);
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
  } else {
    static_assert(N == 8, "8, 16 or 32 columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(addr));
  }
}

// Barrier over the kSWarps position warps.
__device__ __forceinline__ void warps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSWarps * 32) : "memory");
}
// The same barrier, joined with an AND over its threads: every warp takes the same decision to
// go on or to leave, so none is left waiting in it.
__device__ __forceinline__ bool warps_all(bool mine) {
  int all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(mine ? 1 : 0), "n"(kSWarps * 32)
      : "memory");
  return all != 0;
}

// Long lists: a new logit costs a pass over the list. At K = 32 and 48 positions the first of nine
// tiles takes the position warps 12 us and the others 38 us together; with bids between the CTAs,
// as the GEMM route's tiles make them (stats.cu), 14 us and 17 us (a tile arrives every 10 us).
// Lists of 8 take 5 us and 13 us without; they have none, and no launch that zeroes them.
constexpr int kBidGroups = 32;
constexpr bool has_bids(int K) { return K >= kBidGroups; }

struct StreamArgs {
  const int* y;         // given tokens, or nullptr
  // by position, so that the finish reads whole lines
  float4* part;         // [n, CTAs] (m, S, T, -)
  float* zy;            // [n]
  float2* top;          // [n, CTAs * kSSegs] the lists' first entries (logit, id)
  float2* rest;         // [n, CTAs * kSSegs, K - 1] and the others
  uint32_t* bids;       // [kBidGroups, n] (K = 32), zeroed before the launch
  int n, V, k_blocks;
  int rows;             // vocabulary rows per tile
};

// Where the join finds this form's results (stats_join.cuh).
struct StreamSets {
  const float4* part;
  const float2 *top, *rest;
  int V, ctas, rows;
  static constexpr int kFrom = 1;            // list entries that the sets' keys already are
  __device__ __forceinline__ int sums() const { return ctas; }
  __device__ __forceinline__ float4 sum(int p, int k) const {
    return __ldcg(part + static_cast<long long>(p) * ctas + k);
  }
  __device__ __forceinline__ int sets() const { return ctas * kSSegs; }
  __device__ __forceinline__ uint32_t floor_of(int, int) const { return 0; }
  __device__ __forceinline__ unsigned long long key(int p, int k, uint32_t) const {
    return entry_key(__ldcg(top + static_cast<long long>(p) * sets() + k));
  }
  // by CTA: a short tile leaves some segments without rows, and a group without logits bounds
  // nothing
  template <int K>
  __device__ __forceinline__ int group(int k) const {
    return k / kSSegs % K;
  }
  template <int K>
  __device__ __forceinline__ float2 entry(int p, unsigned long long key, int j) const {
    const int set = StreamSplit{V, ctas, rows}.list_of(key_id(key));
    return __ldcg(rest + (static_cast<long long>(p) * sets() + set) * (K - 1) + (j - 1));
  }
};
static_assert(kStreamCtas * kSSegs <= kJoinSets, "room for every list");

template <int NT, int K>
__global__ void __launch_bounds__(kSThreads, 1)
    k_stats_stream(const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmH, StreamArgs a, DevCtl ctl) {
  using Sh = StreamShape<NT>;
  constexpr int kStages = Sh::kStages;
  constexpr int kList = K > 0 ? K : 1;
  constexpr int kBatch = join_batch<K, StreamSets>();
  constexpr int kPitch = Sh::kPitch;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sW = smem;
  uint8_t* sH = sW + kStages * kSWBytes;
  float* z = reinterpret_cast<float*>(sH + kStages * Sh::kHBytes);
  int* sy = reinterpret_cast<int*>(z + NT * Sh::kPitch);
  float* share = reinterpret_cast<float*>(sy + NT);    // [2][kSSegs][NT], by the tile's parity
  uint32_t* bound = reinterpret_cast<uint32_t*>(share + 2 * kSSegs * NT);   // [kSSegs][NT] of the bids
  uint64_t* bars = reinterpret_cast<uint64_t*>(bound + kSSegs * NT);
  // bars: [0, S) full, [S, 2S) empty, 2S + {0,1} acc_full, 2S + {2,3} acc_empty, 2S + 4 drain
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = smem_u32(bars + kStages);
  const uint32_t accf0 = smem_u32(bars + 2 * kStages);
  const uint32_t acce0 = smem_u32(bars + 2 * kStages + 2);
  const uint32_t drain = smem_u32(bars + 2 * kStages + 4);

  const StreamSplit split{a.V, static_cast<int>(gridDim.x), a.rows};
  const int tiles = split.tiles(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, kSWarps * 32);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmH);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Sh::kTmem);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < NT; i += kSThreads)
    sy[i] = a.y != nullptr && i < a.n ? __ldg(a.y + i) : -1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  uint32_t issued_mask = 0, issued_par = 0;   // for the teardown, as in the GEMM kernels

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = 0; t < tiles && ok; ++t) {
      const int r0 = split.first(blockIdx.x, t);
      const uint32_t bytes = a.rows * kBK * 2 + Sh::kHBytes;   // rows past V arrive as zeros
      for (int kb = 0; kb < a.k_blocks; ++kb) {
        if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, ctl, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t fb = full0 + 8 * stage;
        mbar_arrive_expect_tx(fb, bytes);
        const uint32_t w_dst = smem_u32(sW + stage * kSWBytes);
        tma_load_2d(w_dst, &tmW, fb, kb * kBK, r0);
        tma_load_2d(smem_u32(sH + stage * Sh::kHBytes), &tmH, fb, kb * kBK, 0);
        issued_mask |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {
      record_status(ctl, kStatusTimeout);
      *abort_flag = 1;
    }
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = idesc_bf16_f32(kSRows, NT, false, false);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = 0; t < tiles && ok; ++t) {
      const int acc = t & 1;
      if (!mbar_wait(acce0 + 8 * acc, ((t >> 1) & 1) ^ 1, ctl, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int kb = 0; kb < a.k_blocks; ++kb) {
        if (!mbar_wait(full0 + 8 * stage, phase, ctl, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t w0 = smem_u32(sW + stage * kSWBytes);
        const uint32_t h0 = smem_u32(sH + stage * Sh::kHBytes);
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)
          tc_mma_f16(tmem_base + acc * NT, sw128_desc(w0 + k * 32, 16, 1024),
                     sw128_desc(h0 + k * 32, 16, 1024), idesc, (kb != 0 || k != 0) ? 1u : 0u);
        tc_commit(empty0 + 8 * stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      tc_commit(accf0 + 8 * acc);
    }
    if (!ok) {
      record_status(ctl, kStatusTimeout);
      *abort_flag = 1;
    }
    tc_commit(drain);                       // no MMA may be in flight when TMEM is freed
    volatile int never = 0;
    if (!mbar_wait(drain, 0, ctl, &never)) record_status(ctl, kStatusTimeout);
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- positions
    const int pt = threadIdx.x - 64;
    const int quad = warp & 3;              // TMEM lanes this warp may read
    constexpr int kCols = NT / 2;           // and its half of the columns
    const int c0 = ((warp - 2) >> 2) * kCols;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int p = pt % NT, seg = pt / NT;   // this thread's position and segment
    const bool mine = pt < NT * kSSegs && p < a.n;
    const int set = blockIdx.x * kSSegs + seg;
    float m = kFloor, s = 0.f, tt = 0.f;
    float bid = kFloor;                     // the largest logit bid so far
    float val[kList];
    int id[kList];
#pragma unroll
    for (int j = 0; j < kList; ++j) {
      val[j] = kFloor;
      id[j] = -1;
    }
    bool ok = true;
    for (int t = 0; t < tiles; ++t) {
      const int acc = t & 1;
      ok = mbar_wait(accf0 + 8 * acc, (t >> 1) & 1, ctl, abort_flag);
      // also: every warp is done with the last tile's z
      if (!warps_all(ok)) {
        if (!ok) record_status(ctl, kStatusTimeout);
        *abort_flag = 1;
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t low_bid = 0xffffffffu;         // this thread's share of the groups
      if (has_bids(K) && mine) {
#pragma unroll
        for (int g = 0; g < kBidGroups / kSSegs; ++g)
          low_bid = min(low_bid, __ldcg(a.bids + (seg * (kBidGroups / kSSegs) + g) * a.n + p));
      }
      {
        uint32_t v[kCols];
        tmem_cols<kCols>(tmem_base + lanes + acc * NT + c0, v);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(acce0 + 8 * acc);
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          z[(c0 + c) * kPitch + quad * 32 + lane] = __uint_as_float(v[c]);
      }
      if (has_bids(K) && mine) bound[seg * NT + p] = low_bid;
      warps_sync();
      const int r0 = split.first(blockIdx.x, t);
      const int rows = min(a.rows, a.V - r0);
      const float* zp = z + p * kPitch + (seg % kSSegs) * kSegRows;
      float x[kSegRows];
      float cm = -INFINITY;
#pragma unroll
      for (int j = 0; j < kSegRows; ++j) {
        x[j] = seg * kSegRows + j < rows ? zp[j] : -INFINITY;
        cm = fmaxf(cm, x[j]);
      }
      if (mine && seg == 0 && sy[p] >= r0 && sy[p] < r0 + rows) a.zy[p] = z[p * kPitch + sy[p] - r0];
      // rounded products (no fused multiply-add): back is exactly 0 while the maximum stands
      const float nm = fmaxf(m, cm);
      const float nref = __fmul_rn(nm, kLog2eS);
      const float back = __fmul_rn(m, kLog2eS) - nref;
      const float f = ex2_approx(back);
      tt = f * fmaf(s, back, tt);
      s *= f;
      m = nm;
      float ds = 0.f, dt = 0.f;              // the tile's own sums: short chains of additions
#pragma unroll
      for (int j = 0; j < kSegRows; ++j) {
        const float b = fmaf(x[j], kLog2eS, -nref);
        const float ex = ex2_approx(b);
        ds += ex;
        dt = fmaf(ex, fmaxf(b, -1e30f), dt);               // the bound keeps 0 * -inf out of T
      }
      s += ds;
      tt += dt;
      if (K > 0) {
        // K / 4 logits of each of the position's 4 threads are K logits: one below the smallest of
        // their (K / 4)-th is no alternative (nor one equal to it: its id would be the highest)
        float low = val[kList - 1];
        if (K >= kSSegs && t > 0 && mine) {
          const float* last = share + ((t - 1) & 1) * kSSegs * NT;
          float all = last[p];
#pragma unroll
          for (int g = 1; g < kSSegs; ++g) all = fminf(all, last[g * NT + p]);
          low = fmaxf(low, all);
        }
        float tauv = -INFINITY;
        if (has_bids(K) && mine) {
          uint32_t th = bound[p];
#pragma unroll
          for (int g = 1; g < kSSegs; ++g) th = min(th, bound[g * NT + p]);
          tauv = from_ordered(th);
        }
        uint32_t hit = 0;
        if (mine && cm > low && cm >= tauv) {
#pragma unroll
          for (int j = 0; j < kSegRows; ++j) hit |= (x[j] > low && x[j] >= tauv ? 1u : 0u) << j;
        }
        while (hit != 0) {
          const int j = __ffs(hit) - 1;
          hit &= hit - 1;
          insert_sorted<kList>(val, id, zp[j], r0 + seg * kSegRows + j);
        }
        if (has_bids(K) && mine && t + 1 < tiles && val[0] > bid) {
          bid = val[0];
          atomicMax(a.bids + blockIdx.x % kBidGroups * a.n + p, ordered(bid));
        }
        // read after the next tile's barrier; not in the place that the last tile's are read from:
        // this tile's logits have higher ids in other segments
        if (K >= kSSegs && mine)
          share[((t & 1) * kSSegs + seg) * NT + p] = val[kList >= kSSegs ? kList / kSSegs - 1 : 0];
      }
    }
    // a position's segments join in a fixed order, in z's place; one set of sums per CTA
    if (warps_all(ok)) {
      const float r = fmaf(-m, kLog2eS, __fmul_rn(m, kLog2eS));   // what m * log2(e) lost
      if (seg < kSSegs) {
        float* q = z + (seg * NT + p) * 3;
        q[0] = m;
        q[1] = fmaf(s, r * kLn2S, s);
        q[2] = fmaf(s, r, tt) * kLn2S;
      }
      warps_sync();
      if (mine && seg == 0) {
        Sums j;
        for (int g = 0; g < kSSegs; ++g) {
          const float* w = z + (g * NT + p) * 3;
          j.join(w[0], w[1], w[2]);
        }
        a.part[static_cast<long long>(p) * gridDim.x + blockIdx.x] =
            make_float4(j.M, static_cast<float>(j.s), static_cast<float>(j.t), 0.f);
      }
      if (K > 0 && mine) {
        const long long at = static_cast<long long>(p) * gridDim.x * kSSegs + set;
        a.top[at] = make_float2(val[0], __int_as_float(id[0]));
        // entries that K others are ahead of are left out: the finish reads a batch at a time and
        // goes on to the next only from a full one
        float low = kFloor;
        if (K >= kSSegs) {
          const float* last = share + ((tiles - 1) & 1) * kSSegs * NT;
          low = last[p];
#pragma unroll
          for (int g = 1; g < kSSegs; ++g) low = fminf(low, last[g * NT + p]);
        }
        float2* l = a.rest + at * (kList - 1);
        bool open = true;
#pragma unroll
        for (int j = 1; j < kList; ++j) {
          const bool keep = val[j] > kFloor && val[j] >= low;
          if (open)
            l[j - 1] = keep ? make_float2(val[j], __int_as_float(id[j])) : make_float2(kFloor, 0.f);
          if (j % (kBatch > 0 ? kBatch : 1) == 0) open = keep;
        }
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_flag) {
    // after an abort, loads may still be landing: wait (bounded) for each stage's last one
    volatile int never = 0;
    DevCtl c2 = ctl;
    c2.budget_ns = ctl.budget_ns / 4 + 1000000ull;
    for (int s = 0; s < kStages; ++s)
      if (issued_mask & (1u << s))
        (void)mbar_wait(full0 + 8 * s, (issued_par >> s) & 1u, c2, &never);
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, Sh::kTmem);
  }
}

template <int NT, int K>
cudaError_t stream_launch(const CUtensorMap& mW, const CUtensorMap& mH, const StreamArgs& a,
                          int grid, const DevCtl& ctl, cudaStream_t st) {
  auto kern = k_stats_stream<NT, K>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             StreamShape<NT>::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kSThreads, StreamShape<NT>::kSmem, st>>>(mW, mH, a, ctl);
  return cudaGetLastError();
}

template <int K>
cudaError_t stream_by_positions(const CUtensorMap& mW, const CUtensorMap& mH, const StreamArgs& a,
                                int ctas, const StatsOut& out, const DevCtl& ctl,
                                cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (has_bids(K)) e = cudaMemsetAsync(a.bids, 0, sizeof(uint32_t) * kBidGroups * a.n, st);
  if (e != cudaSuccess) return e;
  switch (stats_stream_cols(a.n)) {
    case 16: e = stream_launch<16, K>(mW, mH, a, ctas, ctl, st); break;
    case 32: e = stream_launch<32, K>(mW, mH, a, ctas, ctl, st); break;
    default: e = stream_launch<64, K>(mW, mH, a, ctas, ctl, st); break;
  }
  if (e != cudaSuccess) return e;
  return launch_join<K>(StreamSets{a.part, a.top, a.rest, a.V, ctas, a.rows}, a.y, a.zy, a.n, a.V, out,
                        ctl, st);
}

}  // namespace

int stats_stream_cols(int n) { return n <= 16 ? 16 : n <= 32 ? 32 : 64; }

// One CTA per SM, of 8 rows at least.
int stats_stream_ctas(int V, int sms) {
  return std::min(std::min(sms, kStreamCtas), (V + 7) / 8);
}

int stats_stream_rows(int V, int ctas) {
  const int tiles = (V + kSRows * ctas - 1) / (kSRows * ctas);      // per CTA
  return (V + ctas * tiles - 1) / (ctas * tiles);
}

cudaError_t launch_stats_stream(const CUtensorMap& mapW, const CUtensorMap& mapH,
                                const StatsBuf& b, const StatsOut& out, int n, int V, int d,
                                const int* y, int ctas, const DevCtl& ctl, cudaStream_t st) {
  const size_t sets = static_cast<size_t>(n) * ctas * kSSegs;
  const StreamArgs a{y, reinterpret_cast<float4*>(b.part), b.zy, b.list, b.list + sets, b.tau, n, V,
                     (d + kBK - 1) / kBK, stats_stream_rows(V, ctas)};
  switch (stats_list_len(out.n_top)) {
    case 0: return stream_by_positions<0>(mapW, mapH, a, ctas, out, ctl, st);
    case 1: return stream_by_positions<1>(mapW, mapH, a, ctas, out, ctl, st);
    case 8: return stream_by_positions<8>(mapW, mapH, a, ctas, out, ctl, st);
    default: return stream_by_positions<32>(mapW, mapH, a, ctas, out, ctl, st);
  }
}

}  // namespace dpo
