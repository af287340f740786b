// Choice of the cached tokens that stay: per sequence, the first n_sink, the last
// n_recent and the best of the rest by attention mass, as ascending indices.
//
// A cluster of 1 to 8 CTAs takes one sequence, each CTA a contiguous part of it.
// The mass values become unsigned keys in the same order (NaN above all, -0 equal
// to +0) and are read from memory once, into shared memory.  The key of the last
// token that stays is found by narrowing a key range: the range is cut into 2048 bins,
// their counts are summed over the cluster, and the bin that holds the wanted rank
// becomes the next range.  The first bins are 2^17 keys wide (64 to a factor of two)
// over the values from 2^-24 to 2^8, where masses lie, and the outer two hold all
// beyond: so the keys spread over many bins (shared-memory atomics on one bin
// serialise), and the second round mostly ends it with a bin that is kept whole.  A later
// round divides the range by 2048: four rounds at most.  Last, each warp counts what it
// keeps, and the counts before it (over warps and lower CTAs) are its place in the
// ascending output; of the tokens equal to the threshold the lowest indices stay.
//
// Keys past the staged ones are read again in every pass.  A mass that another stream still
// writes gives a wrong choice, but the rounds are counted and a place past the new length is
// not written: no loop without end, nothing outside the sequence's row.
//
// Latency binds it (2 MB of mass are read in well under a microsecond): one cluster
// barrier a round, which the counts of groups of bins cross; the bins of the one group that
// matters are read from the other CTAs' shared memory after it.  Measured: 4.5 us for 1000
// tokens, 12.0 for 16 x 32768, 17 for 8 x 131072 (the mass itself at 0.25 TB/s).
#include "common.cuh"
#include "evict.h"
#include "sm100.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int kMinThreads = 512, kMaxThreads = 1024;
constexpr int kBins = 2048, kGroups = kBins / 32;
constexpr int kFirstShift = 17;
constexpr int kMaxRounds = 4;          // bins of 2^17 keys (an outer one: below 2^32), of 2^21, 2^10 and 1 at most
constexpr uint32_t kFirstLo = 0x80000000u | ((127u - 24u) << 23);   // key of 2^-24
constexpr int kMaxCluster = 8;
constexpr int kMaxStaged = 40960;      // keys of a CTA kept in shared memory (160 KB); later ones are read again

struct SelectSmem {
  // The rounds alternate between two copies of both counts.  What a CTA or its peers read of
  // round r's copy after that round's cluster barrier is written again in round r + 2 at the
  // earliest, behind the barrier of round r + 1, where every reader arrives after its reads.
  uint32_t hist[2][kBins];                     // this CTA's counts
  uint32_t coarse[2][kMaxCluster][kGroups];    // each CTA's counts in groups of 32 bins
  uint32_t kept[kMaxCluster], ties[kMaxCluster];
  uint32_t warp_a[32], warp_b[32];
  uint32_t found_bin, found_above, found_count;   // the bin of the wanted rank
};

// Unsigned key in the order of the value: larger mass, larger key.  The smallest is
// -infinity's 0x007FFFFF; below lie kNoKey, for places past the end, and kNoTie; above
// all, the key of a token that stays whatever its mass.
constexpr uint32_t kNoKey = 0, kNoTie = 1, kNanKey = 0xFFFFFFFEu, kStays = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t mass_key(float v) {
  if (isnan(v)) return kNanKey;
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void st_remote(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_remote(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t warp_inclusive(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// In a warp whose lanes hold counts from the top down: the lane in which the
// `need`-th falls, and the count before it.
__device__ __forceinline__ int lane_of_rank(uint32_t v, uint32_t need, int lane, uint32_t* before) {
  const uint32_t incl = warp_inclusive(v, lane);
  const int at = __ffs(__ballot_sync(0xffffffffu, incl >= need)) - 1;
  *before = __shfl_sync(0xffffffffu, incl - v, at);
  return at;
}

__global__ void __launch_bounds__(kMaxThreads, 1)
evict_select_kernel(const SelectArgs a, const int cluster, const int staged_max) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SelectSmem* sm = reinterpret_cast<SelectSmem*>(smem_raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem_raw + ((sizeof(SelectSmem) + 15) & ~size_t(15)));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int threads = blockDim.x, warps = threads >> 5;
  const int rank = (int)cluster_ctarank();
  const int b = blockIdx.x / cluster;
  auto sync = [&] {
    if (cluster > 1) cluster_sync(); else __syncthreads();
  };
  for (int i = tid; i < kBins; i += threads) sm->hist[0][i] = 0;

  grid_dependency_wait();
  allow_dependent_launch();
  const int len = a.seq_lens[b];
  const int budget = a.budgets[b];
  const int new_len = min(len, budget);
  // every CTA of the cluster takes the same way out
  if (len < 0 || len > a.mass_stride || budget < 0 || new_len > a.keep_stride) {
    if (rank == 0 && tid == 0) {
      record_status(a.dev_status, MLA_ERR_RANGE);
      a.new_lens[b] = 0;
    }
    return;
  }
  if (rank == 0 && tid == 0) a.new_lens[b] = new_len;
  int32_t* out = a.keep_idx + (size_t)b * a.keep_stride;
  if (new_len == len) {
    for (int i = rank * threads + tid; i < len; i += cluster * threads) out[i] = i;
    return;
  }
  if (cluster > 1) cluster_arrive_relaxed();             // answered before the first access to another CTA's memory
  const int first = min(a.n_sink, new_len);              // [0, first) stay
  const int last = len - min(a.n_recent, new_len - first);   // [last, len) stay
  uint32_t need = new_len - first - (len - last);        // of [first, last)

  // this CTA's part: whole groups of 128 tokens (four for each lane of a warp), in order over
  // the ranks
  const int part = ((len + cluster - 1) / cluster + 127) & ~127;
  const int begin = min(rank * part, len), end = min(begin + part, len);
  const int staged = min((end - begin + 127) & ~127, staged_max);
  const float* mass = a.mass + (size_t)b * a.mass_stride;
  auto key_for = [&](int i, float v) { return i >= end ? kNoKey : i < first || i >= last ? kStays : mass_key(v); };
  auto key_of = [&](int i) { return key_for(i, i < end ? mass[i] : 0.f); };
  auto quad_at = [&](int i) {                            // the keys of four tokens, i - begin a multiple of 4
    return i - begin < staged ? *reinterpret_cast<const uint4*>(keys + (i - begin))
                              : make_uint4(key_of(i), key_of(i + 1), key_of(i + 2), key_of(i + 3));
  };

  constexpr int kLoads = 8;                              // in flight at a time
  for (int i0 = tid; i0 < staged; i0 += kLoads * threads) {
    float v[kLoads];
#pragma unroll
    for (int e = 0; e < kLoads; ++e) {
      const int i = begin + i0 + e * threads;
      v[e] = i < end ? mass[i] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kLoads; ++e)
      if (i0 + e * threads < staged) keys[i0 + e * threads] = key_for(begin + i0 + e * threads, v[e]);
  }
  __syncthreads();
  if (cluster > 1) cluster_wait();                       // every CTA has started

  // narrow [lo, hi] to the key of the last token that stays; `need` of the tokens in
  // it stay, and `whole` says that all of them do
  bool whole = false;
  uint32_t lo = kNoTie + 1, hi = kNanKey;
  for (int round = 0; need > 0 && !whole && lo < hi && round < kMaxRounds; ++round) {
    // bin i holds the keys from base + (i << shift) on, the first and the last all beyond
    const int shift = round == 0 ? kFirstShift : max(0, 21 - __clz(hi - lo));   // (hi - lo) >> shift < kBins
    const uint32_t base = round == 0 ? kFirstLo : lo;
    uint32_t* hist = sm->hist[round & 1];
    auto& coarse = sm->coarse[round & 1];
    auto count = [&](uint32_t k) {
      if (k >= lo && k <= hi) atomicAdd(&hist[k < base ? 0 : min((k - base) >> shift, kBins - 1u)], 1u);
    };
#pragma unroll 2
    for (int i = begin + 4 * tid; i < end; i += 4 * threads) {
      const uint4 q = quad_at(i);
      count(q.x), count(q.y), count(q.z), count(q.w);
    }
    __syncthreads();
    uint32_t sum[kGroups / (kMinThreads / 32)];
#pragma unroll
    for (int j = 0; j < kGroups / (kMinThreads / 32); ++j) {
      const int g = warp + j * warps;
      sum[j] = __reduce_add_sync(0xffffffffu, g < kGroups ? hist[g * 32 + lane] : 0);
    }
#pragma unroll
    for (int j = 0; j < kGroups / (kMinThreads / 32); ++j) {
      const int g = warp + j * warps;
      if (g < kGroups && lane < cluster) st_remote(mapa(smem_u32(&coarse[rank][g]), lane), sum[j]);
    }
    sync();
    // the other counts were read before this barrier
    for (int i = tid; i < kBins; i += threads) sm->hist[(round + 1) & 1][i] = 0;
    if (warp == 0) {
      // from the top: the pair of groups, the group, then the bin with the wanted rank
      uint32_t c[2] = {0, 0}, v = 0, above, in_pair, in_group;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        c[0] += r < cluster ? coarse[r][kGroups - 1 - 2 * lane] : 0;
        c[1] += r < cluster ? coarse[r][kGroups - 2 - 2 * lane] : 0;
      }
      const int pair = lane_of_rank(c[0] + c[1], need, lane, &above);
      in_pair = __shfl_sync(0xffffffffu, c[0], pair);
      const bool second = above + in_pair < need;
      if (second) above += in_pair;
      const int bin0 = (kGroups - 1 - 2 * pair - (second ? 1 : 0)) * 32;
      if (cluster > 1) {
        uint32_t of[kMaxCluster];                        // all on their way before the first is used
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          of[r] = ld_remote(mapa(smem_u32(&hist[bin0 + 31 - lane]), min(r, cluster - 1)));
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) v += r < cluster ? of[r] : 0;
      } else {
        v = hist[bin0 + 31 - lane];
      }
      const int at = lane_of_rank(v, need - above, lane, &in_group);
      if (lane == at) {
        sm->found_bin = bin0 + 31 - at;
        sm->found_above = above + in_group;
        sm->found_count = v;
      }
    }
    __syncthreads();
    need -= sm->found_above;
    whole = need == sm->found_count;
    const uint32_t bin = sm->found_bin, from = base + (bin << shift);
    if (bin < kBins - 1u) hi = from + min(hi - from, (1u << shift) - 1u);
    if (bin > 0) lo = from;
  }
  // keys above `over` stay, and of those equal to `tie` the first `need`: of the keys in
  // [lo, hi] all when `whole`, else (lo == hi) the first ones
  const uint32_t over = need == 0 ? kNanKey : whole ? lo - 1 : hi;
  const uint32_t tie = need == 0 || whole ? kNoTie : hi;

  // each warp's place: counts of the lower ranks, then of the lower warps
  const int per_warp = ((end - begin + warps - 1) / warps + 127) & ~127;
  const int wb = min(begin + warp * per_warp, end), we = min(wb + per_warp, end);
  uint32_t n_stay = 0, n_tie = 0;
#pragma unroll 2
  for (int i = wb + 4 * lane; i < we; i += 128) {
    const uint4 q = quad_at(i);
    n_stay += (q.x > over) + (q.y > over) + (q.z > over) + (q.w > over);
    n_tie += (q.x == tie) + (q.y == tie) + (q.z == tie) + (q.w == tie);
  }
  n_stay = __reduce_add_sync(0xffffffffu, n_stay);
  n_tie = __reduce_add_sync(0xffffffffu, n_tie);
  if (lane == 0) { sm->warp_a[warp] = n_stay; sm->warp_b[warp] = n_tie; }
  __syncthreads();
  const uint32_t s = warp_inclusive(lane < warps ? sm->warp_a[lane] : 0, lane);
  const uint32_t t = warp_inclusive(lane < warps ? sm->warp_b[lane] : 0, lane);
  uint32_t stay0 = __shfl_sync(0xffffffffu, s, warp) - n_stay;
  uint32_t tie0 = __shfl_sync(0xffffffffu, t, warp) - n_tie;
  if (cluster > 1) {
    if (warp == 0) {
      const uint32_t stay_all = __shfl_sync(0xffffffffu, s, 31), tie_all = __shfl_sync(0xffffffffu, t, 31);
      if (lane < cluster) {
        st_remote(mapa(smem_u32(&sm->kept[rank]), lane), stay_all);
        st_remote(mapa(smem_u32(&sm->ties[rank]), lane), tie_all);
      }
    }
    sync();
    for (int r = 0; r < rank; ++r) {
      stay0 += sm->kept[r];
      tie0 += sm->ties[r];
    }
  }
  // the places that the counts give; `below` says which may be written
  auto write = [&](auto below) {
#pragma unroll 2
    for (int i0 = wb; i0 < we; i0 += 128) {
      const int i = i0 + 4 * lane;
      const uint4 q = quad_at(i);
      const uint32_t k[4] = {q.x, q.y, q.z, q.w};
      uint32_t mine = 0;                                 // what stays, and the ties in the upper half
#pragma unroll
      for (int e = 0; e < 4; ++e) mine += (k[e] > over ? 1u : 0u) + (k[e] == tie ? 0x10000u : 0u);
      const uint32_t incl = warp_inclusive(mine, lane), before = incl - mine;
      uint32_t stay = stay0 + (before & 0xFFFFu), ties = tie0 + (before >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is_tie = k[e] == tie;
        const uint32_t at = stay + min(ties, need);
        if ((k[e] > over || (is_tie && ties < need)) && below(at)) out[at] = i + e;
        stay += k[e] > over;
        ties += is_tie;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
      stay0 += all & 0xFFFFu;
      tie0 += all >> 16;
    }
  };
  // keys in shared memory are the counted ones; those read again may have changed (looking at
  // every place took 3 % more of 16 x 32768)
  if (part <= staged_max) write([](uint32_t) { return true; });
  else write([&](uint32_t at) { return at < (uint32_t)new_len; });
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs& a, int sms, cudaStream_t stream) {
  // CTAs per sequence: as many as give each about 2048 tokens, while every CTA has an SM of
  // its own.  Clusters of 8 do not pack onto all SMs: 12 of them ran at once on 148, 16 in
  // two waves (of 1024 threads) or two to an SM (of 512), so they may take two thirds.
  // Threads: 8 tokens each before the block doubles.  GPU time, us, by cluster x threads:
  //   16 x 2048     1 x 512  5.9    2 x 512  7.1
  //   16 x 8192     1 x 1024 10.4   2 x 512  8.7    4 x 512  7.7    8 x 512  9.1
  //    8 x 16384                    4 x 512  9.0    8 x 512  8.3
  //   12 x 32768                    4 x 1024 11.9   8 x 512  9.9
  //   16 x 32768    2 x 1024 16.1   4 x 1024 12.1   8 x 512 12.4    8 x 1024 20.4
  //   16 x 65536                    4 x 1024 16.4   8 x 512 16.6    8 x 1024 24.2
  //    8 x 131072                   4 x 1024 24.3   8 x 512 18.4    8 x 1024 17.0
  //   64 ragged to 65536   1 x 1024 53.9   2 x 512 30.7   2 x 1024 26.8   4 x 1024 33.1
  int cluster = 1;
  while (cluster < kMaxCluster && a.mass_stride > (int64_t)2048 * cluster &&
         (int64_t)2 * cluster * a.batch <= (2 * cluster < kMaxCluster ? sms : sms * 2 / 3))
    cluster *= 2;
  const int64_t part = ((a.mass_stride + cluster - 1) / cluster + 127) & ~int64_t(127);
  int threads = kMinThreads;
  while (threads < kMaxThreads && threads * 8 < part) threads *= 2;
  const int staged = (int)(part < kMaxStaged ? part : kMaxStaged);
  const int smem = (int)((sizeof(SelectSmem) + 15) & ~size_t(15)) + staged * 4;
  // always the most: calls of other sizes may be on their way from other host threads
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(SelectSmem) + 16 + kMaxStaged * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch * cluster, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cluster, staged);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace mla
