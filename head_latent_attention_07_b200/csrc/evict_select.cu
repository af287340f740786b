// Choice of the cached tokens that stay: per sequence, the first n_sink, the last
// n_recent and the best of the rest by attention mass, as ascending indices.
//
// A cluster of 1 to 8 CTAs takes one sequence, each CTA a contiguous part of it.
// The mass values become unsigned keys in the same order (NaN above all, -0 equal
// to +0) and are read from memory once, into shared memory.  The key of the last
// token that stays is found by narrowing a key range: the range (at first from the
// smallest to the largest key) is cut into 2048 bins, their counts are summed over
// the cluster, and the bin that holds the wanted rank becomes the next range.
// Each round divides the range by 2048, so at most three are needed, and most
// selections end in the second with a bin that is kept whole.  Starting
// from the keys' own range instead of their top bits spreads the masses, which
// share a few exponents, over all bins: shared-memory atomics on one bin serialise.
// Last, each warp counts what it keeps, and the counts before it (over warps and
// lower CTAs) are its place in the ascending output; of the tokens equal to the
// threshold the lowest indices stay.
#include "common.cuh"
#include "evict.h"
#include "sm100.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxStaged = 49152;      // keys of a CTA kept in shared memory (192 KB); later ones are read again

struct SelectSmem {
  uint32_t hist[kBins];
  uint32_t lo[kMaxCluster], hi[kMaxCluster];   // smallest and largest key of each CTA
  uint32_t total[kMaxCluster];                 // a round's count in each CTA's share of the bins
  uint32_t found[2];                           // the bin of the wanted rank, and the count above it within its share
  uint32_t found_count;
  uint32_t kept[kMaxCluster], ties[kMaxCluster];
  uint32_t warp_a[kWarps], warp_b[kWarps];
};

// Unsigned key in the order of the value: larger mass, larger key.
__device__ __forceinline__ uint32_t mass_key(float v) {
  if (isnan(v)) return 0xFFFFFFFFu;
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

__global__ void __launch_bounds__(kThreads, 1)
evict_select_kernel(const SelectArgs a, const int cluster, const int staged_max) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SelectSmem* sm = reinterpret_cast<SelectSmem*>(smem_raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem_raw + ((sizeof(SelectSmem) + 15) & ~size_t(15)));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const int b = blockIdx.x / cluster;
  auto sync = [&] {
    if (cluster > 1) cluster_sync(); else __syncthreads();
  };
  // the same word of shared memory in every CTA of the cluster
  auto tell_all = [&](uint32_t* where, uint32_t v) {
    for (int r = 0; r < cluster; ++r) st_remote(mapa(smem_u32(where), r), v);
  };

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
    for (int i = rank * kThreads + tid; i < len; i += cluster * kThreads) out[i] = i;
    return;
  }
  const int first = min(a.n_sink, new_len);              // [0, first) stay
  const int last = len - min(a.n_recent, new_len - first);   // [last, len) stay
  uint32_t need = new_len - first - (len - last);        // of [first, last)

  // this CTA's part: whole 32-token groups, in order over the ranks
  const int part = ((len + cluster - 1) / cluster + 31) & ~31;
  const int begin = min(rank * part, len), end = min(begin + part, len);
  const int staged = min(end - begin, staged_max);
  const float* mass = a.mass + (size_t)b * a.mass_stride;
  auto key_at = [&](int i) { return i - begin < staged ? keys[i - begin] : mass_key(mass[i]); };

  uint32_t kmin = 0xFFFFFFFFu, kmax = 0;
#pragma unroll 4
  for (int i = begin + tid; i < end; i += kThreads) {
    const uint32_t k = mass_key(mass[i]);
    if (i - begin < staged) keys[i - begin] = k;
    if (i >= first && i < last) {
      kmin = min(kmin, k);
      kmax = max(kmax, k);
    }
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0) { sm->warp_a[warp] = kmin; sm->warp_b[warp] = kmax; }
  for (int i = tid; i < kBins; i += kThreads) sm->hist[i] = 0;
  // a CTA of the cluster must have started before its shared memory is written
  sync();
  if (warp == 0) {
    kmin = __reduce_min_sync(0xffffffffu, sm->warp_a[lane]);
    kmax = __reduce_max_sync(0xffffffffu, sm->warp_b[lane]);
    if (lane == 0) {
      tell_all(&sm->lo[rank], kmin);
      tell_all(&sm->hi[rank], kmax);
    }
  }
  sync();
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  for (int r = 0; r < cluster; ++r) {
    lo = min(lo, sm->lo[r]);
    hi = max(hi, sm->hi[r]);
  }

  // narrow [lo, hi] to the key of the last token that stays; `need` of the tokens in
  // it stay, and `whole` says that all of them do
  bool whole = false;
  const int share = kBins / cluster;                     // bins summed by each CTA
  while (need > 0 && !whole && lo < hi) {
    int shift = 0;
    while (((hi - lo) >> shift) >= (uint32_t)kBins) ++shift;
    for (int i = max(begin, first) + tid; i < min(end, last); i += kThreads) {
      const uint32_t k = key_at(i);
      if (k >= lo && k <= hi) atomicAdd(&sm->hist[(k - lo) >> shift], 1u);
    }
    sync();
    // CTA r sums bins [r * share, (r + 1) * share) of all CTAs, two per thread at most,
    // and scans its sums from the top bin down
    uint32_t mine[2] = {0, 0};
    const int top = (rank + 1) * share - 1;              // thread t holds bins top - 2t, top - 2t - 1
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (2 * tid + e < share)
        for (int r = 0; r < cluster; ++r) mine[e] += ld_remote(mapa(smem_u32(&sm->hist[top - 2 * tid - e]), r));
    const uint32_t incl = warp_inclusive(mine[0] + mine[1], lane);
    if (lane == 31) sm->warp_a[warp] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t t = sm->warp_a[w];
      if (w < warp) before += t;
      all += t;
    }
    before += incl - mine[0] - mine[1];                  // count in this share above this thread's bins
    if (tid == 0) tell_all(&sm->total[rank], all);
    sync();
    // the counts are read: clear them for the next round
    for (int i = tid; i < kBins; i += kThreads) sm->hist[i] = 0;
    uint32_t above = 0;                                  // count in the shares above this one
    for (int r = rank + 1; r < cluster; ++r) above += sm->total[r];
    above += before;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (mine[e] > 0 && above < need && need <= above + mine[e]) {
        tell_all(&sm->found[0], (uint32_t)(top - 2 * tid - e));
        tell_all(&sm->found[1], above);
        tell_all(&sm->found_count, mine[e]);
      }
      above += mine[e];
    }
    sync();
    need -= sm->found[1];
    whole = need == sm->found_count;
    lo += sm->found[0] << shift;                         // stays at or below hi
    hi = lo + min(hi - lo, (1u << shift) - 1u);
  }
  // keys above hi stay; of those in [lo, hi]: all when `whole`, else (lo == hi) the
  // first `need`
  const bool none = need == 0;
  auto classify = [&](int i, bool* stays, bool* tie) {
    *stays = false;
    *tie = false;
    if (i >= end) return;
    if (i < first || i >= last) { *stays = true; return; }
    if (none) return;
    const uint32_t k = key_at(i);
    *stays = whole ? k >= lo : k > hi;
    *tie = !whole && k == hi;
  };

  // each warp's place: counts of the lower ranks, then of the lower warps
  const int per_warp = ((end - begin + kWarps - 1) / kWarps + 31) & ~31;
  const int wb = min(begin + warp * per_warp, end), we = min(wb + per_warp, end);
  uint32_t n_stay = 0, n_tie = 0;
  for (int i = wb; i < we; i += 32) {
    bool stays, tie;
    classify(i + lane, &stays, &tie);
    n_stay += __popc(__ballot_sync(0xffffffffu, stays));
    n_tie += __popc(__ballot_sync(0xffffffffu, tie));
  }
  __syncthreads();                                       // warp_a of the last round has been read
  if (lane == 0) { sm->warp_a[warp] = n_stay; sm->warp_b[warp] = n_tie; }
  __syncthreads();
  uint32_t stay0 = 0, tie0 = 0, stay_all = 0, tie_all = 0;
  for (int w = 0; w < kWarps; ++w) {
    const uint32_t s = sm->warp_a[w], t = sm->warp_b[w];
    if (w < warp) { stay0 += s; tie0 += t; }
    stay_all += s;
    tie_all += t;
  }
  if (tid == 0) {
    tell_all(&sm->kept[rank], stay_all);
    tell_all(&sm->ties[rank], tie_all);
  }
  sync();
  for (int r = 0; r < rank; ++r) {
    stay0 += sm->kept[r];
    tie0 += sm->ties[r];
  }
  for (int i = wb; i < we; i += 32) {
    bool stays, tie;
    classify(i + lane, &stays, &tie);
    const uint32_t sb = __ballot_sync(0xffffffffu, stays), tb = __ballot_sync(0xffffffffu, tie);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t ties_before = tie0 + __popc(tb & below);
    if (stays || (tie && ties_before < need))
      out[stay0 + __popc(sb & below) + min(ties_before, need)] = i + lane;
    stay0 += __popc(sb);
    tie0 += __popc(tb);
  }
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs& a, int sms, cudaStream_t stream) {
  // CTAs per sequence: as many as give each about 2048 tokens, while all fit the GPU
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)2 * cluster * a.batch <= sms && a.mass_stride > (int64_t)2048 * cluster)
    cluster *= 2;
  const int64_t part = ((a.mass_stride + cluster - 1) / cluster + 31) & ~int64_t(31);
  const int staged = (int)(part < kMaxStaged ? part : kMaxStaged);
  const int smem = (int)((sizeof(SelectSmem) + 15) & ~size_t(15)) + staged * 4;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch * cluster, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cluster, staged);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace mla
