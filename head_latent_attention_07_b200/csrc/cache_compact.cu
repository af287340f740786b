// In-place compaction of the paged latent cache: row j of a sequence becomes its row
// keep_idx[j] >= j, the RoPE part turned by the angle of j - keep_idx[j], and the
// token's attention mass moves along.
//
// Every kept row that moves is read once and written once, and nothing is staged in
// memory.  In place that is safe in this order: row j may be overwritten once every
// reader of row j has read it, and its readers sit at positions j' <= j (keep_idx[j'] =
// j >= j').  A CTA walks the positions upward in tiles, loads run ahead, and a tile is
// written after a barrier that says that all reads of it and of the tiles below are
// done; loads of later tiles touch rows that no write so far has reached.
//
// Work is split by columns: a CTA takes one 128-byte slice of the row of one sequence
// (nine slices of a 576-wide row), and the slices know nothing of each other.  With few
// sequences, a cluster of CTAs shares a slice: each takes every cluster-size-th tile,
// and the barrier becomes the cluster's.  One more slice per sequence moves the mass.
//
// Bytes bind it: two row widths per moved row.  The copies are cp.async into a ring of
// tiles that each thread fills and empties for itself (a thread writes out the pieces
// that it loaded, so shared memory needs no barrier of its own), with the indices and
// page ids of a tile fetched one tile earlier than its rows.
#include "common.cuh"
#include "evict.h"
#include "sm100.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr int kPieces = 4;                       // 16-byte pieces of a tile per thread
constexpr int kTileBytes = kThreads * kPieces * 16;   // 16 KB: 128 rows of a 128-byte slice
constexpr int kStages = 6;                       // ring of tiles: 96 KB, two CTAs per SM
constexpr int kSliceVecs = 8;                    // 16-byte pieces of a row per slice
constexpr int kTileRows = kThreads * kPieces / kSliceVecs;
constexpr int kMassRows = 8;                     // mass values per thread and tile
constexpr int kMaxCluster = 8;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// (x, y) of a RoPE pair turned by delta positions; turn = 2^64 times the pair's
// rotation per position as a fraction of a full turn.  delta * turn modulo 2^64 is the
// whole rotation modulo one turn, exactly, so far moves keep their phase; its upper 32 bits
// give the angle in [-pi, pi) to 2^-32 turns, and the hardware sine and cosine there are
// good to 2^-21, against the 2^-9 of the bf16 result.
__device__ __forceinline__ uint32_t turn_pair(uint32_t xy, int delta, uint64_t turn) {
  const int32_t phase = (int32_t)(((uint64_t)(int64_t)delta * turn) >> 32);
  const float ang = (float)phase * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float c = __cosf(ang), s = __sinf(ang);
  const float x = bf16_lo(xy), y = bf16_hi(xy);
  return pack_bf16x2(x * c - y * s, x * s + y * c);
}

struct Seq {
  int len, new_len;
  const int32_t* idx;      // keep_idx of the sequence
  const int32_t* pages;    // page table row
};

// Row index of the pool for cache index n, or -1 (and a recorded range error) when
// the page table names a page outside the pool.
__device__ __forceinline__ int64_t pool_row(const CompactArgs& a, const Seq& q, int n, int shift) {
  const int pg = shift >= 0 ? n >> shift : n / a.page_size;
  const int id = q.pages[pg];
  if (id < 0 || id >= a.num_pages) {
    record_status(a.dev_status, MLA_ERR_RANGE);
    return -1;
  }
  return (int64_t)id * a.page_size + (n - pg * a.page_size);
}

// The cache index that moves to position j, or -1 when nothing moves there: j past the
// end, a row that stays, an index outside [j, len) (a recorded range error).
__device__ __forceinline__ int source_of(const CompactArgs& a, const Seq& q, int j) {
  if (j >= q.new_len) return -1;
  const int n = q.idx[j];
  if (n == j) return -1;
  if (n < j || n >= q.len) {
    record_status(a.dev_status, MLA_ERR_RANGE);
    return -1;
  }
  return n;
}

__global__ void __launch_bounds__(kThreads)
cache_compact_kernel(const __grid_constant__ CompactArgs a, const int cluster, const int page_shift) {
  extern __shared__ __align__(16) unsigned char ring[];
  const int tid = threadIdx.x;
  const int rank = (int)cluster_ctarank();
  const int slice = blockIdx.x / cluster;
  const int b = blockIdx.y;
  const int rv = (a.d_c + a.d_rope) / 8;
  const int slices = (rv + kSliceVecs - 1) / kSliceVecs;
  auto sync = [&] {
    if (cluster > 1) cluster_sync(); else __syncthreads();
  };

  grid_dependency_wait();
  allow_dependent_launch();
  Seq q;
  q.len = a.seq_lens[b];
  q.new_len = a.new_lens[b];
  q.idx = a.keep_idx + (size_t)b * a.keep_stride;
  q.pages = a.page_table + (size_t)b * a.max_pages;
  if (q.len < 0 || q.len > a.max_pages * a.page_size || q.new_len < 0 || q.new_len > q.len ||
      q.new_len > a.keep_stride) {
    if (blockIdx.x == 0 && tid == 0) record_status(a.dev_status, MLA_ERR_RANGE);
    return;                                    // the whole cluster
  }

  if (slice == slices) {
    // ---------------------------------------------------------------- attention mass
    float* mass = a.mass + (size_t)b * a.mass_stride;
    constexpr int kRows = kThreads * kMassRows;
    const int rounds = (q.new_len + kRows * cluster - 1) / (kRows * cluster);
    for (int r = 0; r < rounds; ++r) {
      const int j0 = (r * cluster + rank) * kRows + tid;
      int n[kMassRows];
      float v[kMassRows];
#pragma unroll
      for (int k = 0; k < kMassRows; ++k) n[k] = source_of(a, q, j0 + k * kThreads);
#pragma unroll
      for (int k = 0; k < kMassRows; ++k) v[k] = n[k] >= 0 ? *(volatile float*)(mass + n[k]) : 0.f;
      sync();                                  // every value of this round has been read
#pragma unroll
      for (int k = 0; k < kMassRows; ++k)
        if (n[k] >= 0) mass[j0 + k * kThreads] = v[k];
    }
    return;
  }

  // ------------------------------------------------------------------ one slice of the rows
  const int vec = slice * kSliceVecs + tid % kSliceVecs;   // this thread's 16-byte piece of the row
  const bool live = vec < rv;
  const int pair0 = a.rerotate ? (vec * 8 - a.d_c) / 2 : -1;   // its first RoPE pair
  const bool turns = a.rerotate && vec * 8 >= a.d_c && live;
  uint64_t turn[4] = {0, 0, 0, 0};
  if (turns)
#pragma unroll
    for (int k = 0; k < 4; ++k) turn[k] = a.turn[pair0 + k];
  const int row_in_tile = tid / kSliceVecs;
  constexpr int kRowStep = kThreads / kSliceVecs;
  char* pool = reinterpret_cast<char*>(a.pool);
  const int64_t row_bytes = (int64_t)rv * 16;
  const int rounds = (q.new_len + kTileRows * cluster - 1) / (kTileRows * cluster);
  const uint32_t ring0 = smem_u32(ring) + tid * 16;
  auto position = [&](int r, int k) { return (r * cluster + rank) * kTileRows + row_in_tile + k * kRowStep; };

  // the piece of tile r goes to stage r % kStages; returns which of the pieces move
  auto load = [&](int r) {
    if (r < rounds && live) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int n = source_of(a, q, position(r, k));
        if (n < 0) continue;
        const int64_t row = pool_row(a, q, n, page_shift);
        if (row < 0) continue;
        cp_async16(ring0 + (r % kStages) * kTileBytes + k * kThreads * 16, pool + row * row_bytes + vec * 16);
      }
    }
    cp_async_commit();
  };

  for (int r = 0; r < kStages - 1; ++r) load(r);
  for (int r = 0; r < rounds; ++r) {
    load(r + kStages - 1);
    cp_async_wait<kStages - 1>();
    sync();                                    // all reads of tiles <= r, in every CTA, are done
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int j = position(r, k);
      const int n = source_of(a, q, j);
      if (n < 0 || pool_row(a, q, n, page_shift) < 0) continue;
      const int64_t row = pool_row(a, q, j, page_shift);
      if (row < 0) continue;
      uint4 u = *reinterpret_cast<const uint4*>(ring + (r % kStages) * kTileBytes + k * kThreads * 16 + tid * 16);
      if (turns) {
        const int delta = j - n;
        u.x = turn_pair(u.x, delta, turn[0]);
        u.y = turn_pair(u.y, delta, turn[1]);
        u.z = turn_pair(u.z, delta, turn[2]);
        u.w = turn_pair(u.w, delta, turn[3]);
      }
      *reinterpret_cast<uint4*>(pool + row * row_bytes + vec * 16) = u;
    }
  }
}

}  // namespace

cudaError_t launch_cache_compact(const CompactArgs& a, int sms, cudaStream_t stream) {
  const int rv = (a.d_c + a.d_rope) / 8;
  const int slices = (rv + kSliceVecs - 1) / kSliceVecs;
  // CTAs sharing a slice: as many as still give every CTA an SM
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)2 * cluster * slices * a.batch <= sms) cluster *= 2;
  int shift = -1;
  if ((a.page_size & (a.page_size - 1)) == 0)
    for (shift = 0; (1 << shift) < a.page_size; ++shift) {}
  const int smem = kStages * kTileBytes;
  cudaError_t e = cudaFuncSetAttribute(cache_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((slices + (a.mass != nullptr ? 1 : 0)) * cluster, a.batch, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, cache_compact_kernel, a, cluster, shift);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace mla
