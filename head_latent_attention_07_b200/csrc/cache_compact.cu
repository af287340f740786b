// In-place compaction of the paged latent cache: row j of a sequence becomes its row
// keep_idx[j] >= j, the RoPE part turned by the angle of j - keep_idx[j], and the
// token's attention mass moves along.
//
// Every kept row that moves is read once and written once, and nothing is staged in
// memory.  In place that is safe in this order: row j may be overwritten once every
// reader of row j has read it, and its readers sit at positions j' <= j (keep_idx[j'] =
// j >= j').  A sequence's positions are walked upward in tiles, loads run ahead, and a
// tile is written when all reads of it and of the tiles below are done; loads of later
// tiles touch rows that no write so far has reached.
//
// Bytes bind it: two row widths per moved row.  The parallel work comes from splitting
// the rows into slices of columns, which know nothing of each other, and from a
// cluster of CTAs per slice, each taking every cluster-size-th tile.  Every slice has
// its share of the latent and of the RoPE columns, so that all CTAs take the same time
// (turning costs more than moving); the mass moves with the last slice.
//
// A CTA's threads go round by round, a tile each: start the copies of a later tile
// (cp.async into a ring), wait until this round's tile has landed in all CTAs of the
// cluster, write it.  A thread writes the 16-byte pieces that it loaded, the same of every
// tile, so the ring needs no barrier of its own; the latent pieces of a tile come first,
// then those of the RoPE part, so that few warps turn and all their lanes do.  An
// index leads to two page ids and those to the rows: each thread looks up one row of
// every kBatch tiles, and its three dependent loads are a batch apart.  (One bulk copy per
// row, by one thread, was bound by its issue, 40 ns each; roles in warps of their own,
// by the six hand-overs of a tile.)  Measured: 16 x 32768, half kept, 110 us, 5.5 TB/s of read
// and written rows, 0.83 of a copy; without turning 111, and 106 without a mass either.
#include "common.cuh"
#include "evict.h"
#include "sm100.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kPieces = 2;                       // 16-byte pieces of a tile per thread
constexpr int kTileBytes = kThreads * kPieces * 16;   // 16 KB
constexpr int kAhead = 4;                        // rounds from the start of a tile's copies to its write
constexpr int kStages = kAhead + 1;              // ring of tiles: 80 KB, two CTAs per SM
constexpr int kBatch = 4;                        // tiles whose rows are looked up together
constexpr int kMaxTileRows = kThreads / kBatch;
constexpr int kMaxCluster = 16;
constexpr int kMaxSlices = 8;
static_assert(kAhead == kBatch, "a tile's copies start a batch before its write");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// (x, y) of a RoPE pair turned by delta positions; turn = 2^64 times the pair's
// rotation per position as a fraction of a full turn.  delta * turn modulo 2^64 is the
// whole rotation modulo one turn, exactly, so far moves keep their phase.  Its upper 23
// bits, rounded, become a float in [-1/2, 1/2) by their position in it (a conversion would go
// to the unit of the sine and cosine, which is the busy one).  At worst: the angle is off by
// 2 pi 2^-24 from those bits, 2^-23 from the product's rounding and 2^-23.4 from the constant's,
// 2^-20.7 together; the hardware's sine by 2^-21.41 and its cosine by 2^-21.19 on [-pi, pi] (the
// bounds that CUDA documents), 2^-20.8 of the pair's length in one coordinate; the three
// fp32 roundings by 2^-23.  All of it, 2^-19.6 of the length, against the 2^-8 of a bf16 result.
__device__ __forceinline__ uint32_t turn_pair(uint32_t xy, int delta, uint64_t turn) {
  const uint32_t phase = (uint32_t)(((uint64_t)(int64_t)delta * turn) >> 32);
  const float ang = (__uint_as_float(0x3F800000u | ((phase + 0x80000100u) >> 9)) - 1.5f) * 6.283185307f;
  const float c = __cosf(ang), s = __sinf(ang);
  const float x = bf16_lo(xy), y = bf16_hi(xy);
  return pack_bf16x2(x * c - y * s, x * s + y * c);
}

struct Geometry {
  int cluster;                     // CTAs that share a sequence's slice
  int slices;                      // of a row
  int plain_vecs, turn_vecs;       // 16-byte pieces that a slice moves, and moves and turns, at most
  int turn_slice0;                 // the first slice that turns
  int page_shift;                  // log2(page_size), or -1
};

constexpr uint32_t kNone = 0xFFFFFFFFu;

struct CompactSmem {
  uint4 ring[kStages][kThreads * kPieces];
  // the rows of a tile, by batch: pool rows (kNone: the row stays) and the distance
  // moved (0: neither row nor mass moves; the mass lies in no page, so it moves beside a row
  // that stays because a page of it is outside the pool)
  uint32_t src[2][kThreads];
  uint32_t dst[3][kThreads];
  int delta[3][kThreads];
  float mass[3][kThreads];
  uint64_t turn[kMaxRopePairs];
};

__global__ void __launch_bounds__(kThreads, 2)
cache_compact_kernel(const __grid_constant__ CompactArgs a, const __grid_constant__ Geometry geo) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  CompactSmem* sm = reinterpret_cast<CompactSmem*>(smem_raw);
  const int cluster = geo.cluster, shift = geo.page_shift;
  const int tid = threadIdx.x;
  const int rank = (int)cluster_ctarank();
  const int slice = blockIdx.x / cluster;
  const int b = blockIdx.y;
  const bool moves_mass = a.mass != nullptr && slice == geo.slices - 1;

  for (int i = tid; i < a.d_rope / 2; i += kThreads) sm->turn[i] = a.turn[i];
  grid_dependency_wait();
  allow_dependent_launch();
  const int len = a.seq_lens[b], new_len = a.new_lens[b];
  if (len < 0 || len > a.max_pages * a.page_size || new_len < 0 || new_len > len || new_len > a.keep_stride) {
    if (blockIdx.x == 0 && tid == 0) record_status(a.dev_status, MLA_ERR_RANGE);
    return;                                    // the whole cluster
  }

  // this slice: n_plain 16-byte pieces of a row that are only moved, n_turn that are turned
  const int vecs = (a.d_c + a.d_rope) / 8, latent = a.d_c / 8;
  const int plain = a.rerotate ? latent : vecs;
  const int plain0 = slice * geo.plain_vecs, turn0 = plain + (slice - geo.turn_slice0) * geo.turn_vecs;
  const int n_plain = max(0, min(geo.plain_vecs, plain - plain0));
  const int n_turn = slice < geo.turn_slice0 ? 0 : max(0, min(geo.turn_vecs, vecs - turn0));
  const int rows = min(kMaxTileRows, kThreads * kPieces / max(1, n_plain + n_turn));   // of a tile
  const uint32_t row_bytes = vecs * 16;
  float* mass = a.mass + (size_t)b * a.mass_stride;
  const int rounds = (new_len + rows * cluster - 1) / (rows * cluster);

  // this thread's pieces of every tile: the row within the tile (-1: none) and the place in
  // the row
  int row_of[kPieces], turn_of[kPieces];       // its first pair in the turns (-1: only moved)
  char* pool_at[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    int i = tid + k * kThreads, vec = 0;
    row_of[k] = turn_of[k] = -1;
    if (i < rows * n_plain) {
      row_of[k] = i / n_plain;
      vec = plain0 + i % n_plain;
    } else if ((i -= rows * n_plain) < rows * n_turn) {
      row_of[k] = i / n_turn;
      vec = turn0 + i % n_turn;
      turn_of[k] = (vec - latent) * 4;
    }
    pool_at[k] = reinterpret_cast<char*>(a.pool) + vec * 16;
  }
  const uint32_t ring0 = smem_u32(&sm->ring[0][tid]);

  // Indices and page ids by plain loads: this kernel may already be resident while the one before
  // it writes them (the selection, keep_idx), so they are not read-only for its whole life.
  // The row that this thread looks up: row `row` of tile `kBatch * batch + tile`
  const int tile = tid / kMaxTileRows, row = tid % kMaxTileRows;
  const int32_t* idx = a.keep_idx + (size_t)b * a.keep_stride;
  const int32_t* pages = a.page_table + (size_t)b * a.max_pages;
  auto position = [&](int r, int i) { return (r * cluster + rank) * rows + i; };
  auto index_of = [&](int batch) {             // j itself, which stays, where there is no such row
    const int j = position(batch * kBatch + tile, row);
    return row < rows && j < new_len ? idx[j] : j;
  };
  auto page_of = [&](int n) { return pages[shift >= 0 ? n >> shift : n / a.page_size]; };
  auto in_page = [&](int n) { return shift >= 0 ? n & (a.page_size - 1) : n % a.page_size; };
  int n_next = index_of(0);                    // the next batch's index, and what was found with the
  int j_now = 0, n_now = -1;                   // current one's: position, source index (-1: nothing
  int src_page = 0, dst_page = 0;              // moves), page ids and mass
  float mass_now = 0.f;
  auto look_up = [&](int batch) {              // the pages of `batch`, the indices of the one after it
    j_now = position(batch * kBatch + tile, row);
    n_now = n_next;
    if (n_now != j_now && (n_now < j_now || n_now >= len)) record_status(a.dev_status, MLA_ERR_RANGE);
    if (n_now <= j_now || n_now >= len) n_now = -1;
    if (n_now >= 0) {
      src_page = page_of(n_now);
      dst_page = page_of(j_now);
      if (moves_mass) mass_now = __ldcg(mass + n_now);
    }
    n_next = index_of(batch + 1);
  };
  auto resolve = [&](int slot2, int slot3) {   // into these slots of the batches' rings
    uint32_t src = kNone, dst = kNone;
    if (n_now >= 0) {
      if ((uint32_t)src_page < (uint32_t)a.num_pages && (uint32_t)dst_page < (uint32_t)a.num_pages) {
        src = (uint32_t)src_page * a.page_size + in_page(n_now);
        dst = (uint32_t)dst_page * a.page_size + in_page(j_now);
      } else {
        record_status(a.dev_status, MLA_ERR_RANGE);
      }
    }
    sm->src[slot2][tid] = src;
    sm->dst[slot3][tid] = dst;
    sm->delta[slot3][tid] = n_now >= 0 ? j_now - n_now : 0;
    if (moves_mass) sm->mass[slot3][tid] = mass_now;
  };
  // tile r into a stage.  What is read from shared memory is read first: a load does not
  // pass the copies.
  auto load = [&](int r, int stage, const uint32_t* src_of) {
    if (r < rounds) {
      uint32_t src[kPieces];
#pragma unroll
      for (int k = 0; k < kPieces; ++k) src[k] = row_of[k] >= 0 ? src_of[row_of[k]] : kNone;
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        if (src[k] != kNone)
          cp_async16(ring0 + stage * kTileBytes + k * (kThreads * 16), pool_at[k] + (uint64_t)src[k] * row_bytes);
    }
    cp_async_commit();
  };

  look_up(0);
  resolve(0, 0);
  look_up(1);
  resolve(1, 1);
  look_up(2);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kAhead; ++r) load(r, r, &sm->src[0][r * kMaxTileRows]);
  int stage = 0;                               // of tile r
  int now3 = 0;                                // the slot of the batch being written in a ring of three
  for (int batch = 0; batch * kBatch < rounds; ++batch) {
    const int next3 = now3 == 2 ? 0 : now3 + 1, after3 = next3 == 2 ? 0 : next3 + 1;
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      const int r = batch * kBatch + t;
      if (r >= rounds) break;
      load(r + kAhead, stage == 0 ? kStages - 1 : stage - 1, &sm->src[(batch + 1) & 1][t * kMaxTileRows]);
      cp_async_wait<kAhead>();                 // tile r is here
      if (cluster > 1) {
        __syncwarp();
        cluster_arrive_relaxed();              // orders nothing: the copies have landed
      }
      if (t == kBatch - 1) {
        resolve(batch & 1, after3);
        look_up(batch + 3);
        __syncthreads();
      } else if (cluster == 1) {
        __syncthreads();
      }
      if (cluster > 1) cluster_wait();         // all reads of tiles <= r, in every CTA, are done
      const uint32_t* dst_of = &sm->dst[now3][t * kMaxTileRows];
      const int* delta_of = &sm->delta[now3][t * kMaxTileRows];
      uint32_t dst[kPieces];
      uint4 u[kPieces];
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        dst[k] = row_of[k] >= 0 ? dst_of[row_of[k]] : kNone;
        u[k] = sm->ring[stage][tid + k * kThreads];
      }
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        if (dst[k] == kNone) continue;
        if (turn_of[k] >= 0) {
          const uint64_t* turn = sm->turn + turn_of[k];
          const int d = delta_of[row_of[k]];
          u[k].x = turn_pair(u[k].x, d, turn[0]);
          u[k].y = turn_pair(u[k].y, d, turn[1]);
          u[k].z = turn_pair(u[k].z, d, turn[2]);
          u[k].w = turn_pair(u[k].w, d, turn[3]);
        }
        *reinterpret_cast<uint4*>(pool_at[k] + (uint64_t)dst[k] * row_bytes) = u[k];
      }
      if (moves_mass && tid < rows && delta_of[tid] != 0)
        mass[position(r, tid)] = sm->mass[now3][t * kMaxTileRows + tid];
      if (++stage == kStages) stage = 0;
    }
    now3 = next3;
  }
  cp_async_wait<0>();
}

}  // namespace

cudaError_t launch_cache_compact(const CompactArgs& a, int sms, cudaStream_t stream) {
  const int vecs = (a.d_c + a.d_rope) / 8, plain = a.rerotate ? a.d_c / 8 : vecs, turned = vecs - plain;
  Geometry geo;
  // Slices of a row: up to 8 of at least 128 bytes, as many as leave every other SM free of
  // them; then a cluster for each, up to one CTA per SM (two CTAs on an SM slow each other's
  // stores down), or two with few or short sequences, where latency counts, while a CTA has
  // two tiles.  Half kept, us:
  //   sequences x tokens   slices x cluster
  //   64 x 8192            1 x 2  108   2 x 1  104   4 x 1  127
  //   32 x 16384           1 x 4  134   2 x 2  108   4 x 2  128
  //   16 x 32768           2 x 4  134   4 x 2  110   4 x 4  133   8 x 1  147
  //    8 x 32768           4 x 4   72   8 x 2   62   8 x 4   68
  //    4 x 32768           4 x 4   56   8 x 4   44   8 x 8   32
  //    8 x 4096            8 x 2   16   8 x 4   11
  // (64 x 8192 would be 4 % better off with 2 x 1.)  Both numbers only double, so a batch just past
  // a step fills about half of the SMs: 5 x 32768 63 us (2.9 TB/s, against 4.6 at 4 and at 8), 10 x
  // 32768 106 (3.5), 19 x 32768 204 (3.5), 38 x 27584 346 (3.5), 75 x 13952 331 (3.6; 5.9 at 74).
  // "Short" goes by the table's width: 8 x 4096 under a table for 131072 tokens 10.7 us (10.1).
  const int64_t tiles = ((int64_t)a.max_pages * a.page_size + kMaxTileRows - 1) / kMaxTileRows;
  geo.slices = 1;
  while (geo.slices < kMaxSlices && geo.slices * 16 <= plain && (int64_t)4 * geo.slices * a.batch <= sms) geo.slices *= 2;
  int64_t sets = (int64_t)geo.slices * a.batch;
  const int64_t ctas = 4 * sets <= sms || tiles * kMaxTileRows < 8192 ? 2 * sms : sms;
  for (geo.cluster = 1; geo.cluster < kMaxCluster && 2 * geo.cluster * sets <= ctas && 4 * geo.cluster <= tiles;)
    geo.cluster *= 2;
  geo.turn_slice0 = 0;
  if (geo.cluster == kMaxCluster && kMaxCluster * sets < sms) {
    // a sequence alone: SMs are left over for slices of the RoPE part of their own (131072
    // tokens, nine tenths kept: 66 us, against 88)
    geo.plain_vecs = 8;
    geo.turn_vecs = 2;
    geo.turn_slice0 = (plain + 7) / 8;
    geo.slices = geo.turn_slice0 + (turned + 1) / 2;
  } else {
    auto share = [&](int n) { return ((n + geo.slices - 1) / geo.slices + 1) & ~1; };   // whole 32-byte sectors
    geo.plain_vecs = share(plain);
    geo.turn_vecs = share(turned);
  }
  geo.page_shift = -1;
  if ((a.page_size & (a.page_size - 1)) == 0)
    for (geo.page_shift = 0; (1 << geo.page_shift) < a.page_size; ++geo.page_shift) {}
  const int smem = (int)sizeof(CompactSmem);
  cudaError_t e = cudaFuncSetAttribute(cache_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (geo.cluster > 8) e = cudaFuncSetAttribute(cache_compact_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = geo.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(geo.slices * geo.cluster, a.batch, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, cache_compact_kernel, a, geo);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace mla
