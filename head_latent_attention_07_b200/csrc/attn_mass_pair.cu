// Attention mass of the cached tokens on CTA pairs with 2-SM tensor-core
// instructions (tcgen05 .cta_group::2, TMEM, TMA).
//
// Shape: cache rows up to 576 wide (in blocks of 64 columns, the last one filled up with
// zeros by the loads), pages of 8 to 256 tokens, a power of two.  The product is
// transposed against the decode kernel's: the keys are its rows and the query
// rows its columns, S[256 x NT] = K[256 x R] . Q[NT x R]^T, so a key's scores lie in
// one TMEM lane and one thread adds up its weights: no reduction across threads,
// no running maximum (the lse is final) and a fixed order of the sum.
//
//   tile    256 keys of a sequence, 128 per CTA of the pair
//   group   NT query rows (128 or 256), half of them in each CTA's shared memory
// One of the two stays in shared memory while the other goes by
// TMA through a ring of blocks, each done with after its four MMAs; a resident block is
// reloaded as soon as its last MMAs are through.
//   one group   (nq * H <= 256: decode) the group stays, the keys stream: HBM binds, at R =
//               576 with 295 KB per tile and pair, 6700 cycles at the pair's share of the
//               bandwidth, against 4600 of the tensor pipe at NT = 256
//   few groups  the same, the worker taking kSubTiles tiles at a time through all groups,
//               so that the groups after the first find the keys in L2
//   many groups the tile stays and the groups stream.  Both forms are bound by what an SM
//               takes in from L2 (about 30 B/clk against the 32 that the tensor pipe would
//               use): per group and tile 147 + 147 / 4 KB with the group resident, 147 + 147 /
//               groups with the tile resident, so the tile is from more than 4 groups on.
//
// Page ids come by plain loads: this kernel may already be resident while the one before it on
// the stream writes the table, so it is not read-only for the kernel's whole life.
//
// TMEM: two accumulators of NT columns, so that the sum over one tile runs beside the
// next tile's MMAs.  Warps (256 threads): 0 loads (TMA), 1 owns TMEM and, in CTA 0, issues
// the MMAs, 2 brings the groups' lse, 4-7 sum (warp w reads TMEM lanes 32 (w & 3) and
// on).  Every mbarrier wait is bounded: on time-out the kernel records MLA_ERR_TIMEOUT,
// drains its MMAs and ends.
//
// Measured, 128 heads, R = 576, a dozen calls back to back in a graph: 16 x 32768 102 us (6.0
// TB/s, 0.91 of a copy); 64 ragged, 2 tokens each 555 us (4.5 TB/s and 1.13 PFLOP/s: both
// pipes, at 1.4 GHz); 2 x 32768, 32 tokens each 210 to 219 us (1.41 to 1.47 PFLOP/s).  Loops of
// calls from Python run under the power cap: 112 to 120, 570 to 615 and 240 to 246 us, by the box.
#include <cuda.h>

#include "common.cuh"
#include "evict.h"
#include "sm100.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr int kTileKeys = 256;
constexpr int kMaxBlocks = 9;                    // 64-column blocks of a 576-wide row
constexpr int kMaxStages = 12;                   // of the ring
constexpr int kMaxSmem = 232448;
constexpr int kKeyBytes = 128 * 128;             // [128 keys x 64 columns] bf16, 128-byte swizzle
constexpr int kSubTiles = 4;                     // tiles per pass over the groups: 74 pairs hold 87 MB of keys in L2
constexpr long long kDrainCycles = 1ll << 24;

// kKeys: the tile is resident and the groups stream, else the other way round
template <int NT, bool kKeys>
struct Layout {
  static constexpr int kQueryBytes = NT / 2 * 128;                   // one block of this CTA's half of the group
  static constexpr int kResBytes = kKeys ? kKeyBytes : kQueryBytes;  // a block of the resident operand
  static constexpr int kRingBytes = kKeys ? kQueryBytes : kKeyBytes; // ... of the streaming one
  // lse (fp32 [NT], log2 units), barriers, the resident blocks, the ring; 1 KB alignment slack
  static constexpr int kOffBar = NT * 4;
  static constexpr int kOffRes = 2048;
  static int stages(int blocks) {
    const int n = (kMaxSmem - 1024 - kOffRes - blocks * kResBytes) / kRingBytes;
    return n < kMaxStages ? n : kMaxStages;
  }
  static int bytes(int blocks) { return 1024 + kOffRes + blocks * kResBytes + stages(blocks) * kRingBytes; }
};

struct Bars {
  uint64_t ring_full[kMaxStages];   // CTA 0: both CTAs' blocks landed in the stage (2 arrivals + bytes)
  uint64_t ring_empty[kMaxStages];  // both: the MMAs are done with the stage
  uint64_t res_full[kMaxBlocks];    // CTA 0: both CTAs' blocks of the resident operand landed
  uint64_t res_empty[kMaxBlocks];   // both: the MMAs are done with that block
  uint64_t acc_full[2];  // both: a tile's scores are in TMEM
  uint64_t acc_empty[2]; // CTA 0: the 8 summing warps of the pair have read them
  uint64_t lse_full;     // local: a group's lse is in shared memory
  uint64_t lse_empty;    // local: the 4 summing warps have read the last group's
  uint64_t drain;        // both: every MMA issued has completed
  uint32_t tmem_base;
  int abort;
  // beside the lse: the group's rows that saw a key (lse > -inf), 32 a word, and the full words
  uint32_t has_key[8], full_words;
};
static_assert(Layout<256, false>::kOffBar + sizeof(Bars) <= Layout<256, false>::kOffRes, "barrier area");

struct PairMassParams {
  MassArgs m;
  int rows_total;        // nq * H
  int groups;
  int blocks, stages;    // 64-column blocks of a row, stages of the ring
  int page_shift;        // log2(page_size)
  int box_rows;          // keys per TMA box: a page, or half of a 256-token one
  float scale_log2;
  long long spin_limit;
};

// A sequence's tiles; 0 when its length is out of range.
__device__ __forceinline__ int seq_tiles(const MassArgs& a, int b, int* len) {
  *len = a.seq_lens[b];
  return *len < a.nq || *len > a.max_pages * a.page_size ? 0 : (*len + kTileKeys - 1) / kTileKeys;
}

// Worker w's share of the tiles: those of all sequences end to end, in equal parts.  Each
// warp finds it by itself (two passes over the lengths, 32 at a time), so that the start
// needs no barrier after the lengths are known.
struct Share {
  int b, tile, count;    // first sequence, first tile, tiles
};
__device__ __forceinline__ Share find_share(const MassArgs& a, int w, int workers, int lane) {
  auto tiles_of = [&](int b) {
    int len;
    return b < a.batch ? seq_tiles(a, b, &len) : 0;
  };
  int total = 0;
  for (int base = 0; base < a.batch; base += 32) total += __reduce_add_sync(0xffffffffu, tiles_of(base + lane));
  const int t0 = (int)((long long)total * w / workers);
  Share s = {0, 0, (int)((long long)total * (w + 1) / workers) - t0};
  int carry = 0;
  for (int base = 0; base < a.batch && s.count > 0; base += 32) {
    const int v = tiles_of(base + lane);
    int end = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    end += carry;
    const uint32_t hit = __ballot_sync(0xffffffffu, end - v <= t0 && t0 < end);
    if (hit != 0) {
      const int at = __ffs(hit) - 1;
      s.b = base + at;
      s.tile = t0 - __shfl_sync(0xffffffffu, end - v, at);
      break;
    }
    carry = __shfl_sync(0xffffffffu, end, 31);
  }
  return s;
}

// One accumulator's worth of work; every role walks the same ones in the same order.
struct Item {
  int b, len, tile, group;
  bool first, last;      // with what is resident
};
template <bool kKeys>
struct Cursor {
  const PairMassParams& p;
  int b, tile, left;     // next sequence and tile, tiles left of this worker's share
  int len = 0, sub0 = 0, sub1 = 0, t = 0, g = 0;
  __device__ Cursor(const PairMassParams& p_, const Share& s) : p(p_), b(s.b), tile(s.tile), left(s.count) {}
  __device__ bool next(Item* it) {
    // through the groups of a tile (kKeys), or through the tiles [sub0, sub1) of a group
    bool done;
    if (kKeys) {
      done = sub1 == 0 || ++g == p.groups;
    } else if ((done = t == sub1)) {
      t = sub0;
      done = ++g >= p.groups || sub1 == 0;
    }
    if (done) {
      if (left == 0) return false;
      int n;
      while (tile >= (n = seq_tiles(p.m, b, &len))) {
        // (met only when another stream changes the lengths meanwhile: the roles' waits on one
        // another then run out)
        if (++b == p.m.batch) return false;
        tile = 0;
      }
      sub0 = t = tile;
      sub1 = kKeys ? tile + 1 : min(n, tile + left);
      if (!kKeys && p.groups > 1) sub1 = min(sub1, tile + kSubTiles);
      left -= sub1 - sub0;
      tile = sub1;
      g = 0;
    }
    it->b = b;
    it->len = len;
    it->tile = t;
    it->group = g;
    if (kKeys) {
      it->first = g == 0;
      it->last = g == p.groups - 1;
    } else {
      it->first = t == sub0;
      it->last = ++t == sub1;
    }
    return true;
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t is_leader;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is_leader));
  return is_leader != 0;
}

template <int NT, bool kKeys>
__global__ void __launch_bounds__(kThreads, 1)
attn_mass_pair_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tp,
                      const __grid_constant__ PairMassParams prm) {
  using L = Layout<NT, kKeys>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* lse2 = reinterpret_cast<float*>(sm);
  unsigned char* res_s = sm + L::kOffRes;
  unsigned char* ring_s = res_s + prm.blocks * L::kResBytes;
  Bars* bar = reinterpret_cast<Bars*>(sm + L::kOffBar);
  volatile int* abort_flag = &bar->abort;

  const MassArgs& a = prm.m;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t c = cluster_ctarank();
  const int w = blockIdx.x >> 1, workers = gridDim.x >> 1;
  const long long lim = prm.spin_limit;
  int32_t* status = a.dev_status;
  const int blocks = prm.blocks, stages = prm.stages;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&bar->ring_full[s], 2);
      mbar_init(&bar->ring_empty[s], 1);
    }
    for (int s = 0; s < kMaxBlocks; ++s) {
      mbar_init(&bar->res_full[s], 2);
      mbar_init(&bar->res_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->acc_full[s], 1);
      mbar_init(&bar->acc_empty[s], 8);
    }
    mbar_init(&bar->lse_full, 1);
    mbar_init(&bar->lse_empty, 4);
    mbar_init(&bar->drain, 1);
    bar->abort = 0;
    fence_mbar_init();
    tma_prefetch(&tq);
    tma_prefetch(&tp);
  }
  if (warp == 1) {
    tmem_alloc_pair(&bar->tmem_base, 2 * NT);
    tmem_relinquish_pair();
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();        // barriers and TMEM of both CTAs ready before any remote traffic
  tc_fence_after();
  // setup above touches no input: the predecessor on the stream may still run
  grid_dependency_wait();
  allow_dependent_launch();
  if (blockIdx.x == 0) {
    int len;
    for (int b = threadIdx.x; b < a.batch; b += kThreads)
      if (seq_tiles(a, b, &len) == 0) record_status(status, MLA_ERR_RANGE);
  }
  const Share share = find_share(a, w, workers, lane);
  const uint32_t tmem = bar->tmem_base;
  auto wwait = [&](uint64_t* b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, status, lim));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ queries and keys (TMA)
    const uint32_t ring_full0 = mapa(smem_u32(&bar->ring_full[0]), 0);
    const uint32_t res_full0 = mapa(smem_u32(&bar->res_full[0]), 0);
    const int oob_row = a.num_pages << prm.page_shift;   // a box starting here lies outside the pool: zero fill
    // Lane j looks after the j-th box of this CTA's keys (one lane for all, with the rows
    // shuffled to it, held the stream up: 116 against 105 us at 16 x 32768).  The page ids
    // of a tile are fetched while the tile before is loaded.  No eviction policy: marking the
    // keys as first to evict measured 107.
    const int n_boxes = 128 / prm.box_rows, box_bytes = prm.box_rows * 128;
    const bool has_box = lane < n_boxes;
    const int box_key = (int)c * 128 + lane * prm.box_rows;      // its first key within a tile
    Cursor<kKeys> cur(prm, share);
    Item next;
    int next_id = 0;
    auto fetch = [&]() -> bool {
      if (!cur.next(&next)) return false;
      const int n = next.tile * kTileKeys + box_key;
      if (has_box && n < next.len) next_id = a.page_table[(size_t)next.b * a.max_pages + (n >> prm.page_shift)];
      return true;
    };
    int s = 0, ri = -1;                          // the ring's stage, resident operands begun
    uint32_t lap = 0;                            // times round the ring
    bool ok = true, more = fetch();
    while (ok && more) {
      const Item it = next;
      if (it.first) ++ri;
      const int n = it.tile * kTileKeys + box_key;
      int y = oob_row;
      if (has_box && n < it.len) {
        if (next_id >= 0 && next_id < a.num_pages)
          y = (next_id << prm.page_shift) + (n & (a.page_size - 1));
        else
          record_status(status, MLA_ERR_RANGE);
      }
      more = fetch();
      const int qrow = it.b * prm.rows_total + it.group * NT + (int)c * (NT / 2);
      auto load_keys = [&](unsigned char* dst, int blk, uint32_t full) {
        if (lane == 0) mbar_arrive_expect_tx_cluster(full, kKeyBytes);
        __syncwarp();
        if (has_box) tma_load_2d_pair(dst + lane * box_bytes, &tp, 64 * blk, y, full);
      };
      auto load_query = [&](unsigned char* dst, int blk, uint32_t full) {
        if (lane != 0) return;
        mbar_arrive_expect_tx_cluster(full, L::kQueryBytes);
        tma_load_2d_pair(dst, &tq, 64 * blk, qrow, full);
      };
      for (int blk = 0; blk < blocks; ++blk) {
        if (it.first) {
          if (ri > 0 && !(ok = wwait(&bar->res_empty[blk], (ri - 1) & 1))) break;
          unsigned char* dst = res_s + blk * L::kResBytes;
          if (kKeys) load_keys(dst, blk, res_full0 + 8 * blk);
          else load_query(dst, blk, res_full0 + 8 * blk);
          __syncwarp();
        }
        if (lap > 0 && !(ok = wwait(&bar->ring_empty[s], (lap - 1) & 1))) break;
        unsigned char* dst = ring_s + s * L::kRingBytes;
        if (kKeys) load_query(dst, blk, ring_full0 + 8 * s);
        else load_keys(dst, blk, ring_full0 + 8 * s);
        __syncwarp();
        if (++s == stages) { s = 0; ++lap; }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (CTA 0)
    if (c == 0) {
      const uint32_t idesc = idesc_bf16_f32(256, NT, 0, 0);
      const uint32_t res = smem_u32(res_s), ring = smem_u32(ring_s);
      Cursor<kKeys> cur(prm, share);
      Item it;
      int s = 0, ri = -1, t = 0;
      uint32_t lap = 0;
      bool ok = true;
      while (ok && cur.next(&it)) {
        if (it.first) ++ri;
        if (t >= 2 && !wwait(&bar->acc_empty[t & 1], ((t >> 1) - 1) & 1)) break;
        const uint32_t d = tmem + (t & 1) * NT;
        for (int blk = 0; blk < blocks; ++blk) {
          if (it.first && !(ok = wwait(&bar->res_full[blk], ri & 1))) break;
          if (!(ok = wwait(&bar->ring_full[s], lap & 1))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t res_blk = res + blk * L::kResBytes, ring_blk = ring + s * L::kRingBytes;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              const uint64_t da = smem_desc((kKeys ? res_blk : ring_blk) + ks * 32, 16, 1024, kSwizzle128);
              const uint64_t db = smem_desc((kKeys ? ring_blk : res_blk) + ks * 32, 16, 1024, kSwizzle128);
              mma_bf16_pair(d, da, db, idesc, blk + ks > 0 ? 1u : 0u);
            }
            mma_commit_pair(&bar->ring_empty[s]);
            if (it.last) mma_commit_pair(&bar->res_empty[blk]);
            if (blk == blocks - 1) mma_commit_pair(&bar->acc_full[t & 1]);
          }
          __syncwarp();
          if (++s == stages) { s = 0; ++lap; }
        }
        ++t;
      }
      // every MMA and every earlier commit has completed before TMEM and shared memory go away
      if (elect_one()) mma_commit_pair(&bar->drain);
      __syncwarp();
    }
    if (lane == 0) mbar_wait_drain(&bar->drain, 0, kDrainCycles + lim);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ lse of a group's query rows
    Cursor<kKeys> cur(prm, share);
    Item it;
    int gi = 0;
    while (cur.next(&it)) {
      if (!kKeys && !it.first) continue;         // the same group still
      const int cols = prm.rows_total - it.group * NT;
      const float* src = a.lse + (size_t)it.b * prm.rows_total + it.group * NT;
      float l[NT / 32];
#pragma unroll
      for (int i = 0; i < NT / 32; ++i)
        l[i] = i * 32 + lane < cols ? src[i * 32 + lane] * 1.4426950408889634f : -INFINITY;
      if (gi > 0 && !wwait(&bar->lse_empty, (gi - 1) & 1)) break;
#pragma unroll
      for (int i = 0; i < NT / 32; ++i) lse2[i * 32 + lane] = l[i];
      uint32_t full_words = 0;
#pragma unroll
      for (int i = 0; i < NT / 32; ++i) {
        const uint32_t has_key = __ballot_sync(0xffffffffu, l[i] != -INFINITY);
        if (lane == 0) bar->has_key[i] = has_key;
        full_words |= has_key == ~0u ? 1u << i : 0u;
      }
      if (lane == 0) bar->full_words = full_words;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->lse_full);
      ++gi;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ weights and their sum
    const uint32_t acc_empty0 = mapa(smem_u32(&bar->acc_empty[0]), 0);
    const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
    const int row = (int)c * 128 + (warp & 3) * 32 + lane;   // this thread's key within a tile
    // The key's page id and its mass so far are fetched an item ahead: their latency would
    // otherwise add to each tile's sum.
    Cursor<kKeys> cur(prm, share);
    Item next;
    int next_id = -1;
    float next_mass = 0.f;
    auto fetch = [&]() -> bool {
      if (!cur.next(&next)) return false;
      const int n = next.tile * kTileKeys + row;
      if (n < next.len) {
        next_id = a.page_table[(size_t)next.b * a.max_pages + (n >> prm.page_shift)];
        if (next.group == 0 ? a.decay != 0.f : !kKeys) next_mass = a.mass[(size_t)next.b * a.mass_stride + n];
      }
      return true;
    };
    int t = 0, gi = -1;
    uint32_t full_words = 0;
    float sum_so_far = 0.f;                      // what the key has collected
    bool more = fetch();
    while (more) {
      const Item it = next;
      const int n = it.tile * kTileKeys + row;
      const bool live = n < it.len && next_id >= 0 && next_id < a.num_pages;
      if (it.group == 0) {
        const int old_len = a.mass_lens != nullptr ? a.mass_lens[it.b] : it.len - a.nq;
        sum_so_far = a.decay != 0.f && n < old_len ? a.decay * next_mass : 0.f;
      } else if (!kKeys && !(it.first && it.last)) {
        sum_so_far = next_mass;                  // the earlier groups' sum; of a lone tile, still here
      }
      more = fetch();
      const int cols = min(NT, prm.rows_total - it.group * NT);
      if (kKeys || it.first) {
        ++gi;
        if (!wwait(&bar->lse_full, gi & 1)) break;
        full_words = bar->full_words;
      }
      if (!wwait(&bar->acc_full[t & 1], (t >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t acc = lanes + (t & 1) * NT;
      // key n is seen by query i when n <= len - nq + i: by query rows from H * (n - (len - nq)) on
      const int first = max(0, n - (it.len - a.nq)) * a.n_heads - it.group * NT;
      const bool all = __all_sync(0xffffffffu, first <= 0);
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int c0 = 0; c0 < cols; c0 += 32) {
        float v[32];
        tmem_ld32(acc + c0, v);
        tmem_wait_ld();
        // A row that saw no key gives nothing, whatever its query holds (padding: NaN too), so it is
        // left out and not multiplied away.
        if (all && (full_words >> (c0 / 32) & 1)) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 l = *reinterpret_cast<const float4*>(lse2 + c0 + i);
            sum[0] += ex2(fmaf(v[i], prm.scale_log2, -l.x));
            sum[1] += ex2(fmaf(v[i + 1], prm.scale_log2, -l.y));
            sum[2] += ex2(fmaf(v[i + 2], prm.scale_log2, -l.z));
            sum[3] += ex2(fmaf(v[i + 3], prm.scale_log2, -l.w));
          }
        } else {
          const uint32_t rows = bar->has_key[c0 / 32];
          const uint32_t seen = first <= c0 ? rows : first >= c0 + 32 ? 0 : rows & (~0u << (first - c0));
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float e = ex2(fmaf(v[i], prm.scale_log2, -lse2[c0 + i]));
            if (seen >> i & 1) sum[i & 3] += e;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cluster(acc_empty0 + 8 * (t & 1));
        if (kKeys || it.last) mbar_arrive(&bar->lse_empty);
      }
      sum_so_far += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (live && (!kKeys || it.last)) a.mass[(size_t)it.b * a.mass_stride + n] = sum_so_far;
      ++t;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // after a time-out, copies this CTA issued may still be in flight (their
    // completion is counted in CTA 0): give them time to land before exiting
    const long long t0 = clock64();
    while (clock64() - t0 < 200000) __nanosleep(1000);
  }
  cluster_sync();        // the peer no longer touches this CTA's shared memory or TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * NT);
  }
}

template <int NT, bool kKeys>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tp, PairMassParams prm, int workers,
                   cudaStream_t stream) {
  prm.stages = Layout<NT, kKeys>::stages(prm.blocks);
  const int smem = Layout<NT, kKeys>::bytes(prm.blocks);
  // always the most: calls of other sizes may be on their way from other host threads
  cudaError_t e = cudaFuncSetAttribute(attn_mass_pair_kernel<NT, kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * workers, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, attn_mass_pair_kernel<NT, kKeys>, tq, tp, prm);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

// Wherever its loads can go: against the mma.sync kernel (pages of 48 tokens), 13.2 and 13.8 us
// at 8 x 4096 with 32 heads, 99 and 458 at 16 x 32768 with 128.
bool attn_mass_pair_supported(const MassArgs& a) {
  return a.d_c + a.d_rope <= 64 * kMaxBlocks && a.page_size >= 8 && (a.page_size & (a.page_size - 1)) == 0 &&
         (int64_t)a.num_pages * a.page_size < INT32_MAX;   // a load's coordinates are 32 bits, its row past the pool too
}

cudaError_t launch_attn_mass_pair(const MassArgs& a, int sms, long long spin_limit, cudaStream_t stream) {
  PairMassParams prm;
  prm.m = a;
  prm.rows_total = a.nq * a.n_heads;
  const int nt = prm.rows_total > 128 ? 256 : 128;
  prm.groups = (prm.rows_total + nt - 1) / nt;
  prm.scale_log2 = a.scale * 1.4426950408889634f;
  prm.spin_limit = spin_limit;
  const int row = a.d_c + a.d_rope;
  prm.blocks = (row + 63) / 64;
  prm.page_shift = 0;
  while ((1 << prm.page_shift) < a.page_size) ++prm.page_shift;
  prm.box_rows = a.page_size < 128 ? a.page_size : 128;
  CUtensorMap tq, tp;
  if (!encode_rows(&tq, a.q_lat, (uint64_t)a.batch * prm.rows_total, row, nt / 2) ||
      !encode_rows(&tp, a.pool, (uint64_t)a.num_pages * a.page_size, row, prm.box_rows))
    return cudaErrorInvalidValue;
  // one pair per two SMs, but no more pairs than the batch can have tiles
  const int64_t tiles = a.batch * (((int64_t)a.max_pages * a.page_size + kTileKeys - 1) / kTileKeys);
  const int workers = (int)(tiles < sms / 2 ? tiles : sms / 2);
  if (nt == 128) return launch<128, false>(tq, tp, prm, workers, stream);
  // 16 groups over 2 x 32768 keys: 207 us with the tile resident, 232 with the group
  return prm.groups > kSubTiles ? launch<256, true>(tq, tp, prm, workers, stream)
                                : launch<256, false>(tq, tp, prm, workers, stream);
}

}  // namespace mla
