// Internal interface between the cache-eviction entry points (evict_api.cu) and
// their kernels: attention mass, selection, compaction.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "decode.h"

namespace mla {

struct MassArgs {
  const uint16_t* q_lat;      // [B, nq, H, R]
  const uint16_t* pool;       // [num_pages, P, R]
  const int32_t* page_table;  // [B, max_pages]
  const int32_t* seq_lens;    // [B]
  const float* lse;           // [B, nq, H]
  const int32_t* mass_lens;   // [B] or null: seq_lens - nq
  float* mass;                // [B, mass_stride]
  int32_t* dev_status;        // or null
  int64_t mass_stride;
  int batch, nq, n_heads, d_c, d_rope, page_size, max_pages, num_pages;
  float scale, decay;
};

struct SelectArgs {
  const float* mass;          // [B, mass_stride]
  const int32_t* seq_lens;    // [B]
  const int32_t* budgets;     // [B]
  int32_t* keep_idx;          // [B, keep_stride]
  int32_t* new_lens;          // [B]
  int32_t* dev_status;        // or null
  int64_t mass_stride, keep_stride;
  int batch, n_sink, n_recent;
};

struct CompactArgs {
  uint16_t* pool;             // [num_pages, P, R]
  const int32_t* page_table;  // [B, max_pages]
  const int32_t* seq_lens;    // [B]
  const int32_t* keep_idx;    // [B, keep_stride]
  const int32_t* new_lens;    // [B]
  float* mass;                // [B, mass_stride] or null
  int32_t* dev_status;        // or null
  int64_t mass_stride, keep_stride;
  int batch, d_c, d_rope, page_size, max_pages, num_pages;
  int rerotate;
  uint64_t turn[kMaxRopePairs];  // theta^(-2i/d_rope) / (2 pi) of pair i, as a fraction of a turn times 2^64
};

// Tensor-core pairs (rows up to 576 wide, pages of a power of two), and any other shape.
bool attn_mass_pair_supported(const MassArgs& a);
cudaError_t launch_attn_mass_pair(const MassArgs& a, int sms, long long spin_limit, cudaStream_t stream);
cudaError_t launch_attn_mass(const MassArgs& a, cudaStream_t stream);
cudaError_t launch_evict_select(const SelectArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_cache_compact(const CompactArgs& a, int sms, cudaStream_t stream);

}  // namespace mla
