// Attention mass of the cached tokens, any supported shape (mma.sync).
//
//   w[b][n]    = sum over query rows (i, h) that see key n of exp(scale * q . row_n - lse)
//   mass[b][n] = decay * mass[b][n] + w[b][n]
// The lse of the step's attention is final, so a key's weight needs no running
// maximum and no rescaling: one score product, one exponential and one add per
// (query row, key).  Keys are the rows of the product and query rows its columns,
// so that the sum over query rows stays inside a thread quad and every mass value
// is summed by one warp in a fixed order (no atomics: results do not depend on
// the schedule).
//
// One CTA takes 128 keys of a sequence, 16 per warp, and walks the nq * H query
// rows in blocks of 64 columns, each staged in shared memory.  The key rows go from
// global memory straight into fragments (16-byte pieces, see mma_frag.cuh), two slices ahead
// of their products, and are read again from L2 for every block.
//
// Latency binds it, of the keys' loads and of the staging, at 16 warps per SM: 16 x 32768
// tokens 640 wide take 497 us at 128 heads (173 TFLOP/s) and 174 us at 16 (3.9 TB/s).  With
// each slice loaded when it was needed it was 848 and 260 us, with the query rows staged
// through registers 551 and 181.  It is for the shapes that the CTA-pair kernel does not
// take: rows over 576, other page sizes.
#include "common.cuh"
#include "evict.h"
#include "mma_frag.cuh"
#include "sm100.cuh"

namespace mla {

namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 128;       // keys per CTA, 16 per warp
constexpr int kCols = 64;        // query rows per block
constexpr int kAhead = 2;        // 32-column slices of the keys on their way (114 registers, no spills; 4 spilled)
constexpr float kLog2e = 1.4426950408889634f;

// Bytes of one staged query row: whole 32-column slices, and 64 bytes modulo 128,
// so that the 16-byte reads of two neighbouring rows fall into different banks.
__host__ __device__ inline int q_row_bytes(int row) { return (row * 2 + 127) / 128 * 128 + 64; }

// 16 bytes from src to shared memory, or zeros (`any` is then a valid address, not read)
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, const void* any, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(in ? src : any), "r"(in ? 16 : 0)
               : "memory");
}

__global__ void __launch_bounds__(kThreads)
attn_mass_kernel(const MassArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  float* lse2 = reinterpret_cast<float*>(smem);            // [kCols], log2 units
  unsigned char* q_s = smem + kCols * sizeof(float);       // [kCols][q_row_bytes]
  const int R = a.d_c + a.d_rope;
  const int rv = R / 8;                                    // 16-byte pieces per row
  const uint32_t q_dst = sm100::smem_u32(q_s);
  const int slices = (R + 31) / 32;
  const int q_bytes = q_row_bytes(R);
  const int rows_total = a.nq * a.n_heads;
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, quad = lane & 3;

  grid_dependency_wait();
  allow_dependent_launch();
  const int len = a.seq_lens[b];
  if (len < a.nq || len > a.max_pages * a.page_size) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_status(a.dev_status, MLA_ERR_RANGE);
    return;
  }
  if ((int)blockIdx.x * kKeys >= len) return;

  // this thread's two keys, and their rows (null: past the end, or a bad page)
  int n[2];
  const uint4* src[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    n[j] = blockIdx.x * kKeys + warp * 16 + g + 8 * j;
    src[j] = nullptr;
    if (n[j] < len) {
      const int id = a.page_table[(size_t)b * a.max_pages + n[j] / a.page_size];
      if (id >= 0 && id < a.num_pages)
        src[j] = reinterpret_cast<const uint4*>(a.pool + ((size_t)id * a.page_size + n[j] % a.page_size) * R);
      else if (quad == 0)
        record_status(a.dev_status, MLA_ERR_RANGE);
    }
  }
  float w[2] = {0.f, 0.f};
  const float sl2 = a.scale * kLog2e;

  for (int c0 = 0; c0 < rows_total; c0 += kCols) {
    const int cols = min(kCols, rows_total - c0);
    const int tiles = (cols + 7) >> 3;
    // the pieces of the next kAhead slices are on their way while these are multiplied
    uint4 ahead[kAhead][2];
    auto fetch = [&](int s, uint4 (&r)[2]) {
      const int v = s * 4 + quad;
#pragma unroll
      for (int j = 0; j < 2; ++j) r[j] = src[j] != nullptr && v < rv ? src[j][v] : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(k, ahead[k]);
    if (c0 > 0) __syncthreads();                           // the previous block has been read
    const uint16_t* qb = a.q_lat + ((size_t)b * rows_total + c0) * R;
    const int per_row = slices * 4;                        // pieces per staged row, zeros past R
    for (int c = warp; c < tiles * 8; c += kThreads / 32)
      for (int v = lane; v < per_row; v += 32)
        cp_async16_or_zero(q_dst + c * q_bytes + v * 16, qb + (size_t)c * R + v * 8, qb, c < cols && v < rv);
    bool keyless = false;                                  // lse = -inf: the row saw no key
    if ((int)threadIdx.x < cols) {
      const float l = a.lse[(size_t)b * rows_total + c0 + threadIdx.x] * kLog2e;
      lse2[threadIdx.x] = l;
      keyless = l == -INFINITY;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    const bool some_keyless = __syncthreads_or(keyless);

    float acc[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[t][k] = 0.f;
    for (int s0 = 0; s0 < slices; s0 += kAhead) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (s0 + k < slices) {
          const uint4 ra = ahead[k][0], rb = ahead[k][1];
          fetch(s0 + k + kAhead, ahead[k]);
#pragma unroll
          for (int t = 0; t < 8; ++t)
            if (t < tiles)
              mma_k32(acc[t], ra, rb, *reinterpret_cast<const uint4*>(q_s + (t * 8 + g) * q_bytes + ((s0 + k) * 4 + quad) * 16));
        }
      }
    }

    // key n is seen by query i when n <= len - nq + i: by query rows from H * (n - (len - nq)) on.
    // A row that saw no key gives nothing, whatever its query holds; a block of queries without
    // such a row does not look for them (looking in every block: 524 us against 497).
    auto add = [&](auto look) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int first = max(0, n[j] - (len - a.nq)) * a.n_heads - c0;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int col = t * 8 + quad * 2 + k;
            if (col < cols && col >= first && (!look() || lse2[col] != -INFINITY))
              w[j] += sm100::ex2(fmaf(acc[t][j * 2 + k], sl2, -lse2[col]));
          }
      }
    };
    if (some_keyless) add([] { return true; });
    else add([] { return false; });
  }

#pragma unroll
  for (int j = 0; j < 2; ++j) {
    w[j] += __shfl_xor_sync(0xffffffffu, w[j], 1);
    w[j] += __shfl_xor_sync(0xffffffffu, w[j], 2);
    if (quad == 0 && src[j] != nullptr) {
      float* m = a.mass + (size_t)b * a.mass_stride + n[j];
      const int old_len = a.mass_lens != nullptr ? a.mass_lens[b] : len - a.nq;
      *m = a.decay != 0.f && n[j] < old_len ? fmaf(a.decay, *m, w[j]) : w[j];
    }
  }
}

}  // namespace

cudaError_t launch_attn_mass(const MassArgs& a, cudaStream_t stream) {
  const int smem = kCols * (int)sizeof(float) + kCols * q_row_bytes(a.d_c + a.d_rope);
  // always the most (rows of 512 + 256): calls of other sizes may be on their way from other
  // host threads
  cudaError_t e = cudaFuncSetAttribute(attn_mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kCols * (int)sizeof(float) + kCols * q_row_bytes(768));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)a.max_pages * a.page_size + kKeys - 1) / kKeys), a.batch);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_mass_kernel, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace mla
