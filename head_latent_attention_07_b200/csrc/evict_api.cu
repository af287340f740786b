// C ABI of the cache-eviction calls: argument validation and launches.  The
// declarations and the contract of every entry point are in include/mla.h.
#include <math.h>
#include <stdlib.h>

#include "../../include/mla.h"
#include "evict.h"
#include "plan.cuh"

namespace {

constexpr int32_t kMaxNq = 1024;                 // the bounds of the decode calls, whose rows these are
constexpr int64_t kMaxTokens = 1 << 18;
constexpr int64_t kMaxLength = 1 << 30;          // tokens of one sequence: tiles past its end keep 32-bit indices

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// What the cache rows of these calls need of the dimensions: the bounds of the decode
// calls on the row and the page (the projections' widths are not looked at).
int check_cache_dims(const mla_dims* d) {
  if (d == nullptr) return MLA_ERR_INVALID_ARG;
  if (d->n_heads < 1 || d->d_c < 1 || d->d_rope < 0 || d->qk_nope < 1 || d->page_size < 1)
    return MLA_ERR_INVALID_ARG;
  if (d->d_rope == 0) return MLA_ERR_UNSUPPORTED;
  if (d->n_heads > 128 || d->d_c > 512 || d->d_c % 8 || d->d_rope > 256 || d->d_rope % 8 || d->page_size > 256)
    return MLA_ERR_UNSUPPORTED;
  if (!(d->softmax_scale >= 0.f) || isinf(d->softmax_scale) || !(d->rope_theta >= 0.f) || isinf(d->rope_theta))
    return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

int check_cache_shape(const mla_dims* d, int32_t batch, int32_t max_pages, int32_t num_pages) {
  if (batch < 1 || max_pages < 1 || num_pages < 1) return MLA_ERR_INVALID_ARG;
  if (batch > mla::kMaxBatch || (int64_t)max_pages * d->page_size > kMaxLength) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? MLA_OK : mla::record_cuda_error(e); }

int device_sms(int* sms) {
  int dev = 0;
  const int st = cuda_status(cudaGetDevice(&dev));
  if (st != MLA_OK) return st;
  return cuda_status(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
}

// Rows of `width` bytes, `stride` bytes apart, at p (null: not given).
struct Buffer {
  const void* p;
  __int128 rows, width, stride;                  // a row stride may be as large as 64 bits hold
};
Buffer dense(const void* p, int64_t rows, int64_t width, int size) {
  return {p, 1, (__int128)rows * width * size, (__int128)rows * width * size};
}
Buffer strided(const void* p, int64_t rows, int64_t width, int64_t stride, int size) {
  return {p, rows, (__int128)width * size, (__int128)stride * size};
}
// The kernels read lengths, indices and masses more than once, in several CTAs: a buffer that
// is written while others still read it would leave them with different sizes.  True when a
// row of `out` shares a byte with one of the dense `others`; between its rows they may lie.
template <int N>
bool overlaps(const Buffer& out, const Buffer (&others)[N]) {
  if (out.p == nullptr) return false;
  const __int128 p = reinterpret_cast<uintptr_t>(out.p);
  for (const Buffer& o : others) {
    if (o.p == nullptr) continue;
    const __int128 q = reinterpret_cast<uintptr_t>(o.p);
    if (q >= p + (out.rows - 1) * out.stride + out.width || p >= q + o.width) continue;   // as a rule
    const __int128 row = q < p + out.width ? 0 : (q - p - out.width) / out.stride + 1;   // the first that ends behind q
    if (row < out.rows && p + row * out.stride < q + o.width) return true;
  }
  return false;
}

// Spin budget of each bounded wait, as for the decode calls: kSpinLimitCycles, or the
// environment variable MLA_SPIN_LIMIT (cycles, >= 0) when it is set.
long long spin_limit_cycles() {
  const char* e = getenv("MLA_SPIN_LIMIT");
  if (e != nullptr && *e != 0) {
    char* end = nullptr;
    const long long v = strtoll(e, &end, 10);
    if (end != nullptr && *end == 0 && v >= 0) return v;
  }
  return mla::kSpinLimitCycles;
}

}  // namespace

extern "C" {

int mla_attn_mass(const mla_dims* dims, const mla_bf16* q_lat, const mla_bf16* pool, const int32_t* page_table,
                  const int32_t* seq_lens, const float* lse, int32_t batch, int32_t nq, int32_t max_pages,
                  int32_t num_pages, float decay, const int32_t* mass_lens, float* mass, int64_t mass_stride,
                  int32_t* dev_status, void* stream) {
  int st = check_cache_dims(dims);
  if (st != MLA_OK) return st;
  if (nq < 1 || !(decay >= 0.f && decay <= 1.f)) return MLA_ERR_INVALID_ARG;
  if ((st = check_cache_shape(dims, batch, max_pages, num_pages)) != MLA_OK) return st;
  if (nq > kMaxNq || (int64_t)batch * nq > kMaxTokens) return MLA_ERR_UNSUPPORTED;
  if (!q_lat || !pool || !page_table || !seq_lens || !lse || !mass) return MLA_ERR_INVALID_ARG;
  if (mass_stride < (int64_t)max_pages * dims->page_size) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_lat) || !aligned16(pool) || !aligned16(page_table) || !aligned16(seq_lens) || !aligned16(lse) ||
      !aligned16(mass) || (mass_lens && !aligned16(mass_lens)) || (dev_status && !aligned16(dev_status)))
    return MLA_ERR_MISALIGNED;
  const int64_t rows = (int64_t)batch * nq * dims->n_heads, row = dims->d_c + dims->d_rope;
  const int64_t tokens = (int64_t)max_pages * dims->page_size;
  const Buffer read[] = {dense(q_lat, rows, row, 2), dense(pool, (int64_t)num_pages * dims->page_size, row, 2),
                         dense(page_table, batch, max_pages, 4), dense(seq_lens, batch, 1, 4),
                         dense(mass_lens, batch, 1, 4), dense(lse, rows, 1, 4)};
  if (overlaps(strided(mass, batch, tokens, mass_stride, 4), read)) return MLA_ERR_INVALID_ARG;
  mla::MassArgs a;
  a.q_lat = q_lat; a.pool = pool; a.page_table = page_table; a.seq_lens = seq_lens; a.lse = lse;
  a.mass_lens = mass_lens; a.mass = mass; a.dev_status = dev_status; a.mass_stride = mass_stride;
  a.batch = batch; a.nq = nq; a.n_heads = dims->n_heads; a.d_c = dims->d_c; a.d_rope = dims->d_rope;
  a.page_size = dims->page_size; a.max_pages = max_pages; a.num_pages = num_pages;
  a.scale = dims->softmax_scale > 0.f ? dims->softmax_scale : 1.0f / sqrtf((float)(dims->qk_nope + dims->d_rope));
  a.decay = decay;
  if (!mla::attn_mass_pair_supported(a))
    return cuda_status(mla::launch_attn_mass(a, (cudaStream_t)stream));
  int sms = 0;
  if ((st = device_sms(&sms)) != MLA_OK) return st;
  return cuda_status(mla::launch_attn_mass_pair(a, sms, spin_limit_cycles(), (cudaStream_t)stream));
}

int mla_evict_select(const float* mass, int64_t mass_stride, const int32_t* seq_lens, const int32_t* budgets,
                     int32_t batch, int32_t n_sink, int32_t n_recent, int32_t* keep_idx, int64_t keep_stride,
                     int32_t* new_lens, int32_t* dev_status, void* stream) {
  if (batch < 1 || mass_stride < 1 || keep_stride < 1 || n_sink < 0 || n_recent < 0) return MLA_ERR_INVALID_ARG;
  if (batch > mla::kMaxBatch || mass_stride > kMaxLength) return MLA_ERR_UNSUPPORTED;
  if (!mass || !seq_lens || !budgets || !keep_idx || !new_lens) return MLA_ERR_INVALID_ARG;
  if (!aligned16(mass) || !aligned16(seq_lens) || !aligned16(budgets) || !aligned16(keep_idx) ||
      !aligned16(new_lens) || (dev_status && !aligned16(dev_status)))
    return MLA_ERR_MISALIGNED;
  // how much of a row of mass or keep_idx counts only the lengths say: the first element of each
  const Buffer lens = dense(new_lens, batch, 1, 4), keep = strided(keep_idx, batch, 1, keep_stride, 4);
  const Buffer sizes[] = {dense(seq_lens, batch, 1, 4), dense(budgets, batch, 1, 4)};
  if (overlaps(lens, sizes) || overlaps(keep, sizes) || overlaps(keep, {lens}) ||
      overlaps(strided(mass, batch, 1, mass_stride, 4), {lens, dense(keep_idx, 1, 1, 4)}))
    return MLA_ERR_INVALID_ARG;
  int sms = 0, st = device_sms(&sms);
  if (st != MLA_OK) return st;
  mla::SelectArgs a;
  a.mass = mass; a.seq_lens = seq_lens; a.budgets = budgets; a.keep_idx = keep_idx; a.new_lens = new_lens;
  a.dev_status = dev_status; a.mass_stride = mass_stride; a.keep_stride = keep_stride;
  a.batch = batch; a.n_sink = n_sink; a.n_recent = n_recent;
  return cuda_status(mla::launch_evict_select(a, sms, (cudaStream_t)stream));
}

int mla_cache_compact(const mla_dims* dims, mla_bf16* pool, const int32_t* page_table, const int32_t* seq_lens,
                      const int32_t* keep_idx, int64_t keep_stride, const int32_t* new_lens, int32_t batch,
                      int32_t max_pages, int32_t num_pages, int32_t rerotate, float* mass, int64_t mass_stride,
                      int32_t* dev_status, void* stream) {
  int st = check_cache_dims(dims);
  if (st != MLA_OK) return st;
  if (keep_stride < 1 || (rerotate != 0 && rerotate != 1)) return MLA_ERR_INVALID_ARG;
  if ((st = check_cache_shape(dims, batch, max_pages, num_pages)) != MLA_OK) return st;
  if ((int64_t)num_pages * dims->page_size >= UINT32_MAX) return MLA_ERR_UNSUPPORTED;   // row numbers are 32 bits
  if (!pool || !page_table || !seq_lens || !keep_idx || !new_lens) return MLA_ERR_INVALID_ARG;
  if (mass && mass_stride < (int64_t)max_pages * dims->page_size) return MLA_ERR_INVALID_ARG;
  if (!aligned16(pool) || !aligned16(page_table) || !aligned16(seq_lens) || !aligned16(keep_idx) ||
      !aligned16(new_lens) || (mass && !aligned16(mass)) || (dev_status && !aligned16(dev_status)))
    return MLA_ERR_MISALIGNED;
  const Buffer rows = dense(pool, (int64_t)num_pages * dims->page_size, dims->d_c + dims->d_rope, 2);
  const Buffer moved = strided(mass, batch, (int64_t)max_pages * dims->page_size, mass_stride, 4);
  const Buffer read[] = {dense(page_table, batch, max_pages, 4), dense(seq_lens, batch, 1, 4),
                         dense(new_lens, batch, 1, 4), dense(keep_idx, 1, 1, 4)};
  if (overlaps(moved, {rows}) || overlaps(moved, read) || overlaps(rows, read)) return MLA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_sms(&sms)) != MLA_OK) return st;
  mla::CompactArgs a;
  a.pool = pool; a.page_table = page_table; a.seq_lens = seq_lens; a.keep_idx = keep_idx; a.new_lens = new_lens;
  a.mass = mass; a.dev_status = dev_status; a.mass_stride = mass_stride; a.keep_stride = keep_stride;
  a.batch = batch; a.d_c = dims->d_c; a.d_rope = dims->d_rope; a.page_size = dims->page_size;
  a.max_pages = max_pages; a.num_pages = num_pages; a.rerotate = rerotate;
  // the pairs' rotation per position in turns, theta^(-2i / d_rope) / (2 pi); whole turns
  // change nothing, only the fraction counts
  const long double theta = dims->rope_theta > 0.f ? dims->rope_theta : 10000.f;
  const long double ratio = powl(theta, -2.0L / dims->d_rope);
  long double f = 1.0L / 6.283185307179586476925286766559L;
  for (int i = 0; i < dims->d_rope / 2; ++i, f *= ratio)
    a.turn[i] = (uint64_t)((f >= 1.0L ? f - floorl(f) : f) * 18446744073709551616.0L);
  return cuda_status(mla::launch_cache_compact(a, sms, (cudaStream_t)stream));
}

}  // extern "C"
