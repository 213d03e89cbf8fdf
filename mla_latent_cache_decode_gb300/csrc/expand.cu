// mla_expand_kv kernel: cached latent rows back to per-head keys and values,
// through the weights the absorption uses.  For output row t, which is token
// t - kv_offsets[b] of request b, with C[t] the 512 latent dims of its cached
// row:
//   k_nope[t, h, d] = sum_j C[t, j] W_UK[h, d, j]     (d < 128)
//   v[t, h, n]      = sum_j C[t, j] W_UV[h, j, n]     (n < 128)
//   k_pe[t, :]      = the row's 64 rotary dims
// Sums in fp32, one rounding to bf16.
#include <cmath>

#include "common.cuh"
#include "fp8.cuh"
#include "ragged.cuh"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace expand {

constexpr int kRows = 16;   // output rows of a block
constexpr int kDims = 128;  // key dims and value dims of a head
constexpr int kThreads = 256;

struct Params {
  const void *cache;
  int64_t num_slots;
  int32_t block_size;
  const int32_t *block_table;
  int32_t max_blocks_per_seq;
  const int32_t *kv_offsets;
  int32_t batch;
  int64_t total_kv;
  const __nv_bfloat16 *w_uk, *w_uv;
  int32_t heads;
  float kv_scale;
  __nv_bfloat16 *k_nope, *v, *k_pe;
  int32_t *dev_status;
};

// Cache row of output row t, -1 for a row behind the last request (left as it
// is), -2 for one whose page lies outside the pool or the table (reported).
__device__ int64_t cache_row(const Params &p, int64_t t) {
  if (t >= p.total_kv || t < p.kv_offsets[0] || t >= p.kv_offsets[p.batch]) return -1;
  const int32_t lo = ragged::request_of(p.kv_offsets, p.batch, (int32_t)t);
  const int64_t pos = t - p.kv_offsets[lo];
  const int64_t page = pos / p.block_size;
  if (page >= p.max_blocks_per_seq) return -2;
  const int32_t blk = p.block_table[(int64_t)lo * p.max_blocks_per_seq + page];
  const int64_t row = (int64_t)blk * p.block_size + pos % p.block_size;
  return blk < 0 || row >= p.num_slots ? -2 : row;
}

template <bool kFp8>
__device__ float element(const Params &p, int64_t row, int j) {
  if (!kFp8) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p.cache)[row * kRow + j]);
  const uint32_t two = e4m3x2_to_f16x2(static_cast<const uint8_t *>(p.cache)[row * kRow + j]);
  __half_raw h;
  h.x = (unsigned short)two;
  return __half2float(__half(h)) * p.kv_scale;
}

// grid = (ceil(total_kv / 16), heads): thread n < 128 sums key dim n of 16
// rows, thread 128 + n value dim n.
template <bool kFp8>
__global__ void __launch_bounds__(kThreads) expand_kernel(const Params p) {
  __shared__ int64_t row[kRows];
  __shared__ float latent[kRows][kVDim];
  const int64_t t0 = (int64_t)blockIdx.x * kRows;
  const int h = blockIdx.y;
  if (blockIdx.x == 0 && h == 0)
    ragged::check_offsets(p.kv_offsets, p.batch, (int32_t)p.total_kv, threadIdx.x, kThreads,
                          p.dev_status);
  if (threadIdx.x < kRows) {
    row[threadIdx.x] = cache_row(p, t0 + threadIdx.x);
    if (row[threadIdx.x] == -2) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kVDim; i += kThreads)
    latent[i / kVDim][i % kVDim] = row[i / kVDim] < 0 ? 0.f : element<kFp8>(p, row[i / kVDim], i % kVDim);
  __syncthreads();
  const bool value = threadIdx.x >= kDims;
  const int n = threadIdx.x % kDims;
  float sum[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) sum[r] = 0.f;
  for (int j = 0; j < kVDim; ++j) {
    const float w = __bfloat162float(value ? p.w_uv[((int64_t)h * kVDim + j) * kDims + n]
                                           : p.w_uk[((int64_t)h * kDims + n) * kVDim + j]);
#pragma unroll
    for (int r = 0; r < kRows; ++r) sum[r] += latent[r][j] * w;
  }
  __nv_bfloat16 *out = value ? p.v : p.k_nope;
  for (int r = 0; r < kRows; ++r)
    if (row[r] >= 0) out[((t0 + r) * p.heads + h) * kDims + n] = __float2bfloat16(sum[r]);
  if (h == 0)
    for (int i = threadIdx.x; i < kRows * MLA_ROPE_DIM; i += kThreads) {
      const int r = i / MLA_ROPE_DIM, e = i % MLA_ROPE_DIM;
      if (row[r] >= 0)
        p.k_pe[(t0 + r) * MLA_ROPE_DIM + e] = __float2bfloat16(element<kFp8>(p, row[r], kVDim + e));
    }
}

mla_status_t invalid(const char *why) {
  set_error_detail(why);
  return MLA_ERR_INVALID_ARGUMENT;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

mla_status_t run(Params p, int64_t num_blocks, bool fp8, void *stream) {
  set_error_detail("");
  if (p.batch < 0 || p.total_kv < 0 || p.total_kv > INT32_MAX)
    return invalid("batch < 0, or total_kv outside [0, 2^31)");
  if (p.block_size <= 0 || num_blocks <= 0 || num_blocks > INT32_MAX)
    return invalid("block_size and num_blocks must be > 0");
  if (p.max_blocks_per_seq <= 0) return invalid("max_blocks_per_seq must be > 0");
  if (p.heads < 1 || p.heads > kHeads) {
    set_error_detail("num_heads outside [1, 128]");
    return MLA_ERR_UNSUPPORTED;
  }
  if (p.batch == 0 || p.total_kv == 0) return MLA_OK;
  if (!p.cache || !p.block_table || !p.kv_offsets || !p.w_uk || !p.w_uv || !p.k_nope || !p.v ||
      !p.k_pe)
    return invalid("null pointer");
  if (!aligned(p.cache, 16) || !aligned(p.w_uk, 16) || !aligned(p.w_uv, 16) ||
      !aligned(p.k_nope, 16) || !aligned(p.v, 16) || !aligned(p.k_pe, 16))
    return invalid("cache, weights and outputs must be 16-byte aligned");
  if (!aligned(p.block_table, 4) || !aligned(p.kv_offsets, 4))
    return invalid("block_table and kv_offsets must be 4-byte aligned");
  p.num_slots = num_blocks * (int64_t)p.block_size;
  const dim3 grid((unsigned)((p.total_kv + kRows - 1) / kRows), (unsigned)p.heads);
  if (fp8) expand_kernel<true><<<grid, kThreads, 0, (cudaStream_t)stream>>>(p);
  else expand_kernel<false><<<grid, kThreads, 0, (cudaStream_t)stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return MLA_OK;
  set_error_detail(cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

Params params(const void *cache, int32_t block_size, const int32_t *block_table,
              int32_t max_blocks_per_seq, const int32_t *kv_offsets, int32_t batch,
              int64_t total_kv, const void *w_uk, const void *w_uv, int32_t num_heads,
              float kv_scale, void *k_nope, void *v, void *k_pe, int32_t *dev_status) {
  Params p;
  p.cache = cache;
  p.num_slots = 0;
  p.block_size = block_size;
  p.block_table = block_table;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.kv_offsets = kv_offsets;
  p.batch = batch;
  p.total_kv = total_kv;
  p.w_uk = (const __nv_bfloat16 *)w_uk;
  p.w_uv = (const __nv_bfloat16 *)w_uv;
  p.heads = num_heads;
  p.kv_scale = kv_scale;
  p.k_nope = (__nv_bfloat16 *)k_nope;
  p.v = (__nv_bfloat16 *)v;
  p.k_pe = (__nv_bfloat16 *)k_pe;
  p.dev_status = dev_status;
  return p;
}

}  // namespace expand
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_expand_kv(const void *cache, int64_t num_blocks, int32_t block_size,
                           const int32_t *block_table, int32_t max_blocks_per_seq,
                           const int32_t *kv_offsets, int32_t batch, int64_t total_kv,
                           const void *w_uk, const void *w_uv, int32_t num_heads, void *k_nope,
                           void *v, void *k_pe, int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_expand_kv");
  return expand::run(expand::params(cache, block_size, block_table, max_blocks_per_seq, kv_offsets,
                                    batch, total_kv, w_uk, w_uv, num_heads, 1.f, k_nope, v, k_pe,
                                    dev_status),
                     num_blocks, false, stream);
}

mla_status_t mla_expand_kv_fp8(const void *cache8, int64_t num_blocks, int32_t block_size,
                               const int32_t *block_table, int32_t max_blocks_per_seq,
                               const int32_t *kv_offsets, int32_t batch, int64_t total_kv,
                               const void *w_uk, const void *w_uv, int32_t num_heads,
                               float kv_scale, void *k_nope, void *v, void *k_pe,
                               int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_expand_kv_fp8");
  if (!std::isfinite(kv_scale) || !(kv_scale > 0.f))
    return expand::invalid("kv_scale must be positive and finite");
  return expand::run(expand::params(cache8, block_size, block_table, max_blocks_per_seq,
                                    kv_offsets, batch, total_kv, w_uk, w_uv, num_heads, kv_scale,
                                    k_nope, v, k_pe, dev_status),
                     num_blocks, true, stream);
}

}  // extern "C"
