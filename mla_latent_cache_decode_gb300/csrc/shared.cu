// Decode of a batch whose requests begin with the same tokens (sm_103a), see
// mla_decode_shared.  A block takes a head of a request: each warp every eighth
// token with a running maximum and sum, the warps' results joined at the end.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "sm100.cuh"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace shared {

using namespace sm100;

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Params {
  const __nv_bfloat16 *q, *cache;
  const int32_t *shared_table, *shared_blocks, *block_table, *seq_lens;
  __nv_bfloat16 *out;
  float *lse;
  int32_t *dev_status;
  int32_t num_blocks, block_size, max_shared_blocks, max_blocks_per_seq, batch, heads;
  float scale;
};

__global__ void __launch_bounds__(kThreads) shared_kernel(const Params p) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_acc[kWarps][kVDim];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.heads, h = blockIdx.x % p.heads;
  griddep_wait();
  int32_t shared = *p.shared_blocks, L = p.seq_lens[b];
  if (shared < 0 || shared > p.max_shared_blocks) {
    report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    shared = min(max(shared, 0), p.max_shared_blocks);
  }
  if (L < 0 || L > p.max_blocks_per_seq * p.block_size) {
    report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    L = min(max(L, 0), p.max_blocks_per_seq * p.block_size);
  }
  float q[18], acc[16], m = -INFINITY, l = 0.f;
  const __nv_bfloat16 *qr = p.q + ((int64_t)b * p.heads + h) * kRow;
#pragma unroll
  for (int i = 0; i < 18; ++i) q[i] = __bfloat162float(qr[32 * i + lane]) * p.scale;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int32_t t = warp; t < L; t += kWarps) {
    const int32_t page = t / p.block_size;
    const int32_t blk = page < shared ? p.shared_table[page] : p.block_table[(int64_t)b * p.max_blocks_per_seq + page];
    if (blk < 0 || blk >= p.num_blocks) {
      report(p.dev_status, MLA_ERR_DEVICE_RANGE);
      continue;
    }
    const __nv_bfloat16 *row = p.cache + ((int64_t)blk * p.block_size + t % p.block_size) * kRow;
    float x[18], s = 0.f;
#pragma unroll
    for (int i = 0; i < 18; ++i) {
      x[i] = __bfloat162float(row[32 * i + lane]);
      s += x[i] * q[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (s == -INFINITY) continue;
    const float top = fmaxf(m, s), keep = m == -INFINITY ? 0.f : expf(m - top), w = expf(s - top);
    m = top;
    l = l * keep + w;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = acc[i] * keep + w * x[i];
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int i = 0; i < 16; ++i) s_acc[warp][32 * i + lane] = acc[i];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  for (int d = tid; d < kVDim; d += kThreads) {
    float o = 0.f;
    total = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w] == -INFINITY ? 0.f : expf(s_m[w] - top);
      o += f * s_acc[w][d];
      total += f * s_l[w];
    }
    p.out[((int64_t)b * p.heads + h) * kVDim + d] = __float2bfloat16_rn(total == 0.f ? 0.f : o / total);
  }
  if (tid == 0 && p.lse) p.lse[(int64_t)b * p.heads + h] = total == 0.f ? -INFINITY : top + logf(total);
}

mla_status_t invalid(const char *why) {
  set_error_detail(why);
  return MLA_ERR_INVALID_ARGUMENT;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace shared
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_decode_shared_workspace_size(int32_t batch, int32_t num_heads) {
  if (batch < 0 || num_heads < 1 || num_heads > kHeads) return 0;
  return 256;
}

mla_status_t mla_decode_shared(const void *q, const void *cache, int64_t num_blocks, int32_t block_size, const int32_t *shared_table,
                               const int32_t *shared_blocks, int32_t max_shared_blocks, const int32_t *block_table,
                               int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t batch, int32_t num_heads,
                               float softmax_scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                               int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_decode_shared");
  using namespace mla::shared;
  set_error_detail("");
  if (batch < 0 || max_shared_blocks < 0) return invalid("batch < 0 or max_shared_blocks < 0");
  if (num_heads < 1 || num_heads > kHeads) {
    set_error_detail("num_heads outside [1, 128]");
    return MLA_ERR_UNSUPPORTED;
  }
  if (block_size <= 0) return invalid("block_size must be > 0");
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128 && block_size != 256) {
    set_error_detail("block_size not in {16,32,64,128,256}");
    return MLA_ERR_UNSUPPORTED;
  }
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return invalid("softmax_scale must be positive and finite");
  if (num_blocks <= 0 || num_blocks > INT32_MAX || max_blocks_per_seq <= 0 || (int64_t)max_blocks_per_seq * block_size > 1 << 30 ||
      (int64_t)max_shared_blocks * block_size > 1 << 30)
    return invalid("num_blocks, max_blocks_per_seq or max_shared_blocks out of range");
  if (batch > 1 << 20) return invalid("batch > 2^20");
  if (batch == 0) return MLA_OK;
  if (!q || !cache || !shared_blocks || (max_shared_blocks > 0 && !shared_table) || !block_table || !seq_lens || !out || !workspace)
    return invalid("null pointer");
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16)) return invalid("q, cache and out must be 16-byte aligned");
  if (!aligned(shared_table, 4) || !aligned(shared_blocks, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4))
    return invalid("shared_table, shared_blocks, block_table, seq_lens and lse must be 4-byte aligned");
  if (!aligned(workspace, 256)) return invalid("workspace must be 256-byte aligned");
  const size_t need = mla_decode_shared_workspace_size(batch, num_heads);
  if (workspace_bytes < need) {
    set_error_detail("workspace is smaller than mla_decode_shared_workspace_size()");
    return MLA_ERR_WORKSPACE_TOO_SMALL;
  }
  Params p;
  p.q = (const __nv_bfloat16 *)q;
  p.cache = (const __nv_bfloat16 *)cache;
  p.shared_table = shared_table;
  p.shared_blocks = shared_blocks;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = (__nv_bfloat16 *)out;
  p.lse = lse;
  p.dev_status = dev_status;
  p.num_blocks = (int32_t)num_blocks;
  p.block_size = block_size;
  p.max_shared_blocks = max_shared_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.batch = batch;
  p.heads = num_heads;
  p.scale = softmax_scale;
  shared_kernel<<<batch * num_heads, kThreads, 0, (cudaStream_t)stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return MLA_OK;
  set_error_detail(cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

}  // extern "C"
