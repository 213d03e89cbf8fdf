// The attention weight that a step's queries give each cached token (sm_103a):
//   mass[b, t] = decay * previous[b, t] + sum_h exp(scale q[b,h] . row_t - lse[b,h])
// with the log-sum-exps that the step's decode wrote.  A warp takes a token: its
// row in registers, one head after the other.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "fp8.cuh"
#include "sm100.cuh"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace mass {

using namespace sm100;

constexpr int kThreads = 256;

struct Params {
  const __nv_bfloat16 *q;
  const uint8_t *cache;
  const int32_t *block_table;
  const int32_t *seq_lens;
  const float *lse;
  const float *previous;
  float *mass;
  int64_t previous_stride, mass_stride;
  int32_t *dev_status;
  int32_t num_blocks, block_size, max_blocks_per_seq, batch, heads, max_tokens;
  float scale_log2, decay;
};

template <bool kFp8>
__global__ void __launch_bounds__(kThreads) mass_kernel(const Params p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    int32_t L = p.seq_lens[b];
    const int32_t most = min(p.max_tokens, p.max_blocks_per_seq * p.block_size);
    if (L < 0 || L > most) {
      report(p.dev_status, MLA_ERR_DEVICE_RANGE);
      L = min(max(L, 0), most);
    }
    for (int32_t t = blockIdx.x * (kThreads / 32) + warp; t < L; t += gridDim.x * (kThreads / 32)) {
      const int32_t blk = p.block_table[(int64_t)b * p.max_blocks_per_seq + t / p.block_size];
      if (blk < 0 || blk >= p.num_blocks) {
        report(p.dev_status, MLA_ERR_DEVICE_RANGE);
        continue;
      }
      const int64_t row = ((int64_t)blk * p.block_size + t % p.block_size) * kRow;
      float x[18];
#pragma unroll
      for (int i = 0; i < 18; ++i) {
        const int d = 32 * i + lane;
        if (kFp8) {
          const uint32_t h = e4m3x2_to_f16x2(p.cache[row + d]);
          asm("{.reg .b16 l, u; mov.b32 {l, u}, %1; cvt.f32.f16 %0, l;}" : "=f"(x[i]) : "r"(h));
        } else {
          x[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.cache)[row + d]);
        }
      }
      float sum = 0.f;
      for (int h = 0; h < p.heads; ++h) {
        const __nv_bfloat16 *q = p.q + ((int64_t)b * p.heads + h) * kRow;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 18; ++i) s += x[i] * __bfloat162float(q[32 * i + lane]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float l = p.lse[(int64_t)b * p.heads + h];
        sum += l == -INFINITY ? 0.f : ex2_approx(s * p.scale_log2 - l * 1.4426950408889634f);
      }
      if (lane == 0) {
        if (p.previous) sum += p.decay * p.previous[(int64_t)b * p.previous_stride + t];
        p.mass[(int64_t)b * p.mass_stride + t] = sum;
      }
    }
  }
}

mla_status_t invalid(const char *why) {
  set_error_detail(why);
  return MLA_ERR_INVALID_ARGUMENT;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Args {
  const void *q, *cache;
  int64_t num_blocks;
  int32_t block_size;
  const int32_t *block_table;
  int32_t max_blocks_per_seq;
  const int32_t *seq_lens;
  int32_t batch, heads;
  float scale, kv_scale;
  const float *lse, *previous;
  int64_t previous_stride;
  float decay;
  float *mass;
  int64_t mass_stride;
  int32_t max_tokens;
  int32_t *dev_status;
  bool fp8;
};

mla_status_t run(const Args &a, void *stream) {
  set_error_detail("");
  if (a.batch < 0 || a.max_tokens < 0) return invalid("batch < 0 or max_tokens < 0");
  if (a.heads < 1 || a.heads > kHeads) {
    set_error_detail("num_heads outside [1, 128]");
    return MLA_ERR_UNSUPPORTED;
  }
  if (a.block_size <= 0) return invalid("block_size must be > 0");
  if (a.block_size != 16 && a.block_size != 32 && a.block_size != 64 && a.block_size != 128 && a.block_size != 256) {
    set_error_detail("block_size not in {16,32,64,128,256}");
    return MLA_ERR_UNSUPPORTED;
  }
  if (!std::isfinite(a.scale) || !(a.scale > 0.f)) return invalid("softmax_scale must be positive and finite");
  if (!std::isfinite(a.kv_scale) || !(a.kv_scale > 0.f) || !std::isfinite(a.scale * a.kv_scale) || !(a.scale * a.kv_scale > 0.f))
    return invalid("kv_scale, and its product with softmax_scale, must be positive and finite");
  if (!std::isfinite(a.decay) || !(a.decay >= 0.f)) return invalid("decay must be finite and not negative");
  if (a.num_blocks <= 0 || a.num_blocks > INT32_MAX || a.max_blocks_per_seq <= 0 ||
      (int64_t)a.max_blocks_per_seq * a.block_size > 1 << 30)
    return invalid("num_blocks or max_blocks_per_seq out of range");
  if ((int64_t)a.batch * kHeads > INT32_MAX) return invalid("batch too large");
  if (a.batch == 0 || a.max_tokens == 0) return MLA_OK;
  if (!a.q || !a.cache || !a.block_table || !a.seq_lens || !a.lse || !a.mass) return invalid("null pointer");
  if (!aligned(a.q, 16) || !aligned(a.cache, 16)) return invalid("q and cache must be 16-byte aligned");
  if (!aligned(a.block_table, 4) || !aligned(a.seq_lens, 4) || !aligned(a.lse, 4) || !aligned(a.previous, 4) || !aligned(a.mass, 4))
    return invalid("block_table, seq_lens, lse, previous and mass must be 4-byte aligned");
  if (a.batch > 1 && (a.mass_stride < a.max_tokens || (a.previous && a.previous_stride < a.max_tokens)))
    return invalid("mass_stride or previous_stride is below max_tokens");
  Params p;
  p.q = (const __nv_bfloat16 *)a.q;
  p.cache = (const uint8_t *)a.cache;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.lse = a.lse;
  p.previous = a.previous;
  p.mass = a.mass;
  p.previous_stride = a.previous_stride;
  p.mass_stride = a.mass_stride;
  p.dev_status = a.dev_status;
  p.num_blocks = (int32_t)a.num_blocks;
  p.block_size = a.block_size;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.batch = a.batch;
  p.heads = a.heads;
  p.max_tokens = a.max_tokens;
  p.scale_log2 = a.scale * a.kv_scale * 1.4426950408889634f;
  p.decay = a.decay;
  const dim3 grid(std::min(4096, (a.max_tokens + 7) / 8), std::min(a.batch, 65535));
  if (a.fp8) mass_kernel<true><<<grid, kThreads, 0, (cudaStream_t)stream>>>(p);
  else mass_kernel<false><<<grid, kThreads, 0, (cudaStream_t)stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return MLA_OK;
  set_error_detail(cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

}  // namespace mass
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_attention_mass(const void *q, const void *cache, int64_t num_blocks, int32_t block_size, const int32_t *block_table,
                                int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t batch, int32_t num_heads,
                                float softmax_scale, const float *lse, const float *previous, int64_t previous_stride, float decay,
                                float *mass, int64_t mass_stride, int32_t max_tokens, int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_attention_mass");
  return mass::run(mass::Args{q, cache, num_blocks, block_size, block_table, max_blocks_per_seq, seq_lens, batch, num_heads, softmax_scale,
                              1.f, lse, previous, previous_stride, decay, mass, mass_stride, max_tokens, dev_status, false},
                   stream);
}

mla_status_t mla_attention_mass_fp8(const void *q, const void *cache8, int64_t num_blocks, int32_t block_size,
                                    const int32_t *block_table, int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t batch,
                                    int32_t num_heads, float softmax_scale, float kv_scale, const float *lse, const float *previous,
                                    int64_t previous_stride, float decay, float *mass, int64_t mass_stride, int32_t max_tokens,
                                    int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_attention_mass_fp8");
  return mass::run(mass::Args{q, cache8, num_blocks, block_size, block_table, max_blocks_per_seq, seq_lens, batch, num_heads,
                              softmax_scale, kv_scale, lse, previous, previous_stride, decay, mass, mass_stride, max_tokens, dev_status,
                              true},
                   stream);
}

}  // extern "C"
