// mla_prefill kernel: attention of prompt tokens over expanded keys and values.
// Request b owns query rows [q_offsets[b], q_offsets[b+1]) and key rows
// [kv_offsets[b], kv_offsets[b+1]); with i, j counted inside the request,
//   s_ij = softmax_scale * (q_nope_i . k_nope_j + q_pe_i . k_pe_j)
//   j visible to i: j < nk, and when causal also j <= nk - nq + i
//   out_i = sum_j softmax(s_i)_j v_j,   lse_i = log sum_j exp(s_ij)
// A row that sees no key gets out = 0 and lse = -inf.
#include <cmath>

#include "common.cuh"
#include "ragged.cuh"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace prefill {

constexpr int kNope = 128, kRope = MLA_ROPE_DIM, kV = 128;
constexpr int kWarps = 8;

struct Strided {
  const __nv_bfloat16 *p;
  int64_t token, head;  // elements
};

struct Params {
  Strided q_nope, q_pe, k_nope, k_pe, v;
  const int32_t *q_offsets, *kv_offsets;
  int32_t batch, heads;
  int64_t total_q, total_kv;
  int32_t causal;
  float scale;
  __nv_bfloat16 *out;
  float *lse;
  int32_t *dev_status;
};

// One warp per query row and head, one pass over its keys with the running
// maximum and sum.
__global__ void __launch_bounds__(32 * kWarps) prefill_kernel(const Params p) {
  const int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  const int h = blockIdx.y, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && h == 0) {
    ragged::check_offsets(p.q_offsets, p.batch, (int32_t)p.total_q, threadIdx.x, 32 * kWarps,
                          p.dev_status);
    ragged::check_offsets(p.kv_offsets, p.batch, (int32_t)p.total_kv, threadIdx.x, 32 * kWarps,
                          p.dev_status);
  }
  if (t >= p.total_q || t < p.q_offsets[0] || t >= p.q_offsets[p.batch]) return;
  const int32_t lo = ragged::request_of(p.q_offsets, p.batch, (int32_t)t);
  const int64_t i = t - p.q_offsets[lo], nq = p.q_offsets[lo + 1] - p.q_offsets[lo];
  const int64_t k0 = p.kv_offsets[lo], k1 = p.kv_offsets[lo + 1];
  if (k0 < 0 || k1 < k0 || k1 > p.total_kv) {
    if (lane == 0) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    return;
  }
  const int64_t nk = k1 - k0;
  const int64_t last = p.causal ? min(nk, nk - nq + i + 1) : nk;
  float q[6], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < 4; ++e)
    q[e] = __bfloat162float(p.q_nope.p[t * p.q_nope.token + h * p.q_nope.head + lane + 32 * e]);
  for (int e = 0; e < 2; ++e)
    q[4 + e] = __bfloat162float(p.q_pe.p[t * p.q_pe.token + h * p.q_pe.head + lane + 32 * e]);
  for (int64_t j = k0; j < k0 + last; ++j) {
    float s = 0.f;
    for (int e = 0; e < 4; ++e)
      s += q[e] * __bfloat162float(p.k_nope.p[j * p.k_nope.token + h * p.k_nope.head + lane + 32 * e]);
    for (int e = 0; e < 2; ++e)
      s += q[4 + e] * __bfloat162float(p.k_pe.p[j * p.k_pe.token + lane + 32 * e]);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale;
    const float m_new = fmaxf(m, s);
    const float a = expf(m - m_new), w = expf(s - m_new);
    l = l * a + w;
    for (int e = 0; e < 4; ++e)
      o[e] = o[e] * a + w * __bfloat162float(p.v.p[j * p.v.token + h * p.v.head + lane + 32 * e]);
    m = m_new;
  }
  const float inv = last > 0 ? 1.f / l : 0.f;
  for (int e = 0; e < 4; ++e)
    p.out[(t * p.heads + h) * kV + lane + 32 * e] = __float2bfloat16(o[e] * inv);
  if (p.lse && lane == 0) p.lse[t * p.heads + h] = last > 0 ? m + logf(l) : -INFINITY;
}

mla_status_t invalid(const char *why) {
  set_error_detail(why);
  return MLA_ERR_INVALID_ARGUMENT;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Strides of 16-byte multiples that keep rows of n elements apart
bool strides_ok(const Strided &s, int n) {
  return s.token % 8 == 0 && s.head % 8 == 0 && s.token >= n && s.head >= n &&
         s.token < (1ll << 38) && s.head < (1ll << 38);
}

constexpr size_t kWorkspaceBytes = 32u << 20;

mla_status_t run(const Params &p, void *workspace, size_t workspace_bytes, void *stream) {
  set_error_detail("");
  if (p.batch < 0 || p.total_q < 0 || p.total_kv < 0 || p.total_q > INT32_MAX ||
      p.total_kv > INT32_MAX)
    return invalid("batch < 0, or total_q or total_kv outside [0, 2^31)");
  if (p.heads < 1 || p.heads > kHeads) {
    set_error_detail("num_heads outside [1, 128]");
    return MLA_ERR_UNSUPPORTED;
  }
  if (p.causal != 0 && p.causal != 1) return invalid("causal must be 0 or 1");
  if (!std::isfinite(p.scale) || !(p.scale > 0.f))
    return invalid("softmax_scale must be positive and finite");
  if (p.batch == 0 || p.total_q == 0) return MLA_OK;
  if (!p.q_nope.p || !p.q_pe.p || !p.q_offsets || !p.kv_offsets || !p.out ||
      (p.total_kv > 0 && (!p.k_nope.p || !p.k_pe.p || !p.v.p)))
    return invalid("null pointer");
  if (!aligned(p.q_nope.p, 16) || !aligned(p.q_pe.p, 16) || !aligned(p.k_nope.p, 16) ||
      !aligned(p.k_pe.p, 16) || !aligned(p.v.p, 16) || !aligned(p.out, 16))
    return invalid("queries, keys, values and out must be 16-byte aligned");
  if (!aligned(p.q_offsets, 4) || !aligned(p.kv_offsets, 4) || !aligned(p.lse, 4))
    return invalid("q_offsets, kv_offsets and lse must be 4-byte aligned");
  if (!strides_ok(p.q_nope, kNope) || !strides_ok(p.q_pe, kRope) || !strides_ok(p.k_nope, kNope) ||
      !strides_ok(p.v, kV) || p.k_pe.token % 8 || p.k_pe.token < kRope)
    return invalid("strides must be multiples of 8 elements and at least a row's width");
  if (workspace && (!aligned(workspace, 256) || workspace_bytes < kWorkspaceBytes)) {
    set_error_detail("workspace must be 256-byte aligned and of mla_prefill_workspace_size()");
    return aligned(workspace, 256) ? MLA_ERR_WORKSPACE_TOO_SMALL : MLA_ERR_INVALID_ARGUMENT;
  }
  const dim3 grid((unsigned)((p.total_q + kWarps - 1) / kWarps), (unsigned)p.heads);
  prefill_kernel<<<grid, 32 * kWarps, 0, (cudaStream_t)stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return MLA_OK;
  set_error_detail(cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

}  // namespace prefill
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_prefill_workspace_size(void) { return prefill::kWorkspaceBytes; }

mla_status_t mla_prefill(const void *q_nope, int64_t q_nope_token_stride,
                         int64_t q_nope_head_stride, const void *q_pe, int64_t q_pe_token_stride,
                         int64_t q_pe_head_stride, const void *k_nope,
                         int64_t k_nope_token_stride, int64_t k_nope_head_stride,
                         const void *k_pe, int64_t k_pe_token_stride, const void *v,
                         int64_t v_token_stride, int64_t v_head_stride, const int32_t *q_offsets,
                         const int32_t *kv_offsets, int32_t batch, int64_t total_q,
                         int64_t total_kv, int32_t num_heads, int32_t causal, float softmax_scale,
                         void *out, float *lse, void *workspace, size_t workspace_bytes,
                         int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_prefill");
  using prefill::Strided;
  typedef const __nv_bfloat16 *Bf16;
  prefill::Params p;
  p.q_nope = Strided{(Bf16)q_nope, q_nope_token_stride, q_nope_head_stride};
  p.q_pe = Strided{(Bf16)q_pe, q_pe_token_stride, q_pe_head_stride};
  p.k_nope = Strided{(Bf16)k_nope, k_nope_token_stride, k_nope_head_stride};
  p.k_pe = Strided{(Bf16)k_pe, k_pe_token_stride, 0};
  p.v = Strided{(Bf16)v, v_token_stride, v_head_stride};
  p.q_offsets = q_offsets;
  p.kv_offsets = kv_offsets;
  p.batch = batch;
  p.heads = num_heads;
  p.total_q = total_q;
  p.total_kv = total_kv;
  p.causal = causal;
  p.scale = softmax_scale;
  p.out = (__nv_bfloat16 *)out;
  p.lse = lse;
  p.dev_status = dev_status;
  return prefill::run(p, workspace, workspace_bytes, stream);
}

}  // extern "C"
