// mla_rope_append kernel: what stands between the projection of a step's new
// tokens (kv_a_proj_with_mqa and the query projection) and the attention.
// Per token t, with c = kv[t, 0:512], k = kv[t, 512:576] and the angles of its
// position:
//   c'   = w * c / sqrt(mean(c^2) + eps)              (or c, without a weight)
//   k'   = (a cos - b sin, b cos + a sin) for each of k's 32 pairs (a, b)
//   cache[slot] = [c', k']
//   q'_h = the same rotation of q_pe[t, h, 0:64], for every head h
// A pair is two adjacent elements (interleaved) or elements i and i + 32.
//
// All of it is memory traffic: per token 1,152 bytes in, 1,152 (E4M3: 576)
// out, 256 of the angle table, and 256 bytes a head of query.  A token is one
// job for its row and one for every 32 heads, a warp each; five consecutive
// jobs make a block, a token of 128 heads, so that few heads do not mean idle
// blocks.  A head is rotated by eight threads of 16 bytes (four of twice 16 for
// pairs 32 apart): whole 128-byte lines, 64 bytes a thread in flight, the
// cosines and sines kept over the job's heads.  The row's sum of squares is
// taken in fp32 by warp shuffles.  A bf16 row is computed in fp32 and rounded
// once, to bf16.
//
// An E4M3 row's codes are those of x * (1 / kv_scale) as if nothing had been
// rounded before.  fp32 alone (off by at most 16 of its steps: 21 sums under a
// root, the root, a reciprocal, three products) puts one value in a million,
// next to the middle of two codes, on the wrong one, 6 to 12% off.  So a row
// with a value within 32 steps of such a middle (one in 30) is computed again
// in pairs of fp32, a value and what its rounding left off; the 64 rotary dims
// always are.  In pairs throughout, 8,191 rows of one head took 13.4 us and of
// 16 heads 16.9; so they take 8.5 and 12.5 (6.0 and 11.2
// in fp32; of 128 heads 43.2 us either way).
//
// Measured at 8,191 tokens of 128 heads (290 MB), bf16: 44-45 us, 6.5 TB/s; of
// 16 heads (53 MB) 11.7-12.4 us.  Blocks of eight such jobs 47.5 us, jobs of 16 heads
// with pairs 32 apart 47.0 us, one block of 160 threads per token 16.4 us at
// 16 heads.
#include <cmath>

#include "common.cuh"
#include "fp8.cuh"
#include "sm100.cuh"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace rope {

constexpr int kWarps = 5;
constexpr int kThreads = 32 * kWarps;
constexpr int kJobHeads = 32;
constexpr int kHalf = MLA_ROPE_DIM / 2;  // 32 pairs

struct Params {
  const __nv_bfloat16 *kv;
  int64_t kv_stride;
  const int64_t *positions;
  const float *cos_sin;  // [max_position][32 cosines, 32 sines]
  int64_t max_position;
  const int64_t *slots;
  int64_t num_slots;
  const __nv_bfloat16 *norm_weight;  // [512] or null
  float eps;
  void *cache;
  float inv_scale;
  const __nv_bfloat16 *q;  // null: no query
  int64_t q_token, q_head;
  __nv_bfloat16 *q_out;
  int64_t qo_token, qo_head;
  int32_t heads;
  uint32_t tokens, jobs;  // jobs of a token
  int32_t *dev_status;
};

__device__ __forceinline__ void unpack8(const uint4 w, float *x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

__device__ __forceinline__ uint4 pack8(const float *x) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// The angles of `n` consecutive pairs from pair i0 on (n a multiple of 4).
template <int n>
__device__ __forceinline__ void load_angles(const float *row, int i0, float *c, float *s) {
#pragma unroll
  for (int i = 0; i < n; i += 4) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(row + i0 + i));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(row + kHalf + i0 + i));
    c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
    s[i] = b.x; s[i + 1] = b.y; s[i + 2] = b.z; s[i + 3] = b.w;
  }
}

// Eight elements: four adjacent pairs.
__device__ __forceinline__ void rotate_adjacent(float *x, const float *c, const float *s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i], b = x[2 * i + 1];
    x[2 * i] = a * c[i] - b * s[i];
    x[2 * i + 1] = b * c[i] + a * s[i];
  }
}

// Eight elements of the first half and the eight of the second they pair with.
__device__ __forceinline__ void rotate_halves(float *x, float *y, const float *c, const float *s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = x[i], b = y[i];
    x[i] = a * c[i] - b * s[i];
    y[i] = b * c[i] + a * s[i];
  }
}

// A value as the sum of two fp32: hi, rounded, and lo, what the rounding left
// off.  (The _rn forms are never contracted or reordered.)
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const float t = __fadd_rn(a.hi, b.hi), u = __fsub_rn(t, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(t, u)), __fsub_rn(b.hi, u));
  return Pair{t, __fadd_rn(e, __fadd_rn(a.lo, b.lo))};
}
__device__ __forceinline__ Pair pair_mul(Pair a, float b) {
  const float t = __fmul_rn(a.hi, b);
  return Pair{t, __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -t))};
}
// 1 / sqrt(m): one Newton step from the fp32 value, its residual 1 - m r^2 in pairs.
__device__ __forceinline__ Pair pair_rsqrt(Pair m) {
  const float r = 1.f / sqrtf(m.hi), rr = __fmul_rn(r, r), rest = __fmaf_rn(r, r, -rr);
  const float e = __fmaf_rn(-m.hi, rr, 1.f) - m.hi * rest - m.lo * rr;
  const float lo = 0.5f * r * e;
  return Pair{r, isfinite(lo) ? lo : 0.f};
}
// In fp32, an inexact value as the odd one of its two neighbours: its rounding
// to fewer bits is that of the exact value, a tie only where that is one.
__device__ __forceinline__ float pair_to_odd(Pair a) {
  const float hi = __fadd_rn(a.hi, a.lo), lo = __fsub_rn(a.lo, __fsub_rn(hi, a.hi));
  const float side = hi * lo;  // > 0: hi is the neighbour nearer to zero
  const int32_t bits = __float_as_int(hi);
  if (!(fabsf(a.hi) < INFINITY)) return a.hi;
  return __int_as_float(side > 0.f ? bits | 1 : side < 0.f ? (bits - 1) | 1 : bits);
}

// A value of the row scaled for its code.  One that fp32 holds exactly is scaled in
// fp32, as mla_cache_append_fp8 scales it.
__device__ __forceinline__ Pair scaled(Pair x, float by) {
  Pair y = pair_mul(x, by);
  if (x.lo == 0.f) y.lo = 0.f;
  return y;
}

// Eight elements of a cache row from element e on.
__device__ __forceinline__ void store8(const Params &p, int64_t slot, int e, const float *x) {
  *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.cache) + slot * kRow + e) = pack8(x);
}
__device__ __forceinline__ void store_codes8(const Params &p, int64_t slot, int e, const float *x) {
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) code[i] = f32x2_to_e4m3x2(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.cache) + slot * kRow + e) =
      make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
}

// Whether x lies within 32 steps of fp32 of the middle between two codes: 20
// bits below a code's last one.  Codes below 2^-6 are as far apart as those
// above it.
__device__ __forceinline__ bool near_middle(float x) {
  const float a = fabsf(x);
  return ((__float_as_uint(a < 0.015625f ? a + 0.015625f : a) + 0x80020u) & 0xfffffu) < 0x40u;
}

// The latent dims of an E4M3 row in pairs.  Not inlined: few rows come here.
__device__ __noinline__ void store_latent_exactly(const Params &p, int64_t slot, int lane, const uint4 *row) {
  float x0[8], x1[8], w0[8], w1[8];
  unpack8(row[lane], x0);
  unpack8(row[lane + 32], x1);
  Pair part[8];  // (squares of bf16 are exact)
#pragma unroll
  for (int i = 0; i < 8; ++i) part[i] = pair_add(Pair{__fmul_rn(x0[i], x0[i]), 0.f}, Pair{__fmul_rn(x1[i], x1[i]), 0.f});
#pragma unroll
  for (int n = 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) part[i] = pair_add(part[i], part[i + n]);
  Pair sum = part[0];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    sum = pair_add(sum, Pair{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
  const Pair by = pair_rsqrt(pair_add(pair_mul(sum, 1.f / kVDim), Pair{p.eps, 0.f}));
  const uint4 *weight = reinterpret_cast<const uint4 *>(p.norm_weight);
  unpack8(__ldg(weight + lane), w0);
  unpack8(__ldg(weight + lane + 32), w1);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // (the scale last, as in fp32: its product may overflow, but no zero becomes NaN)
    x0[i] = pair_to_odd(pair_mul(pair_mul(pair_mul(by, w0[i]), x0[i]), p.inv_scale));
    x1[i] = pair_to_odd(pair_mul(pair_mul(pair_mul(by, w1[i]), x1[i]), p.inv_scale));
  }
  store_codes8(p, slot, 8 * lane, x0);
  store_codes8(p, slot, 256 + 8 * lane, x1);
}

// The rotary dims of an E4M3 row, pair `lane` of them: a c - b s and b c + a s,
// always in pairs of fp32, because what cancels loses bits.
template <bool kAdjacent>
__device__ __forceinline__ void store_rotary_codes(const Params &p, int64_t slot, int lane, const __nv_bfloat16 *key,
                                                   const float *angles) {
  const int i = kAdjacent ? 2 * lane : lane, j = kAdjacent ? i + 1 : i + kHalf;
  const float a = __bfloat162float(key[i]), b = __bfloat162float(key[j]);
  const float c = __ldg(angles + lane), s = __ldg(angles + kHalf + lane);
  auto turn = [&](float x, float y, float sine) -> Pair {
    return scaled(pair_add(pair_mul(Pair{x, 0.f}, c), pair_mul(Pair{y, 0.f}, -sine)), p.inv_scale);
  };
  const uint32_t code = f32x2_to_e4m3x2(pair_to_odd(turn(a, b, s)), pair_to_odd(turn(b, a, -s)));
  uint8_t *out = static_cast<uint8_t *>(p.cache) + slot * kRow + kVDim;
  if (kAdjacent) {
    *reinterpret_cast<uint16_t *>(out + i) = (uint16_t)code;
  } else {
    out[i] = (uint8_t)code;
    out[j] = (uint8_t)(code >> 8);
  }
}

template <bool kFp8, bool kAdjacent>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const Params p) {
  sm100::griddep_wait();  // launched as a programmatic dependent
  sm100::griddep_launch_dependents();
  const uint32_t job = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x & 31;
  const int64_t t = job / p.jobs;
  const int part = (int)(job % p.jobs);
  if (t >= p.tokens) return;
  const bool is_row = part == (int)p.jobs - 1;
  const int64_t pos = __ldg(p.positions + t);
  if (pos < 0 || pos >= p.max_position) {  // no such angles: the token is left out
    if (is_row && lane == 0) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    return;
  }
  const float *angles = p.cos_sin + pos * MLA_ROPE_DIM;
  if (!is_row) {
    constexpr int kWords = kAdjacent ? 8 : 4;   // threads per head
    constexpr int kStep = 32 / kWords;          // heads at a time
    constexpr int kBatch = 16 / kStep;          // heads of a thread in flight
    const int w = lane % kWords, h0 = part * kJobHeads + lane / kWords;
    const __nv_bfloat16 *src = p.q + t * p.q_token + 8 * w;
    __nv_bfloat16 *dst = p.q_out + t * p.qo_token + 8 * w;
    float c[kAdjacent ? 4 : 8], s[kAdjacent ? 4 : 8];
    load_angles<kAdjacent ? 4 : 8>(angles, (kAdjacent ? 4 : 8) * w, c, s);
#pragma unroll 1
    for (int hb = h0; hb < min(p.heads, h0 + kJobHeads); hb += 16) {
      uint4 in[kBatch], in2[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = hb + i * kStep;
        if (h >= p.heads) break;
        const uint4 *at = reinterpret_cast<const uint4 *>(src + h * p.q_head);
        in[i] = *at;
        if (!kAdjacent) in2[i] = at[4];
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = hb + i * kStep;
        if (h >= p.heads) break;
        uint4 *to = reinterpret_cast<uint4 *>(dst + h * p.qo_head);
        float x[8], y[8];
        unpack8(in[i], x);
        if (kAdjacent) {
          rotate_adjacent(x, c, s);
          *to = pack8(x);
        } else {
          unpack8(in2[i], y);
          rotate_halves(x, y, c, s);
          to[0] = pack8(x);
          to[4] = pack8(y);
        }
      }
    }
    return;
  }
  // the token's row
  const int64_t slot = __ldg(p.slots + t);
  if (slot < 0 || slot >= p.num_slots) {
    if (slot != -1 && lane == 0) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    return;
  }
  const uint4 *row = reinterpret_cast<const uint4 *>(p.kv + t * p.kv_stride);
  float x0[8], x1[8], y0[8], y1[8];
  unpack8(row[lane], x0);
  unpack8(row[lane + 32], x1);
  constexpr int kRopeLanes = kAdjacent ? 8 : 4;
  if (kFp8) {
    store_rotary_codes<kAdjacent>(p, slot, lane, reinterpret_cast<const __nv_bfloat16 *>(row + 64), angles);
  } else if (lane < kRopeLanes) {
    unpack8(row[64 + lane], y0);
    if (!kAdjacent) unpack8(row[68 + lane], y1);
  }
  if (p.norm_weight) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = 1.f / sqrtf(sum * (1.f / kVDim) + p.eps);
    float w0[8], w1[8];
    const uint4 *weight = reinterpret_cast<const uint4 *>(p.norm_weight);
    unpack8(__ldg(weight + lane), w0);
    unpack8(__ldg(weight + lane + 32), w1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x0[i] = x0[i] * r * w0[i];
      x1[i] = x1[i] * r * w1[i];
    }
  }
  if (kFp8) {
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x0[i] = __fmul_rn(x0[i], p.inv_scale);
      x1[i] = __fmul_rn(x1[i], p.inv_scale);
      near |= near_middle(x0[i]) || near_middle(x1[i]);
    }
    if (p.norm_weight && __any_sync(0xffffffffu, near)) {
      store_latent_exactly(p, slot, lane, row);
      return;
    }
    store_codes8(p, slot, 8 * lane, x0);
    store_codes8(p, slot, 256 + 8 * lane, x1);
    return;
  }
  store8(p, slot, 8 * lane, x0);
  store8(p, slot, 256 + 8 * lane, x1);
  if (lane < kRopeLanes) {
    float c[8], s[8];
    load_angles<kAdjacent ? 4 : 8>(angles, (kAdjacent ? 4 : 8) * lane, c, s);
    if (kAdjacent) {
      rotate_adjacent(y0, c, s);
      store8(p, slot, kVDim + 8 * lane, y0);
    } else {
      rotate_halves(y0, y1, c, s);
      store8(p, slot, kVDim + 8 * lane, y0);
      store8(p, slot, kVDim + kHalf + 8 * lane, y1);
    }
  }
}

mla_status_t invalid(const char *why) {
  set_error_detail(why);
  return MLA_ERR_INVALID_ARGUMENT;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

mla_status_t run(Params p, int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                 int32_t interleaved, bool fp8, void *stream) {
  set_error_detail("");
  if (num_tokens < 0 || num_tokens >= 1 << 27) return invalid("num_tokens outside [0, 2^27)");
  if (block_size <= 0 || num_blocks <= 0) return invalid("block_size and num_blocks must be > 0");
  if (p.max_position <= 0) return invalid("max_position must be > 0");
  if (interleaved != 0 && interleaved != 1) return invalid("interleaved must be 0 or 1");
  if (p.norm_weight && !(std::isfinite(p.eps) && p.eps >= 0.f))
    return invalid("eps must be finite and not negative");
  if ((p.q == nullptr) != (p.q_out == nullptr)) return invalid("q_pe and q_out go together");
  if (p.q && (p.heads < 1 || p.heads > kHeads)) {
    set_error_detail("num_heads outside [1, 128]");
    return MLA_ERR_UNSUPPORTED;
  }
  if (num_tokens == 0) return MLA_OK;
  if (!p.kv || !p.positions || !p.cos_sin || !p.slots || !p.cache) return invalid("null pointer");
  if (!aligned(p.kv, 16) || !aligned(p.cos_sin, 16) || !aligned(p.cache, 16) ||
      !aligned(p.norm_weight, 16) || !aligned(p.q, 16) || !aligned(p.q_out, 16))
    return invalid("kv, cos_sin, cache, norm_weight, q_pe and q_out must be 16-byte aligned");
  if (!aligned(p.positions, 8) || !aligned(p.slots, 8))
    return invalid("positions and slot_mapping must be 8-byte aligned");
  if (p.kv_stride % 8 || p.kv_stride < kRow)
    return invalid("kv_stride must be a multiple of 8 and at least 576");
  if (p.q && (p.q_token % 8 || p.q_head % 8 || p.qo_token % 8 || p.qo_head % 8))
    return invalid("query strides must be multiples of 8");
  if (p.q && (p.q_token < 0 || p.q_head < 0)) return invalid("query strides must not be negative");
  // the rotated heads must not overlap each other
  if (p.q && ((p.heads > 1 && p.qo_head < MLA_ROPE_DIM) ||
              (num_tokens > 1 && p.qo_token < (p.heads - 1) * p.qo_head + MLA_ROPE_DIM &&
               !(p.qo_token >= MLA_ROPE_DIM &&
                 p.qo_head >= (num_tokens - 1) * p.qo_token + MLA_ROPE_DIM))))
    return invalid("q_out strides let rotated heads overlap");
  p.num_slots = num_blocks * (int64_t)block_size;
  p.tokens = (uint32_t)num_tokens;
  p.jobs = 1 + (p.q ? (p.heads + kJobHeads - 1) / kJobHeads : 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.tokens * p.jobs + kWarps - 1) / kWarps);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      fp8 ? (interleaved ? cudaLaunchKernelEx(&cfg, rope_append_kernel<true, true>, p)
                         : cudaLaunchKernelEx(&cfg, rope_append_kernel<true, false>, p))
          : (interleaved ? cudaLaunchKernelEx(&cfg, rope_append_kernel<false, true>, p)
                         : cudaLaunchKernelEx(&cfg, rope_append_kernel<false, false>, p));
  if (e == cudaSuccess) return MLA_OK;
  set_error_detail(cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

Params params(const void *kv, int64_t kv_stride, const int64_t *positions, const float *cos_sin,
              int64_t max_position, const int64_t *slot_mapping, const void *norm_weight,
              float eps, void *cache, const void *q_pe, int64_t q_token_stride,
              int64_t q_head_stride, void *q_out, int64_t q_out_token_stride,
              int64_t q_out_head_stride, int32_t num_heads, int32_t *dev_status) {
  Params p;
  p.kv = (const __nv_bfloat16 *)kv;
  p.kv_stride = kv_stride;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_position = max_position;
  p.slots = slot_mapping;
  p.num_slots = 0;
  p.norm_weight = (const __nv_bfloat16 *)norm_weight;
  p.eps = eps;
  p.cache = cache;
  p.inv_scale = 1.f;
  p.q = (const __nv_bfloat16 *)q_pe;
  p.q_token = q_token_stride;
  p.q_head = q_head_stride;
  p.q_out = (__nv_bfloat16 *)q_out;
  p.qo_token = q_out_token_stride;
  p.qo_head = q_out_head_stride;
  p.heads = num_heads;
  p.dev_status = dev_status;
  return p;
}

}  // namespace rope
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_rope_append(const void *kv, int64_t kv_stride, const int64_t *positions,
                             const float *cos_sin, int64_t max_position,
                             const int64_t *slot_mapping, int64_t num_tokens,
                             const void *norm_weight, float eps, int32_t interleaved, void *cache,
                             int64_t num_blocks, int32_t block_size, const void *q_pe,
                             int64_t q_token_stride, int64_t q_head_stride, void *q_out,
                             int64_t q_out_token_stride, int64_t q_out_head_stride,
                             int32_t num_heads, int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_rope_append");
  return rope::run(rope::params(kv, kv_stride, positions, cos_sin, max_position, slot_mapping,
                                norm_weight, eps, cache, q_pe, q_token_stride, q_head_stride,
                                q_out, q_out_token_stride, q_out_head_stride, num_heads,
                                dev_status),
                   num_tokens, num_blocks, block_size, interleaved, false, stream);
}

mla_status_t mla_rope_append_fp8(const void *kv, int64_t kv_stride, const int64_t *positions,
                                 const float *cos_sin, int64_t max_position,
                                 const int64_t *slot_mapping, int64_t num_tokens,
                                 const void *norm_weight, float eps, int32_t interleaved,
                                 void *cache8, int64_t num_blocks, int32_t block_size,
                                 float kv_scale, const void *q_pe, int64_t q_token_stride,
                                 int64_t q_head_stride, void *q_out, int64_t q_out_token_stride,
                                 int64_t q_out_head_stride, int32_t num_heads,
                                 int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_rope_append_fp8");
  if (!std::isfinite(kv_scale) || !(kv_scale > 0.f) || !std::isfinite(1.f / kv_scale))
    return rope::invalid("kv_scale and its reciprocal must be positive and finite");
  rope::Params p = rope::params(kv, kv_stride, positions, cos_sin, max_position, slot_mapping,
                                norm_weight, eps, cache8, q_pe, q_token_stride, q_head_stride,
                                q_out, q_out_token_stride, q_out_head_stride, num_heads,
                                dev_status);
  p.inv_scale = 1.f / kv_scale;
  return rope::run(p, num_tokens, num_blocks, block_size, interleaved, true, stream);
}

}  // extern "C"
