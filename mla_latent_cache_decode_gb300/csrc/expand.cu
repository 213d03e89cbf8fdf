// mla_expand_kv kernel: cached latent rows back to per-head keys and values,
// through the weights the absorption uses.  For output row t, which is token
// t - kv_offsets[b] of request b, with C[t] the 512 latent dims of its cached
// row:
//   k_nope[t, h, d] = sum_j C[t, j] W_UK[h, d, j]     (d < 128)
//   v[t, h, n]      = sum_j C[t, j] W_UV[h, j, n]     (n < 128)
//   k_pe[t, :]      = the row's 64 rotary dims
// Sums in fp32, one rounding to bf16.
//
// A product of [tokens x 512] with [512 x 256 heads]: 262,144 flops and 512
// output bytes per token and head.  With all heads it is bound by the tensor
// cores from about 300 tokens on (below, by the 256 KB a head of weights).
//
// A CTA keeps 128 output rows: their 512 latent dims sit in tensor memory as
// the A operand (256 columns), gathered from the pages once (each row looked up
// by itself, so any page size and request boundary will do, and E4M3 codes are
// widened to bf16, exactly, on the way), and every head's weights stream past
// through a ring of 16 KB stages (128 output dims x 64 of K).  A from tensor
// memory leaves shared memory's bandwidth to the weights.  Every CTA loads its
// weights for itself, by plain TMA loads into its own shared memory: CTAs depend
// on no other, and the weights may lie in any memory that the GPU can read.
// Accumulators are double-buffered (2 x 128 columns); two groups of four warps
// take turns to round them to bf16, stage them in shared memory and store them
// by TMA, 32 rows a warp (one group cannot keep up with the MMAs: 2,048 cycles a result).
//
// An item is one head's keys or values of a tile of 128 rows; the items (tile
// by tile, head by head) are cut into equal runs, one a CTA.
//
// Measured: 8,192 tokens of 128 heads 203-212 us (1.36-1.30 PFLOP/s, 71-68% of
// the measured bf16 rate), 4,501 tokens from E4M3 110-115 us, 11,051 of 16 heads
// 41-42 us, 286 of 128 heads 18.8 us (53 MB: 8).
//
// What bounds it: the tensor cores are busy 69% of an SM's cycles; in between they
// wait for weights and for results' way out.  Of the first case's 212 us, 164 are
// left without weights loaded, 170 without results stored, 148 without both (of 16
// heads' 42: 37, 37, 35); part of what that gains is the clock, 1.82 GHz under the
// power limit.  No path is at its limit by its counters (L2 51%, its way to the SMs
// 48% at 11 TB/s, HBM 36%, the MMAs' reads of shared memory 31%), and a shorter
// ring changes nothing (11 stages instead of 12: 209 against 212 us).  Results
// stored from registers instead of by TMA were slower (259 us against 182 when this
// was tried).
#include <atomic>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "fp8.cuh"
#include "ragged.cuh"
#include "sm100_issue.cuh"
#include "tmap.h"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace expand {
using namespace sm100;

constexpr int kRows = 128;              // output rows of a CTA
constexpr int kDims = 128;              // key dims, value dims of a head
constexpr int kKChunks = kVDim / 64;    // 64-dim chunks of the latent
constexpr int kStage = kDims * 128;     // 128 output dims x 64 of K: 16 KB
constexpr int kStages = 12;
constexpr int kWarpStage = 4096;        // a warp's 64 dims of its 32 rows, 128-byte swizzle
constexpr int kOutWarps = 8;            // rows in, results out: two groups of four warps
constexpr int kThreads = 32 * (kOutWarps + 3);  // and a warp each for weights, MMAs and rotary dims
constexpr uint32_t kChange = 4;         // a change of rows, in items (see run_start)
constexpr uint32_t kTmemCols = 512, kColA = 0, kColD = 256;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainNs = 10000000ull;

struct Maps {
  CUtensorMap w_uk, w_uv, k_nope, v;
};

struct Params {
  const void *cache;
  int64_t num_slots;
  int32_t block_size;
  const int32_t *block_table;
  int32_t max_blocks_per_seq;
  const int32_t *kv_offsets;
  int32_t batch, total_kv, heads;
  float kv_scale;
  const __nv_bfloat16 *w_uk, *w_uv;
  __nv_bfloat16 *k_nope, *v, *k_pe;
  int32_t *dev_status;
};

struct __align__(1024) Smem {
  uint8_t w[kStages][kStage];
  uint8_t out[2][4 * kWarpStage];
  uint64_t w_full[kStages], w_empty[kStages], d_full[2], d_empty[2], a_full, fin;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory of one SM");

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// Two E4M3 codes (low byte first) as bf16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  return pack2(f.x, f.y);
}

__device__ __forceinline__ void set_abort(Smem &s, int32_t *dev_status) {
  s.abort = 1;
  report(dev_status, MLA_ERR_DEVICE_TIMEOUT);
}

__device__ __forceinline__ bool wait_or_abort(Smem &s, const Params &p, uint64_t &bar, uint32_t parity) {
  if (mbar_wait(smem_u32(&bar), parity, &s.abort, kWaitNs)) return true;
  if (!*(volatile int *)&s.abort) set_abort(s, p.dev_status);
  return false;
}

__device__ __forceinline__ bool warp_wait(Smem &s, const Params &p, uint64_t &bar, uint32_t parity) {
  const bool ok = mbar_wait(smem_u32(&bar), parity, &s.abort, kWaitNs);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0 && !*(volatile int *)&s.abort) set_abort(s, p.dev_status);
  return false;
}

// Cache row of each lane's output row t (by a whole warp), -1 for a row of no
// request (left as it is), -2 for one whose page lies outside the table or the
// pool.
__device__ __forceinline__ int64_t cache_row(const Params &p, int32_t t, int32_t begin, int32_t end) {
  const ragged::Place at = ragged::place_of(p.kv_offsets, p.batch, t);
  if (t < begin || t >= end) return -1;
  if (t < at.offset) return -2;
  const uint32_t pos = (uint32_t)t - (uint32_t)at.offset, page = pos / (uint32_t)p.block_size;
  if (page >= (uint32_t)p.max_blocks_per_seq) return -2;
  const int32_t blk = p.block_table[(int64_t)at.request * p.max_blocks_per_seq + page];
  const int64_t row = (int64_t)blk * p.block_size + pos % (uint32_t)p.block_size;
  return blk < 0 || row >= p.num_slots ? -2 : row;
}

// Half of 32 rows' latent dims (256 each) by a warp: from the cache, a quarter
// of a warp per row and load so that every access is a whole line ...
template <bool kFp8>
struct HalfRows {
  static constexpr int kParts = kFp8 ? 2 : 4;  // of 128 bytes a row
  uint4 v[kParts][8];

  // `row`: the lane's own cache row (< 0: zeros)
  __device__ __forceinline__ void load(const Params &p, int64_t row, int half, int lane) {
    const uint8_t *cache = static_cast<const uint8_t *>(p.cache) + half * kParts * 128 + (lane & 7) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = __shfl_sync(0xffffffffu, row, 4 * i + (lane >> 3));
#pragma unroll
      for (int k = 0; k < kParts; ++k)
        v[k][i] = r < 0 ? make_uint4(0, 0, 0, 0)
                        : *reinterpret_cast<const uint4 *>(cache + r * (kFp8 ? kRow : 2 * kRow) + k * 128);
    }
  }

  // (the same lines towards L2 only)
  static __device__ __forceinline__ void prefetch(const Params &p, int64_t row, int half, int lane) {
    constexpr int kLines = kFp8 ? 3 : 4;  // E4M3 rows start anywhere in a line
    const uint8_t *cache = static_cast<const uint8_t *>(p.cache) + half * kParts * 128;
#pragma unroll
    for (int i = 0; i < kLines; ++i) {
      const int64_t r = __shfl_sync(0xffffffffu, row, (lane + 32 * i) / kLines);
      const int at = (lane + 32 * i) % kLines * 128;
      if (r >= 0)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(cache + r * (kFp8 ? kRow : 2 * kRow) + min(at, kParts * 128 - 16)));
    }
  }

  // ... and through 4 KB of the warp's own shared memory (16-byte units
  // swizzled by the row) into the tensor-memory lane of each row, E4M3 codes
  // as bf16.
  __device__ __forceinline__ void store(uint8_t *stage, uint32_t a_addr, int lane) const {
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3);
        *reinterpret_cast<uint4 *>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) = v[k][i];
      }
      __syncwarp();
#pragma unroll
      for (int w0 = 0; w0 < 8; w0 += kFp8 ? 4 : 8) {  // 32 columns at a time
        uint32_t a[32];
#pragma unroll
        for (int w = 0; w < (kFp8 ? 4 : 8); ++w) {
          const uint4 u = *reinterpret_cast<const uint4 *>(stage + lane * 128 + (((w0 + w) ^ (lane & 7)) << 4));
          const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (kFp8) {
              a[8 * w + 2 * c] = e4m3x2_to_bf16x2(e[c] & 0xffffu);
              a[8 * w + 2 * c + 1] = e4m3x2_to_bf16x2(e[c] >> 16);
            } else {
              a[4 * w + c] = e[c];
            }
          }
        }
        tmem_st32(a_addr + k * (kFp8 ? 64 : 32) + w0 * (kFp8 ? 8 : 4), a);
      }
    }
  }
};

// The 64 rotary dims of a warp's 32 rows (first of them t) as k_pe: eight lanes
// a row.
template <bool kFp8>
__device__ __forceinline__ void copy_rope(const Params &p, int64_t row, int32_t t, int lane) {
  const uint8_t *cache = static_cast<const uint8_t *>(p.cache) + kVDim * (kFp8 ? 1 : 2) + (lane & 7) * (kFp8 ? 8 : 16);
  uint4 in[8];
  int64_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r[i] = __shfl_sync(0xffffffffu, row, 4 * i + (lane >> 3));
    in[i] = make_uint4(0, 0, 0, 0);
    if (r[i] < 0) continue;
    if (kFp8) {
      const uint2 c = *reinterpret_cast<const uint2 *>(cache + r[i] * kRow);
      in[i].x = c.x;
      in[i].y = c.y;
    } else {
      in[i] = *reinterpret_cast<const uint4 *>(cache + r[i] * 2 * kRow);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r[i] < 0) continue;
    uint4 o = in[i];
    if (kFp8) {
      const uint2 c = make_uint2(in[i].x, in[i].y);
      const uint32_t u[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
      uint32_t e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t h = e4m3x2_to_f16x2(u[k]);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        e[k] = pack2(f.x * p.kv_scale, f.y * p.kv_scale);
      }
      o = make_uint4(e[0], e[1], e[2], e[3]);
    }
    reinterpret_cast<uint4 *>(p.k_pe + (int64_t)(t + 4 * i + (lane >> 3)) * MLA_ROPE_DIM)[lane & 7] = o;
  }
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *m, int32_t x, int32_t y, int32_t z, uint32_t src,
                                             uint64_t policy) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2, %3}], [%4], %5;" ::
                   "l"(reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z), "r"(src), "l"(policy)
               : "memory");
}

// Results leave L2 first (90 MB of them, 16 heads of 11,051 tokens: 36 us; with
// the normal policy 44).
__device__ __forceinline__ uint64_t policy_stream() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1) expand_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem &s = *reinterpret_cast<Smem *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.w_full[i]), 1);
      mbar_init(smem_u32(&s.w_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.d_full[i]), 1);
      mbar_init(smem_u32(&s.d_empty[i]), kRows);
    }
    mbar_init(smem_u32(&s.a_full), 2 * kRows);
    mbar_init(smem_u32(&s.fin), 1);
    s.abort = 0;
    fence_mbarrier_init_cluster();
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(smem_u32(&s.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  // Launched as a programmatic dependent: what is above may run while the
  // kernel before this one ends, what is below reads and writes memory.
  griddep_wait();
  griddep_launch_dependents();
  const int32_t rows_begin = ragged::cut(p.kv_offsets[0], p.total_kv), rows_end = ragged::cut(p.kv_offsets[p.batch], p.total_kv);
  // This CTA's run of items [i0, i1): row tile i / per, head and kind i % per.
  // The runs are equal in cost, in which a change of rows counts as kChange
  // items (11,051 tokens of 16 heads 41.7 us with 3, 42.1 with 4, 42.8 with 6, 44.5
  // with 10; 286 of 128 heads 19.2, 18.8, 18.9, 20.0; large calls of 128 heads all
  // the same).  32 bits hold the cost of all rows: at most 2^23 tiles of 260 each.
  const uint32_t per = 2 * p.heads, tiles = (uint32_t)((rows_end + kRows - 1) / kRows);
  const uint32_t cost = tiles == 0 ? 0 : tiles * (per + kChange) - kChange;
  auto run_start = [&](uint32_t k) -> uint32_t {  // of CTA k
    const uint32_t at = cost / gridDim.x * k + cost % gridDim.x * k / gridDim.x + kChange;
    const uint32_t g = at / (per + kChange), in = at % (per + kChange);
    return min(g * per + (in > kChange ? in - kChange : 0), tiles * per);
  };
  const uint32_t i0 = run_start(blockIdx.x), i1 = run_start(blockIdx.x + 1);
  // the first rows' places, while the barriers and the tensor memory are set up
  int64_t first_row = -1;
  if (warp < kOutWarps && i0 < i1)
    first_row = cache_row(p, (int32_t)(i0 / per) * kRows + (warp & 3) * 32 + lane, rows_begin, rows_end);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  if (warp < kOutWarps) {
    // ------------------------------------------------ rows in, results out
    const int side = warp >> 2;             // the group of four warps, and its result buffer
    const int r = (warp & 3) * 32 + lane;   // row = TMEM lane
    uint8_t *const stage = &s.out[side][0] + (warp & 3) * kWarpStage;
    const uint64_t hint = policy_stream();
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // what the staging buffer held has been read
    auto stage_free = [&]() {
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
    };
    // the tile of rows being multiplied: its first row, the lane's cache row,
    // and whether each of the warp's 32 (that the tensors have) is a request's
    int32_t t0 = 0;
    int64_t row = -1, next_row = -1;
    bool whole = false;
    uint32_t item = i0 % per;
    // Item i of the run: its tile's rows first, if they are new, then the
    // result of the item before, so that at a change of rows the MMAs wait no
    // longer than for them.
    for (uint32_t i = i0, n = 0; i <= i1 && i0 < i1; ++i, ++n, item = item + 1 == per ? 0 : item + 1) {
      const int32_t t = t0;
      const int64_t own_row = row;
      const bool store_whole = whole;
      if (i < i1 && (n == 0 || item == 0)) {
        t0 = (int32_t)(i / per) * kRows;
        row = n == 0 ? first_row : next_row;
        if (row == -2 && side == 0) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
        const int32_t tw = t0 + (warp & 3) * 32;
        whole = tw < p.total_kv && tw >= rows_begin && min(tw + 32, p.total_kv) <= rows_end;
        HalfRows<kFp8> rows;
        rows.load(p, row, side, lane);
        // the rows before are done with when the last product is complete, the
        // staging buffer when its last store has read it
        if (n > 0) {
          stage_free();
          if (!warp_wait(s, p, s.d_full[(n - 1) & 1], ((n - 1) >> 1) & 1)) break;
          tc_fence_after();
        }
        rows.store(stage, lanes + kColA + 128 * side, lane);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&s.a_full));
        if (i + per - item < i1) {  // the next tile's rows towards L2 meanwhile
          next_row = cache_row(p, t0 + kRows + r, rows_begin, rows_end);
          HalfRows<kFp8>::prefetch(p, next_row, side, lane);
        }
      }
      if (n == 0 || ((n - 1) & 1) != (uint32_t)side) continue;  // nothing yet, or the other group's
      if (!warp_wait(s, p, s.d_full[side], ((n - 1) >> 1) & 1)) break;
      tc_fence_after();
      uint32_t d[kDims];
#pragma unroll
      for (int k = 0; k < kDims; k += 32) tmem_ld32(lanes + kColD + 128 * side + k, d + k);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < kDims; k += 32) tmem_loaded32(d + k);
      tc_fence_before();
      mbar_arrive(smem_u32(&s.d_empty[side]));
      const float by = kFp8 ? p.kv_scale : 1.f;
      const uint32_t done = (item == 0 ? per : item) - 1;  // the item before
      const int h = (int)(done >> 1);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint4 o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(d[64 * half + 8 * k + e]) * by;
          o[k] = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
        }
        if (store_whole) {
          stage_free();
#pragma unroll
          for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4 *>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) = o[k];
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(done & 1 ? &maps.v : &maps.k_nope, 64 * half, h, t + (warp & 3) * 32, smem_u32(stage), hint);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else if (own_row != -1) {
          uint4 *dst = reinterpret_cast<uint4 *>((done & 1 ? p.v : p.k_nope) +
                                                 ((int64_t)(t + r) * p.heads + h) * kDims + 64 * half);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = o[k];
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  } else if (warp == kOutWarps) {
    // ------------------------------------------------ weights
    if (elect_one_sync()) {
      prefetch_tmap(&maps.w_uk);
      prefetch_tmap(&maps.w_uv);
      prefetch_tmap(&maps.k_nope);
      prefetch_tmap(&maps.v);
      const uint64_t hint = policy_evict_normal();
      uint32_t n = 0;
      bool ok = true;
      uint32_t st = 0, ph = 1;
      uint32_t item = i0 % per;
      for (uint32_t i = i0; i < i1 && ok; ++i, item = item + 1 == per ? 0 : item + 1) {
        const int32_t h = (int32_t)(item >> 1);
        for (int kc = 0; kc < kKChunks; ++kc, ++n) {
          if (!(ok = wait_or_abort(s, p, s.w_empty[st], ph))) break;
          const uint32_t bar = smem_u32(&s.w_full[st]);
          mbar_arrive_expect_tx(bar, kStage);
          const uint32_t dst = smem_u32(s.w[st]);
          if (item & 1) {  // rows: 64 of K for output dims 0-63, then for 64-127
            tma_load_2d_hint(dst, &maps.w_uv, 0, h * kVDim + kc * 64, bar, hint);
            tma_load_2d_hint(dst + kStage / 2, &maps.w_uv, 64, h * kVDim + kc * 64, bar, hint);
          } else {         // rows: output dims
            tma_load_2d_hint(dst, &maps.w_uk, kc * 64, h * kDims, bar, hint);
          }
          if (++st == kStages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      if (*(volatile int *)&s.abort)  // no copy may still be landing when the shared memory is given up
        for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
          (void)mbar_wait(smem_u32(&s.w_full[i % kStages]), (i / kStages) & 1, nullptr, kDrainNs);
    }
  } else if (warp == kOutWarps + 1) {
    // ------------------------------------------------ MMA issuer
    if (elect_one_sync()) {
      const uint32_t d_k = desc_low(s.w[0], 16), d_v = desc_low(s.w[0], kStage / 2);
      uint32_t n = 0, st = 0, ph = 0, loads = 0;  // results, the ring's place and phase, row tiles
      // one item; keys and values differ in how K runs through a stage
      auto product = [&](auto is_value) -> bool {
        constexpr bool kValue = decltype(is_value)::value;
        constexpr uint32_t id = idesc_bf16_f32(kRows, kDims, kValue);
        constexpr uint32_t kStep = kValue ? 128 : 2;  // 16 of K: 16 rows, or 32 bytes
        const uint32_t d = tmem + kColD + 128 * (n & 1);
#pragma unroll
        for (int kc = 0; kc < kKChunks; ++kc) {
          if (!wait_or_abort(s, p, s.w_full[st], ph)) return false;
          tc_fence_after();
          const uint32_t b = (kValue ? d_v : d_k) + st * (kStage >> 4);
          const uint32_t a = tmem + kColA + 32 * kc;
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ts_low(d, a + 8 * k, b + kStep * k, id, (kc > 0 || k > 0) ? 1u : 0u);
          mma_commit(smem_u32(&s.w_empty[st]));
          if (++st == kStages) {
            st = 0;
            ph ^= 1;
          }
        }
        return true;
      };
      uint32_t left = 0;  // items of the current row tile
      bool ok = true;
      for (uint32_t i = i0; i < i1 && ok; ++i, ++n, --left) {
        if (left == 0) {
          left = per - i % per;
          if (!(ok = wait_or_abort(s, p, s.a_full, loads++ & 1))) break;
        }
        if (!(ok = wait_or_abort(s, p, s.d_empty[n & 1], ((n >> 1) & 1) ^ 1))) break;
        tc_fence_after();
        ok = i & 1 ? product(std::true_type{}) : product(std::false_type{});  // per is even
        if (ok) mma_commit(smem_u32(&s.d_full[n & 1]));
      }
      mma_commit(smem_u32(&s.fin));
      if (!mbar_wait(smem_u32(&s.fin), 0, nullptr, kWaitNs)) report(p.dev_status, MLA_ERR_DEVICE_TIMEOUT);
    }
  } else {
    // ------------------------------------------------ rotary dims
    // of the row tiles whose first item is in this run
    for (uint32_t g = (i0 + per - 1) / per; g * per < i1; ++g) {
      const int32_t t = (int32_t)g * kRows;
      int64_t rows[kRows / 32];
#pragma unroll
      for (int q = 0; q < kRows / 32; ++q) rows[q] = cache_row(p, t + 32 * q + lane, rows_begin, rows_end);
#pragma unroll
      for (int q = 0; q < kRows / 32; ++q) copy_rope<kFp8>(p, rows[q], t + 32 * q, lane);
    }
    if (blockIdx.x == 0) ragged::check_offsets(p.kv_offsets, p.batch, p.total_kv, lane, 32, p.dev_status);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- host

mla_status_t invalid(const char *why) {
  set_error_detail(why);
  return MLA_ERR_INVALID_ARGUMENT;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool encode(CUtensorMap *m, const void *base, int rank, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t b1, uint32_t b2) {
  tmap::EncodeTiledFn fn = tmap::encode_fn();
  if (!fn) return false;
  cuuint64_t size[3] = {d0, d1, d2}, strides[2] = {d0 * 2, d0 * d1 * 2};
  cuuint32_t box[3] = {64, b1, b2}, each[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), size, strides, box, each,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFp8>
cudaError_t launch(const Params &p, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  static std::atomic<int> known[64];
  int sms = known[dev].load(std::memory_order_acquire);
  if (sms == 0) {
    e = cudaFuncSetAttribute(expand_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(Smem) + 1024);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    known[dev].store(sms, std::memory_order_release);
  }
  Maps maps;
  if (!encode(&maps.w_uk, p.w_uk, 2, kVDim, (uint64_t)p.heads * kDims, 1, kDims, 1) ||
      !encode(&maps.w_uv, p.w_uv, 2, kDims, (uint64_t)p.heads * kVDim, 1, 64, 1) ||
      !encode(&maps.k_nope, p.k_nope, 3, kDims, p.heads, p.total_kv, 1, 32) ||
      !encode(&maps.v, p.v, 3, kDims, p.heads, p.total_kv, 1, 32))
    return cudaErrorInvalidValue;
  // as many CTAs as SMs, but no more than items
  const int64_t items = ((int64_t)p.total_kv + kRows - 1) / kRows * 2 * p.heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < sms ? items : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem) + 1024;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, expand_kernel<kFp8>, maps, p);
}

mla_status_t run(Params p, int64_t num_blocks, int64_t total_kv, bool fp8, void *stream) {
  set_error_detail("");
  if (p.batch < 0 || total_kv < 0 || total_kv >= 1 << 30)
    return invalid("batch < 0, or total_kv outside [0, 2^30)");
  p.total_kv = (int32_t)total_kv;
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
  const cudaError_t e = fp8 ? launch<true>(p, (cudaStream_t)stream) : launch<false>(p, (cudaStream_t)stream);
  if (e == cudaSuccess) return MLA_OK;
  set_error_detail(cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

Params params(const void *cache, int32_t block_size, const int32_t *block_table,
              int32_t max_blocks_per_seq, const int32_t *kv_offsets, int32_t batch,
              const void *w_uk, const void *w_uv, int32_t num_heads, float kv_scale,
              void *k_nope, void *v, void *k_pe, int32_t *dev_status) {
  Params p;
  p.cache = cache;
  p.num_slots = 0;
  p.total_kv = 0;
  p.block_size = block_size;
  p.block_table = block_table;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.kv_offsets = kv_offsets;
  p.batch = batch;
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
                                    batch, w_uk, w_uv, num_heads, 1.f, k_nope, v, k_pe,
                                    dev_status),
                     num_blocks, total_kv, false, stream);
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
                                    kv_offsets, batch, w_uk, w_uv, num_heads, kv_scale, k_nope,
                                    v, k_pe, dev_status),
                     num_blocks, total_kv, true, stream);
}

}  // extern "C"
