// The attention weight that a step's queries give each cached token (sm_103a):
//   mass[b, t] = decay * previous[b, t] + sum_h exp(scale q[b,h] . row_t - lse[b,h])
// with the log-sum-exps that the step's decode wrote.
//
// What bounds it: a row is 1,152 bytes (576 in E4M3) and 2 * 576 * heads flops,
// 128 flops a byte at 128 heads: memory, if the tensor cores and the loads keep
// out of each other's way.
//
// A pair of SMs shares each MMA (cta_group::2, M = 128: 64 tokens in each SM) with
// tokens as rows and heads as columns, so that a token's heads lie in one lane and
// are summed by its thread:
//   S [128 tokens x N] = K [128 x 576] Q^T
// Each SM keeps the queries of half the heads (B operand) and streams its own
// tokens (A operand, each row once) through a ring of the shared memory that is
// left, 147 KB at 128 heads; a single SM would hold all queries and have half
// the ring.  Lanes 0-63 of the result are the 64 tokens with the first block's
// heads, lanes 64-127 the same tokens with the second's.
//
// E4M3 rows are multiplied as they are (kind::f8f6f4).  A query is the sum of two
// E4M3 numbers: with its head's largest dim scaled to (224, 448] by a power of
// two, hi = E4M3(q) leaves a rest of at most four significant bits, which E4M3
// holds too (down to its smallest step, 2^-9 of a scaled dim: 2^-17 of the
// largest).  So S has columns for hi and lo, and twice the columns at twice the
// rate cost what bf16 costs, without the rows being widened.
//
// A score is off by what the tensor cores cut from each of its sums (24 bits are
// kept) and by its exponent's rounding; both are held down (Sizes::kSums, weight()):
// 5e-7 of the weights at 201 tokens, 1.3e-6 without.
//
// Work: a chain is a request's tokens in units of 128, the units dealt out to the
// pairs in order in runs of equal cost; every block works out the deal (as in
// shared.cu).  Warp roles: 0 loads rows, 1 issues the MMAs (first block of the
// pair), 2 loads bf16 queries, 3 owns the tensor memory, 4-11 weigh (thread = 64
// tokens x 4 quarters of the heads) and split queries for E4M3.  Every wait is
// bounded; one that runs out reports MLA_ERR_DEVICE_TIMEOUT and ends the block's
// others.
//
// Measured: 20 x 4,096 tokens, 128 heads 21.3 us (98 MB, 4.6 TB/s, 68% of the copy
// rate): 2 us of deal and set-up, then the first tiles of all SMs and 11 MB of
// queries at once, then ~1.45 us a tile, which is the memory's rate.  E4M3, 131,072
// + 7 x 1,024 tokens, 16 heads 22 us: 6.6 us until the queries are split and
// the first tile weighed, then 0.75 us a tile, the memory's rate.  Four weighing
// warps instead of eight took 2 us more there; a thread that loads its quarter of
// a query instead of a warp that loads four queries, 2 us.  201 tokens: 5.2 us.
#include <algorithm>
#include <atomic>
#include <cmath>

#include <cuda_fp16.h>

#include "cluster.cuh"
#include "common.cuh"
#include "fp8.cuh"
#include "tmap.h"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace mass {

using namespace sm100;

constexpr int kTile = 128;          // tokens of a unit: 64 in each block of the pair
constexpr int kOwn = kTile / 2;
constexpr int kChunks = kRow / 64;  // 9
constexpr int kThreads = 384, kWeighWarp0 = 4, kWeighWarps = 8;
constexpr int kItemChunks = 3;      // chunks of an item of the ring
constexpr int kMaxSlots = 12;
constexpr int kBuffers = 2;         // of S, by tile
constexpr int64_t kUnitCost = 2, kChainCost = 3;
constexpr int kMaxPairs = 256;
constexpr uint64_t kWaitBudgetNs = 100000000ull;
constexpr uint64_t kDrainBudgetNs = 10000000ull;
constexpr double kLog2eExact = 1.4426950408889634074;
constexpr float kLog2e = (float)kLog2eExact, kLog2eRest = (float)(kLog2eExact - (double)kLog2e);

struct Control {
  // full, q_full and s_free count in the first block; the others in each
  uint64_t full[kMaxSlots], empty[kMaxSlots], q_full, q_free, s_full[kBuffers], s_free[kBuffers], sum_full[2][2], head_full, mma_end;
  // By chain parity: lse and scale for 2^x, each as a number and what its rounding left (an exponent of 40
  // rounded to 24 bits is off by as much as all of a weight's other errors).
  float lse[2][kHeads + 32], lse_rest[2][kHeads + 32], factor[2][kHeads + 32], factor_rest[2][kHeads + 32];
  float sum[2][kOwn][4];                    // of a token's heads, by quarters, by tile parity
  int64_t start_cost, share[2], warp_cost[kThreads / 32];
  int32_t start_chain;
  uint32_t tmem_base, items;  // (items of rows that the loader has asked for)
  int abort;
};

struct Maps {
  CUtensorMap k;   // rows, box {64, min(block_size, 64)}
  CUtensorMap k3;  // {64, rows, 9}, box {64, 64, 3} (pages of 64 rows and more)
  CUtensorMap q;   // {64, batch * heads, 9}, box {64, columns / 2, 3} (bf16)
};

struct Params {
  const __nv_bfloat16 *q;
  const int32_t *block_table;
  const int32_t *seq_lens;
  const float *lse;
  const float *previous;
  float *mass;
  int64_t previous_stride, mass_stride;
  int32_t *dev_status;
  int32_t num_blocks, block_size, page_log2, max_blocks_per_seq, batch, heads, longest, pairs;
  int32_t head_stride;  // heads of the first block
  int32_t half_heads;   // columns for a block's heads, a multiple of 16
  int32_t slots;
  float scale_log2, scale_rest, decay;  // scale * log2(e) is the sum of the first two, the second >= 0
};

template <bool kFp8>
struct Sizes {
  static constexpr int kChunkRow = kFp8 ? 64 : 128;       // bytes of a chunk's row
  static constexpr int kChunkBytes = kOwn * kChunkRow;
  static constexpr int kItemBytes = kItemChunks * kChunkBytes;
  static constexpr int kParts = kFp8 ? 2 : 1;             // columns of a head
  // The tensor cores cut each sum to 24 bits: 36 steps of it were most of a weight's error.  The bf16 form
  // has room for a sum of its own for each third of the dims, added in registers (E4M3: 18 steps, one sum).
  static constexpr int kSums = kFp8 ? 1 : kChunks / kItemChunks;
  static constexpr uint32_t kBuffer = kFp8 ? 128 : 256, kCols = kBuffers * kBuffer;
};

// Dynamic shared memory: the ring, the queries (chunk after chunk, this block's columns as rows), Control.
template <bool kFp8>
__host__ __device__ constexpr int query_bytes(int half_heads) {
  return kChunks * half_heads * Sizes<kFp8>::kParts * Sizes<kFp8>::kChunkRow;
}
template <bool kFp8>
inline int slots_for(int half_heads) {
  const int room = 232448 - 1024 - (int)sizeof(Control) - query_bytes<kFp8>(half_heads);
  return std::min(kMaxSlots, room / Sizes<kFp8>::kItemBytes);
}

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {  // of numbers that are mostly small
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int32_t length_of(const Params &p, int32_t L) { return min(max(L, 0), p.longest); }
__device__ __forceinline__ int64_t cost_of(int32_t L) { return L > 0 ? kChainCost + kUnitCost * ((L + kTile - 1) / kTile) : 0; }

// A pair's pieces in order: tokens [t0, t1) of request b.
struct Walk {
  const Params *p;
  int64_t x0, x1, at;
  int32_t next_b, b, t0, t1;
  __device__ Walk(const Params &params, const Control &s) : p(&params), x0(s.share[0]), x1(s.share[1]), at(s.start_cost), next_b(s.start_chain) {}
  __device__ bool next() {
    while (next_b < p->batch && at < x1) {
      b = next_b++;
      const int32_t L = length_of(*p, p->seq_lens[b]);
      if (L == 0) continue;
      const int32_t units = (L + kTile - 1) / kTile;
      const int64_t place = at + kChainCost;
      at = place + kUnitCost * units;
      const int64_t k0 = x0 <= place ? 0 : (x0 - place + kUnitCost - 1) / kUnitCost;
      const int64_t k1 = x1 <= place ? 0 : min((int64_t)units, (x1 - place + kUnitCost - 1) / kUnitCost);
      if (k0 >= k1) continue;
      t0 = (int32_t)k0 * kTile;
      t1 = min(L, (int32_t)k1 * kTile);
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ void set_abort(Control &s, int32_t *dev_status) {
  s.abort = 1;
  report(dev_status, MLA_ERR_DEVICE_TIMEOUT);
}

// Every lane polls, then the warp agrees.
__device__ __forceinline__ bool warp_wait(Control &s, uint64_t *bar, uint32_t parity, int32_t *dev_status) {
  const bool ok = mbar_wait(smem_u32(bar), parity, &s.abort, kWaitBudgetNs);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0) set_abort(s, dev_status);
  return false;
}

// kBox: rows of a box, min(block_size, 64).
template <bool kFp8, int kBox>
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const __grid_constant__ Maps maps, const Params p) {
  using Z = Sizes<kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *queries = ring + p.slots * Z::kItemBytes;
  Control &s = *reinterpret_cast<Control *>(queries + query_bytes<kFp8>(p.half_heads));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int32_t pair = (int32_t)cluster_id();
  const bool first_block = rank == 0;
  const int cols = p.half_heads * Z::kParts;  // of this block, in N and in tensor memory

  if (tid == 0) {
    auto init = [](uint64_t *bar, int count) { mbar_init(smem_u32(bar), count); };
    for (int i = 0; i < p.slots; ++i) init(&s.full[i], 1), init(&s.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      init(&s.s_full[i], 1);
      init(&s.s_free[i], 2 * kWeighWarps);
      init(&s.sum_full[i][0], 4);
      init(&s.sum_full[i][1], 4);
    }
    init(&s.q_full, kFp8 ? 2 * kWeighWarps : 1);
    init(&s.q_free, 1);
    init(&s.head_full, kWeighWarps);
    init(&s.mma_end, 1);
    s.abort = 0;
    s.items = 0;
    fence_mbarrier_init_cluster();
    prefetch_tmap(kBox >= kOwn ? &maps.k3 : &maps.k);
    if (!kFp8) prefetch_tmap(&maps.q);
  }
  if (warp == 3) {
    tmem_alloc_pair(smem_u32(&s.tmem_base), Z::kCols);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_arrive();  // barriers and tensor memory, to both blocks
  griddep_wait();
  griddep_launch_dependents();

  // ---------------------------------------------------------------- the deal
  {
    int64_t before = 0, mine = 0, start = 0;
    auto sum_up = [&](int32_t b0) {
      const int32_t L = b0 + tid < p.batch ? p.seq_lens[b0 + tid] : 0;
      if (blockIdx.x == 0 && L != length_of(p, L)) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
      mine = cost_of(length_of(p, L));
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s.warp_cost[warp] = incl;
      __syncthreads();
      start = before + incl - mine;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) start += s.warp_cost[w];
        before += s.warp_cost[w];
      }
    };
    for (int32_t b0 = 0; b0 < p.batch; b0 += kThreads) {
      if (b0 > 0) __syncthreads();
      sum_up(b0);
    }
    const int64_t C = before;
    const int64_t x0 = quotient(pair * C + p.pairs - 1, p.pairs);
    if (tid == 0) {
      s.share[0] = x0;
      s.share[1] = quotient((pair + 1) * C + p.pairs - 1, p.pairs);
      s.start_chain = p.batch;
      s.start_cost = C;
    }
    __syncthreads();
    auto find = [&](int32_t b0) {
      if (mine > 0 && start <= x0 && x0 < start + mine) {
        s.start_chain = b0 + tid;
        s.start_cost = start;
      }
    };
    if (p.batch <= kThreads) {
      find(0);
    } else {
      before = 0;
      for (int32_t b0 = 0; b0 < p.batch; b0 += kThreads) {
        sum_up(b0);
        find(b0);
        __syncthreads();
      }
    }
  }
  __syncthreads();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  Walk walk(p, s);
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (mbar_wait(smem_u32(bar), parity, &s.abort, kWaitBudgetNs)) return true;
    set_abort(s, p.dev_status);
    return false;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- rows
    if (elect_one_sync()) {
      constexpr int kBoxes = kOwn / kBox;
      const uint32_t full0 = cluster_addr(smem_u32(&s.full[0]), 0);
      uint32_t sl = 0, turn = 1, items = 0;
      bool ok = true;
      while (ok && walk.next()) {
        const int32_t *table = p.block_table + (int64_t)walk.b * p.max_blocks_per_seq;
        int32_t blk[kBoxes];  // read a tile ahead
        // This block's tokens (both blocks load at least a box of every item, so that neither falls behind
        // the ring's rounds: where the second has none, the tile's first, whose sums nobody stores).
        auto own_of = [&](int32_t tt) { return tt + (int)rank * kOwn < walk.t1 ? tt + (int)rank * kOwn : tt; };
        auto boxes_of = [](int32_t tokens) { return max(1, (min(tokens, kOwn) + kBox - 1) / kBox); };
        auto look_up = [&](int32_t tt) {
          const int32_t own = own_of(tt);
#pragma unroll
          for (int i = 0; i < kBoxes; ++i) blk[i] = own + i * kBox < walk.t1 ? table[(own + i * kBox) >> p.page_log2] : 0;
        };
        look_up(walk.t0);
        for (int32_t tt = walk.t0; ok && tt < walk.t1; tt += kTile) {
          const int32_t n = min(kTile, walk.t1 - tt), own = own_of(tt);
          const int32_t boxes = boxes_of(rank == 0 || n <= kOwn ? n : n - kOwn), others = boxes_of(rank == 1 || n <= kOwn ? n : n - kOwn);
          const uint32_t bytes = (uint32_t)((boxes + others) * kBox * Z::kChunkRow * kItemChunks);
          int32_t y[kBoxes];
#pragma unroll
          for (int i = 0; i < kBoxes; ++i) {
            y[i] = 0;
            if (i < boxes) {
              if (blk[i] < 0 || blk[i] >= p.num_blocks) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
              else y[i] = (blk[i] << p.page_log2) + ((own + i * kBox) & (p.block_size - 1));
            }
          }
          if (tt + kTile < walk.t1) look_up(tt + kTile);
#pragma unroll 1
          for (int c = 0; c < kChunks; c += kItemChunks) {
            if (!(ok = wait(&s.empty[sl], turn))) break;
            if (first_block) mbar_arrive_expect_tx(smem_u32(&s.full[sl]), bytes);
            const uint32_t dst = smem_u32(ring) + sl * Z::kItemBytes, bar = full0 + 8 * sl;
            if (kBox >= kOwn) {
              tma_load_3d_pair(dst, &maps.k3, 0, y[0], c, bar);
            } else {
#pragma unroll
              for (int i = 0; i < kBoxes; ++i)
                if (i < boxes)
#pragma unroll
                  for (int k = 0; k < kItemChunks; ++k)
                    tma_load_2d_pair(dst + k * Z::kChunkBytes + i * kBox * Z::kChunkRow, &maps.k, 64 * (c + k), y[i], bar);
            }
            *(volatile uint32_t *)&s.items = ++items;
            if (++sl == (uint32_t)p.slots) sl = 0, turn ^= 1u;
          }
        }
      }
      // Both blocks stay until the end of all MMAs has been said to both: that is the last arrival of the MMAs at
      // a block's barriers, and the meeting at the end does not wait for them.  (From here on, as the first block's
      // issuer: the budget is that of the last rows, not of the call.)
      if (!first_block && !mbar_wait(smem_u32(&s.mma_end), 0, nullptr, kWaitBudgetNs)) report(p.dev_status, MLA_ERR_DEVICE_TIMEOUT);
      if (s.abort && first_block)  // let the loads in flight land in both blocks
        for (uint32_t i = items > (uint32_t)p.slots ? items - p.slots : 0; i < items; ++i)
          (void)mbar_wait(smem_u32(&s.full[i % p.slots]), (i / p.slots) & 1u, nullptr, kDrainBudgetNs);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S = K Q^T
    if (first_block && elect_one_sync()) {
      const uint32_t n8 = (uint32_t)(2 * cols) >> 3;
      // (E4M3: format 0 of A and B; bf16: 1)
      const uint32_t id = (1u << 4) | (kFp8 ? 0u : (1u << 7) | (1u << 10)) | (n8 << 17) | ((uint32_t)(kTile >> 4) << 24);
      constexpr uint32_t swizzle = kFp8 ? kSwizzle64B : kSwizzle128B, group = 8 * Z::kChunkRow;
      const uint64_t a0 = smem_desc(smem_u32(ring), 16, group, swizzle), b0 = smem_desc(smem_u32(queries), 16, group, swizzle);
      const uint32_t b_chunk = (uint32_t)(cols * Z::kChunkRow) >> 4;
      uint32_t sl = 0, turn = 0, g = 0, piece = 0;
      bool ok = true;
      while (ok && walk.next()) {
        if (!(ok = wait(&s.q_full, piece++ & 1u))) break;
        for (int32_t tt = walk.t0; ok && tt < walk.t1; tt += kTile, ++g) {
          if (g >= kBuffers && !(ok = wait(&s.s_free[g & 1u], ((g >> 1) - 1) & 1u))) break;
          const uint32_t buffer = tmem + Z::kBuffer * (g & 1u);
#pragma unroll 1
          for (int c = 0; c < kChunks; c += kItemChunks) {
            if (!(ok = wait(&s.full[sl], turn))) break;
            tc_fence_after();
            const uint64_t a = a0 + (uint64_t)(sl * (Z::kItemBytes >> 4)), b = b0 + (uint64_t)(c * b_chunk);
            const uint32_t d = buffer + (Z::kSums > 1 ? c / kItemChunks * cols : 0);
            const bool fresh = Z::kSums > 1 || c == 0;
#pragma unroll
            for (int k = 0; k < kItemChunks; ++k)
#pragma unroll
              for (int st = 0; st < Z::kChunkRow / 32; ++st) {
                const uint64_t ak = a + (uint64_t)((k * Z::kChunkBytes + 32 * st) >> 4), bk = b + (uint64_t)(k * b_chunk + 2 * st);
                if (kFp8) mma_ss_pair_fp8(d, ak, bk, id, fresh && (k | st) == 0 ? 0u : 1u);
                else mma_ss_pair(d, ak, bk, id, fresh && (k | st) == 0 ? 0u : 1u);
              }
            mma_commit_pair(smem_u32(&s.empty[sl]));
            if (++sl == (uint32_t)p.slots) sl = 0, turn ^= 1u;
          }
          mma_commit_pair(smem_u32(&s.s_full[g & 1u]));
        }
        mma_commit_pair(smem_u32(&s.q_free));
      }
      mma_commit_pair(smem_u32(&s.mma_end));
      if (!mbar_wait(smem_u32(&s.mma_end), 0, nullptr, kWaitBudgetNs)) report(p.dev_status, MLA_ERR_DEVICE_TIMEOUT);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- queries, bf16
    if (!kFp8 && elect_one_sync()) {
      const uint32_t bar = cluster_addr(smem_u32(&s.q_full), 0);
      uint32_t piece = 0;
      // The last piece's queries are free with its last MMA, which may be any time away: the budget starts
      // again as long as rows come in.
      auto wait_piece = [&](uint32_t parity) {
        for (uint32_t seen = *(volatile uint32_t *)&s.items;;) {
          if (mbar_wait(smem_u32(&s.q_free), parity, &s.abort, kWaitBudgetNs)) return true;
          const uint32_t now = *(volatile uint32_t *)&s.items;
          if (now == seen || *(volatile int *)&s.abort) break;
          seen = now;
        }
        set_abort(s, p.dev_status);
        return false;
      };
      while (walk.next()) {
        if (piece > 0 && !wait_piece((piece - 1) & 1u)) break;
        ++piece;
        if (first_block) mbar_arrive_expect_tx(smem_u32(&s.q_full), (uint32_t)(2 * query_bytes<kFp8>(p.half_heads)));
        for (int c = 0; c < kChunks; c += 3)
          tma_load_3d_pair(smem_u32(queries) + c * cols * Z::kChunkRow, &maps.q, 0, walk.b * p.heads + (int)rank * p.head_stride, c, bar);
      }
      if (s.abort && first_block && piece > 0) (void)mbar_wait(smem_u32(&s.q_full), (piece - 1) & 1u, nullptr, kDrainBudgetNs);
    }
  } else if (warp >= kWeighWarp0) {
    // ---------------------------------------------------------------- weights
    // Thread = a token and a quarter of the heads: half a block's.
    const int quad = warp & 3, half = quad >> 1, rows32 = quad & 1, part = (warp - kWeighWarp0) >> 2;
    const int r = rows32 * 32 + lane, thread = tid - 32 * kWeighWarp0;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t s_bar = cluster_addr(smem_u32(&s.s_free[0]), 0), q_bar = cluster_addr(smem_u32(&s.q_full), 0);
    const int real = min(max(p.heads - half * p.head_stride, 0), p.head_stride);
    const int split = (real / 2 + 15) / 16 * 16, i_from = part == 0 ? 0 : split, i_to = part == 0 ? min(split, real) : real;
    uint32_t g = 0, piece = 0;
    bool ok = true;
    while (ok && walk.next()) {
      const uint32_t turn = piece & 1u;
      // every head's lse and scale, for 2^x; a rest of +inf, which no lse has, marks a head with -inf
      for (int h = thread; h < p.heads; h += 32 * kWeighWarps) {
        const float l = p.lse[(int64_t)walk.b * p.heads + h];
        const float x = l * kLog2e;
        s.lse[turn][h] = x;
        s.lse_rest[turn][h] = l == -INFINITY ? INFINITY : fabsf(x) < INFINITY ? fmaf(l, kLog2e, -x) + l * kLog2eRest : 0.f;
      }
      if (kFp8) {
        // the queries as sums of two E4M3 numbers: both blocks find every head's scale, each splits its own
        // heads; a warp takes four at a time.  (Columns of no head hold what they held.)
        if (piece > 0 && !(ok = warp_wait(s, &s.q_free, (piece - 1) & 1u, p.dev_status))) break;
        for (int h0 = 4 * (warp - kWeighWarp0); h0 < p.heads; h0 += 4 * kWeighWarps) {
          uint4 w[4][3];  // dims 8 x .. 8 x + 7 for x = lane, lane + 32, lane + 64
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.q + ((int64_t)walk.b * p.heads + min(h0 + m, p.heads - 1)) * kRow);
#pragma unroll
            for (int v = 0; v < 3; ++v) w[m][v] = lane + 32 * v < kRow / 8 ? src[lane + 32 * v] : make_uint4(0, 0, 0, 0);
          }
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
            const int h = h0 + m;
            if (h >= p.heads) break;
            uint32_t u[12];
#pragma unroll
            for (int v = 0; v < 3; ++v) u[4 * v] = w[0][v].x, u[4 * v + 1] = w[0][v].y, u[4 * v + 2] = w[0][v].z, u[4 * v + 3] = w[0][v].w;
#pragma unroll
            for (int v = 0; v < 3; ++v) w[0][v] = w[1][v], w[1][v] = w[2][v], w[2][v] = w[3][v];
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 12; ++k) top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xffff0000u))));
            // magnitudes as whole numbers of the same order
            top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            // 2^e with top * 2^e in (224, 448], in two factors that are fp32 numbers; a head of zeros, or of
            // nothing above 2^-100, is scaled as if it had that
            int e = 135 - max((int)(__float_as_uint(top) >> 23), 27);
            const float up0 = __uint_as_float((uint32_t)(127 + e / 2) << 23);
            if (top * up0 * __uint_as_float((uint32_t)(127 + e - e / 2) << 23) > 448.f) --e;
            const float up1 = __uint_as_float((uint32_t)(127 + e / 2) << 23), up2 = __uint_as_float((uint32_t)(127 + e - e / 2) << 23);
            if (lane == 0) s.factor[turn][h] = ldexpf(p.scale_log2, -e), s.factor_rest[turn][h] = ldexpf(p.scale_rest, -e);
            const int i = h - (int)rank * p.head_stride, j = p.half_heads + i;
            if (i < 0 || i >= p.head_stride) continue;
#pragma unroll
            for (int v = 0; v < 3; ++v) {
              uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float x0 = __uint_as_float(u[4 * v + k] << 16) * up1 * up2, x1 = __uint_as_float(u[4 * v + k] & 0xffff0000u) * up1 * up2;
                x0 += x0 - x0, x1 += x1 - x1;  // an infinity, which E4M3 has not, becomes a NaN
                const uint32_t c = f32x2_to_e4m3x2(x0, x1), back = e4m3x2_to_f16x2(c);
                const __half2 h2 = *reinterpret_cast<const __half2 *>(&back);
                const uint32_t d = f32x2_to_e4m3x2(x0 - __low2float(h2), x1 - __high2float(h2));
                hi[k >> 1] |= c << 16 * (k & 1);
                lo[k >> 1] |= d << 16 * (k & 1);
              }
              // chunk x / 8, in which 16-byte units are exchanged by the row (64-byte swizzle)
              const int x = lane + 32 * v, unit = (x >> 1) & 3;
              if (x < kRow / 8) {
                uint8_t *at = queries + (x >> 3) * cols * 64 + (x & 1) * 8;
                *reinterpret_cast<uint2 *>(at + i * 64 + ((unit ^ ((i >> 1) & 3)) << 4)) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2 *>(at + j * 64 + ((unit ^ ((j >> 1) & 3)) << 4)) = make_uint2(lo[0], lo[1]);
              }
            }
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_release_cluster(q_bar);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.head_full));
      if (!(ok = warp_wait(s, &s.head_full, turn, p.dev_status))) break;
      ++piece;
      const int at = half * p.head_stride;
      const float *lse = &s.lse[turn][at], *lse_rest = &s.lse_rest[turn][at], *factor = &s.factor[turn][at], *factor_rest = &s.factor_rest[turn][at];
      auto weight = [&](float x, int h) {
        const float c = kFp8 ? factor[h] : p.scale_log2, rest = kFp8 ? factor_rest[h] : p.scale_rest;
        // (An infinite score stays what it is: the rest is not negative, and where it is 0 the bound takes the NaN.)
        return ex2_approx(fmaf(x, c, -lse[h]) + fminf(fmaf(x, rest, -lse_rest[h]), 1e30f));
      };
      // This warp's heads (32 at most) that count, a bit each: those there are, without those of lse -inf, whose
      // weights, NaN for a score of NaN or +inf, are not added.  (A comparison a weight in place of the bit took
      // 22.3 us for 21.3, 20 x 4,096 tokens of 128 heads, and 17 registers more.)
      const uint32_t live = __ballot_sync(0xffffffffu, i_from + lane < i_to && lse_rest[i_from + lane] < INFINITY);
      for (int32_t tt = walk.t0; tt < walk.t1; tt += kTile, ++g) {
        const int32_t t = tt + (int)rank * kOwn + r;
        const bool mine = half == 0 && part == 0 && t < walk.t1;
        const float before = mine && p.previous ? p.previous[(int64_t)walk.b * p.previous_stride + t] : 0.f;
        if (!(ok = warp_wait(s, &s.s_full[g & 1u], (g >> 1) & 1u, p.dev_status))) break;
        tc_fence_after();
        const uint32_t src = lanes + Z::kBuffer * (g & 1u);
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll 1
        for (int i = i_from; i < i_to; i += 16) {
          const uint32_t counts = live >> (i - i_from);
          // what adds up to a score: hi and lo, or the thirds of the dims
          constexpr int kTerms = kFp8 ? 2 : Z::kSums;
          uint32_t x[kTerms][16];
#pragma unroll
          for (int j = 0; j < kTerms; ++j) tmem_ld16(src + j * (kFp8 ? p.half_heads : cols) + i, x[j]);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < kTerms; ++j) tmem_loaded16(x[j]);
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float a = __uint_as_float(x[0][k]), b = __uint_as_float(x[0][k + 1]);
#pragma unroll
            for (int j = 1; j < kTerms; ++j) a += __uint_as_float(x[j][k]), b += __uint_as_float(x[j][k + 1]);
            a = weight(a, i + k);
            b = weight(b, i + k + 1);
            if (counts & 1u << k) sum0 += a;
            if (counts & 2u << k) sum1 += b;
          }
        }
        s.sum[g & 1u][r][2 * half + part] = sum0 + sum1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.sum_full[g & 1u][rows32]));
        if (!(ok = warp_wait(s, &s.sum_full[g & 1u][rows32], (g >> 1) & 1u, p.dev_status))) break;
        const float4 four = *reinterpret_cast<const float4 *>(s.sum[g & 1u][r]);
        const float sum = (four.x + four.y) + (four.z + four.w);
        // S is read, and nobody needs this tile's sums
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(s_bar + 8 * (g & 1u));
        if (mine) p.mass[(int64_t)walk.b * p.mass_stride + t] = p.previous ? fmaf(p.decay, before, sum) : sum;
      }
    }
  }

  // ---------------------------------------------------------------- the end
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // nobody arrives at a block that has left
  tc_fence_after();
  if (warp == 3) tmem_dealloc_pair(tmem, Z::kCols);
}

// ---------------------------------------------------------------------------- host

mla_status_t invalid(const char *why) {
  set_error_detail(why);
  return MLA_ERR_INVALID_ARGUMENT;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

mla_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  set_error_detail(cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

// Rows of 576 elements (bf16, or bytes) viewed as {64, rows, 9 chunks}: boxes {64, box_rows, chunks}, swizzled
// by a chunk's row (one chunk: as {576, rows}).
bool encode(const void *base, int64_t rows, bool bytes, int box_rows, int chunks, CUtensorMap *m) {
  tmap::EncodeTiledFn fn = tmap::encode_fn();
  if (!fn) return false;
  const cuuint64_t size = bytes ? 1 : 2;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)kChunks}, strides[2] = {kRow * size, 64 * size};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)chunks}, estr[3] = {1, 1, 1};
  if (chunks == 1) dims[0] = kRow;
  return fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, chunks == 1 ? 2 : 3, const_cast<void *>(base), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, bytes ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// All shared memory, a block on every SM, in pairs; as many pairs as run at once.
template <bool kFp8, int kBox>
cudaError_t launch(const Maps &maps, Params p, int dev, cudaStream_t stream) {
  static std::atomic<int> known[64];
  constexpr int kSmem = 232448;
  const auto kernel = mass_kernel<kFp8, kBox>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  int pairs = dev >= 0 && dev < 64 ? known[dev].load(std::memory_order_acquire) : 0;
  if (pairs == 0) {
    int sms = 0;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cfg.gridDim = dim3(sms / 2 * 2);
    cfg.numAttrs = 1;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    pairs = std::min(pairs, kMaxPairs);
    if (dev >= 0 && dev < 64) known[dev].store(pairs, std::memory_order_release);
  }
  p.pairs = pairs;
  p.slots = slots_for<kFp8>(p.half_heads);
  cfg.gridDim = dim3(2 * pairs);
  cfg.stream = stream;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

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
  if (a.num_blocks <= 0 || a.num_blocks > INT32_MAX || a.num_blocks * a.block_size > INT32_MAX || a.max_blocks_per_seq <= 0 ||
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
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status_of(e);
  const int log2 = a.block_size == 16 ? 4 : a.block_size == 32 ? 5 : a.block_size == 64 ? 6 : a.block_size == 128 ? 7 : 8;
  Params p;
  p.q = (const __nv_bfloat16 *)a.q;
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
  p.page_log2 = log2;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.batch = a.batch;
  p.heads = a.heads;
  p.longest = (int32_t)std::min<int64_t>(a.max_tokens, (int64_t)a.max_blocks_per_seq * a.block_size);
  p.head_stride = (a.heads + 1) / 2;
  p.half_heads = (p.head_stride + 15) / 16 * 16;
  const double scale = (double)a.scale * a.kv_scale * kLog2eExact;
  p.scale_log2 = (float)scale;
  if ((double)p.scale_log2 > scale) p.scale_log2 = std::nextafterf(p.scale_log2, 0.f);
  p.scale_rest = (float)(scale - (double)p.scale_log2);
  p.decay = a.decay;
  Maps maps;
  if (!encode(a.cache, a.num_blocks * a.block_size, a.fp8, std::min(a.block_size, kOwn), 1, &maps.k) ||
      !encode(a.cache, a.num_blocks * a.block_size, a.fp8, kOwn, kItemChunks, &maps.k3) ||
      !encode(a.q, (int64_t)a.batch * a.heads, false, p.half_heads, 3, &maps.q)) {
    set_error_detail("cannot describe q or the cache to TMA");
    return MLA_ERR_CUDA;
  }
  const cudaStream_t st = (cudaStream_t)stream;
  e = a.fp8 ? (log2 == 4 ? launch<true, 16>(maps, p, dev, st) : log2 == 5 ? launch<true, 32>(maps, p, dev, st) : launch<true, 64>(maps, p, dev, st))
            : (log2 == 4   ? launch<false, 16>(maps, p, dev, st)
               : log2 == 5 ? launch<false, 32>(maps, p, dev, st)
                           : launch<false, 64>(maps, p, dev, st));
  return status_of(e);
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
