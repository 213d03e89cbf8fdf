// Decode of a batch whose requests begin with the same tokens (sm_103a), see
// mla_decode_shared.
//
// What is computed: the absorbed-form decode of decode_tc.cu, softmax(scale
// q . row) over 576 dims times the rows' first 512, for R = batch * heads query
// rows.  A cached row is 1,152 bytes and 1,088 products a query row: 128 query
// rows that meet it at once (16 heads of 8 requests as well as 128 heads of one)
// need 278,528 flops for those bytes, about this GPU's ratio of the two rates.
// So query rows are packed to 128 over the shared tokens, whatever request they
// are of, and the tokens behind are each request's own (its heads, padded to 128).
//
// Work.  A chain is 128 query rows on a run of tokens: kind A, one for each 128
// packed rows, on the shared tokens; kind B, one for each request, on its own.
// (Packing that leaves as many chains as there are requests, 128 heads for one,
// saves nothing: then there is no kind A and B runs over all tokens.  A request
// shorter than the shared part is a B over what it sees.)  Chains are cut into
// units of 64 tokens (128 where pages hold that) and the units dealt out to the
// pairs of SMs in order, in runs of equal cost; every block works the deal out
// from the lengths, so that there is no plan to keep.  A run's piece of a chain
// leaves a partial result with its log-sum-exp and merge_kernel joins them; a
// whole request in one piece is written at once.
//
// A pair of SMs shares each MMA (cta_group::2, M = 128: 64 rows in each SM,
// 128 lanes hold two halves of N).  An SM's tensor memory then holds O of 64 rows
// x 512 dims (256 columns) and two S of 64 x 256 tokens (128 columns each), which
// no single-SM shape does without computing scores twice.
//   S [128 x 256] = Q K^T   B operand: each block's 128 tokens x 576 dims
//   O [128 x 512] += P V    B operand: all 256 tokens, each block's 256 dims
// So a token's row comes into the pair's shared memory almost twice: 17 items of
// 16 KB a tile and SM, against 4,352 clk of MMAs.  K and V stream through rings of
// four and three slots, each with an issuing thread of its own for its MMAs; P is
// handed over and its room freed by halves of the tile, so that the softmax of
// tile t runs under P V(t-1) and Q K(t+1).
//
// What bounds it: a tile takes ~4,900 clk on the whole chain of 8,192 tokens.  A slot's round
// (its MMAs, the news to the loader, ~900 clk from L2, the news to the issuer) is
// ~1,850 clk, and seven slots of it are 60 bytes a clock of the 64 that the MMAs
// would take; queries (72 KB), P (32 KB) and the rings fill the shared memory.
// Around the tiles a call has ~2 us of deal and set-up, ~4 us until the first P V,
// ~4 us at each change of chain, and 5 us of merge with its launch.  64 requests
// of 128 heads on 8,192 + 1 to 777 tokens: 110 us (1.35 PFLOP/s), 59% of the
// tensor cores' cycles.  Its 28.3 tiles a pair are 139,000 of the kernel's 206,000 clk,
// deal, first P V and changes of chain some 20,000; where the rest, a fifth, goes
// has not been measured.  From the same 64: one ring and one issuing thread 195 us;
// two rings and two threads 163; P by halves 140; eight softmax warps for four
// 110.  Waits that acquire at cluster scope instead of the block's cost a
// microsecond each in such a chain (436 us).  Issuing threads as converged warps
// 116 to 126 us, the K loader so 121, the V loader as one thread 113; each
// tile's maximum found a tile ahead 123; a piece's O stored under the next
// one's first scores 113; rows prefetched to L2 by the tensor copies 111 for 104.
//
// Pieces are f16 in units of a power of two for 64 dims of a row.  bf16 (as
// mla_decode's) made the error of `out` 0.0024 of its size, this 0.0019, for 3% of
// the time; fp32 took 4 to 10%.  P is bf16, as V is: one MMA has one type.
//
// Rows behind the last token of a chain.  Scores of their columns are masked, and
// P V stops at the next multiple of 16 tokens; V rows up to there have to be
// zeros (0 * NaN is NaN), which a tensor copy cannot write for rows that exist.
// The last items of such a chain are copied by a warp's threads instead.
//
// Warp roles: 0 loads Q and K, 1 issues Q K^T (first block of the pair; in the
// other it passes on that P is written), 2 loads V, 3 issues P V and owns the
// tensor memory, 4-11 run the softmax and write results (thread = a row and a
// quarter of a tile's tokens, or of the 512 dims).  Every wait is bounded; one that
// runs out reports MLA_ERR_DEVICE_TIMEOUT and ends the block's other waits.
#include <algorithm>
#include <atomic>
#include <cmath>

#include <cuda_fp16.h>

#include "cluster.cuh"
#include "common.cuh"
#include "tmap.h"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace shared {

using namespace sm100;

constexpr int kRows = 128;          // query rows of a chain
constexpr int kHalf = kRows / 2;    // ... in each block of a pair
constexpr int kTile = 256;          // tokens of a tile
constexpr int kOwn = kTile / 2;     // ... whose scores' operand a block holds
constexpr int kGroup = 64;          // tokens of an item of V
constexpr int kChunks = kRow / 64;  // 9
constexpr int kChunkBytes = kHalf * 128;  // 8 KB: 64 rows x 64 dims
constexpr int kItemBytes = 16384;
// Queries of few heads (kind B, up to kFew): 16 rows a chunk.  Their MMAs read 64 rows from each chunk's
// start on, the rest being what follows: rows of no query, whose results nobody reads.
constexpr int kFew = 16, kFewChunkBytes = kFew * 128, kFewBytes = 32768;
constexpr int kSlotsK = 4, kSlotsV = 3;
constexpr int kThreads = 384;
constexpr int kSoftmaxWarp0 = 4, kSoftmaxWarps = 8;
constexpr uint32_t kColO = 0, kColS = 256, kCols = 512;
// A chain's start (queries and first keys without MMAs under them, its end's O) costs as much as eight units:
// 12 and 20 instead of 16 took 49.5 and 51.5 us for 49 (159 requests of 16 heads on 4,096 + 16 to 1,024 tokens).
constexpr int64_t kUnitCost = 2, kChainCost = 16;
constexpr int kMaxPairs = 256;
constexpr uint64_t kWaitBudgetNs = 100000000ull;
constexpr uint64_t kDrainBudgetNs = 10000000ull;
constexpr float kRescaleThreshold = 8.0f;  // log2 units, as in decode_tc.cu

struct __align__(1024) Smem {
  uint8_t k[kSlotsK][kItemBytes];
  uint8_t v[kSlotsV][kItemBytes];
  uint8_t q[kChunks][kChunkBytes];
  uint8_t p[kTile / 64][kChunkBytes];  // P: 64 rows x 64 tokens each
  float max[2][kHalf][4];              // of a row's quarters of the tokens, by tile parity
  float sum[kHalf][4];
  // Loads (k_full, v_full, q_full) and what the MMAs wait for (s_free, p_full, o_free, tail_full) count
  // in the first block, whose loaders announce the bytes of both blocks' loads; the others in each.
  // P is handed over and freed by halves (128 tokens), so that a tile's is written while the P V of
  // the tile before still runs.
  uint64_t k_full[kSlotsK], k_empty[kSlotsK], v_full[kSlotsV], v_empty[kSlotsV], q_full[2], q_free[2];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2], pv_done[2], o_free, mma_end;  // (s, pv_done: by tile parity; p: by half)
  uint64_t tail_full;                    // the other block has filled its items with zeros
  uint64_t p_here[2];                    // the other block: its P is written, to be said to the first
  uint64_t max_full[2][2], sum_full[2];  // [tile parity][32 rows]: their four warps have written
  int64_t total, start_cost, share[2], warp_cost[kThreads / 32];  // of all chains; where the first starts; this pair's
  int32_t start_chain;
  uint32_t tmem_base;
  int abort;
};
static_assert(kChunks * kFewChunkBytes <= kFewBytes && kFewBytes + (kChunks - 1) * kFewChunkBytes + kChunkBytes <= kChunks * kChunkBytes,
              "two sets of few heads' queries, and what is read behind them, lie in q");
static_assert(kSlotsV < 4, "two items with zeros have to be read before two more are filled: tail_full holds one round");
static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory");

struct Maps {
  CUtensorMap k;  // {576, rows}, box {64, min(block_size, 128)}
  CUtensorMap v;  // {64, rows, 9}, box {64, 64, 2} (pages of 64 rows and more)
  CUtensorMap q;  // {64, batch * heads, 9}, box {64, 64, 3}
  CUtensorMap q_few;  // the same, box {64, kFew, 9}
};

// What a piece's result needs is kept by chain: its pieces are those of the pairs first to last, in
// slots chain + pair (chains counted in their kind; pairs and chains both ascend, so slots do).
struct Pieces {
  int32_t first, last;
};

struct Params {
  const __nv_bfloat16 *cache;
  const int32_t *shared_table, *shared_blocks, *block_table, *seq_lens;
  __nv_bfloat16 *out;
  float *lse;
  int32_t *dev_status;
  Pieces *pieces_a, *pieces_b;
  __half *o_a, *o_b;         // [slot][row][512], in units of
  float *unit_a, *unit_b;    // [slot][8][row], one for 64 dims
  float *lse_a, *lse_b;      // [slot][row]
  int32_t num_blocks, block_size, page_log2, max_shared_blocks, max_blocks_per_seq, batch, heads, pairs;
  float scale_log2;
};

// The chains of a call, from what the device holds.
struct Chains {
  int32_t shared;  // tokens in common
  int32_t packed;  // chains of kind A, 0: none
  int32_t longest;
  int32_t unit;    // tokens that chains are dealt out by: 64, or the rows of a box where that is more
  __device__ Chains(const Params &p, int32_t shared_blocks, bool speak) {
    if (shared_blocks < 0 || shared_blocks > p.max_shared_blocks) {
      if (speak) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
      shared_blocks = min(max(shared_blocks, 0), p.max_shared_blocks);
    }
    shared = shared_blocks << p.page_log2;
    packed = (int32_t)(((int64_t)p.batch * p.heads + kRows - 1) / kRows);
    if (packed >= p.batch || shared == 0) packed = 0;
    longest = p.max_blocks_per_seq << p.page_log2;
    unit = p.block_size >= kOwn ? kOwn : kGroup;
  }
  __device__ int32_t length(int32_t L) const { return min(max(L, 0), longest); }
  // The first token of the own chain of a request of L tokens.
  __device__ int32_t from(int32_t L) const { return packed > 0 && L >= shared ? shared : 0; }
  __device__ int32_t units(int32_t L) const { return (L - from(L) + unit - 1) / unit; }
  __device__ int32_t units_a() const { return (shared + unit - 1) / unit; }
  static __device__ int64_t cost(int32_t units) { return units > 0 ? kChainCost + kUnitCost * units : 0; }
  __device__ int64_t cost_a() const { return packed * cost(units_a()); }
};

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {  // of numbers that are mostly small
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Pair w's share of cost C over n pairs is [bound(w), bound(w + 1)); a unit belongs where its place,
// its chain's start and kChainCost and kUnitCost for each unit before it, lies.
__device__ __forceinline__ int64_t bound(int64_t C, int32_t n, int32_t w) { return quotient(w * C + n - 1, n); }
// No pair's share is shorter than a unit, so that a chain has no hole between its first and last pair.
__device__ __forceinline__ int32_t pairs_for(int64_t C, int32_t pairs) {
  return (int32_t)min((int64_t)pairs, max((int64_t)1, C / kUnitCost));
}
__device__ __forceinline__ Pieces pieces_of(int64_t start, int32_t units, int64_t C, int32_t n) {
  Pieces r;
  r.first = (int32_t)quotient((start + kChainCost) * n, C);
  r.last = (int32_t)quotient((start + kChainCost + kUnitCost * (units - 1)) * n, C);
  return r;
}

// A pair's pieces in order.
struct Walk {
  const Params *p;
  const Chains *ch;
  int64_t x0, x1, at;  // the pair's share, the next chain's start
  int32_t next_chain;
  // the current piece: kind, chain, tokens [t0, t1), all of the chain
  bool packed, whole;
  int32_t chain, t0, t1;
  __device__ Walk(const Params &params, const Chains &c, const Smem &s) : p(&params), ch(&c) {
    x0 = s.share[0];
    x1 = s.share[1];
    at = s.start_cost;
    next_chain = s.start_chain;
  }
  __device__ bool next() {
    const int32_t all = ch->packed + p->batch;
    while (next_chain < all && at < x1) {
      packed = next_chain < ch->packed;
      chain = packed ? next_chain : next_chain - ch->packed;
      const int32_t end = packed ? ch->shared : ch->length(p->seq_lens[chain]);
      const int32_t first = packed ? 0 : ch->from(end);
      const int32_t unit = ch->unit, units = (end - first + unit - 1) / unit;
      ++next_chain;
      if (units <= 0) continue;
      const int64_t place = at + kChainCost;
      at = place + kUnitCost * units;
      const int64_t k0 = x0 <= place ? 0 : (x0 - place + kUnitCost - 1) / kUnitCost;
      const int64_t k1 = x1 <= place ? 0 : min((int64_t)units, (x1 - place + kUnitCost - 1) / kUnitCost);
      if (k0 >= k1) continue;
      t0 = first + (int32_t)k0 * unit;
      t1 = min(end, first + (int32_t)k1 * unit);
      whole = !packed && first == 0 && t0 == 0 && t1 == end;
      return true;
    }
    return false;
  }
  __device__ bool few() const { return !packed && p->heads <= kFew; }
  // The packed query row of the piece's first.
  __device__ int32_t row() const { return packed ? chain * kRows : chain * p->heads; }
};

// The chains' pieces, for the merge; by a warp.
__device__ void write_pieces(const Params &p, const Chains &ch, int64_t C) {
  const int lane = threadIdx.x & 31;
  const int32_t n = pairs_for(C, p.pairs);
  for (int32_t i = lane; i < ch.packed; i += 32) p.pieces_a[i] = pieces_of(i * ch.cost(ch.units_a()), ch.units_a(), C, n);
  int64_t before = ch.cost_a();
  for (int32_t b0 = 0; b0 < p.batch; b0 += 32) {
    const int32_t units = b0 + lane < p.batch ? ch.units(ch.length(p.seq_lens[b0 + lane])) : 0;
    int64_t incl = ch.cost(units);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (units > 0) p.pieces_b[b0 + lane] = pieces_of(before + incl - ch.cost(units), units, C, n);
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

__device__ __forceinline__ int groups_of(int n) { return (n + kGroup - 1) / kGroup; }

__device__ __forceinline__ void set_abort(Smem &s, int32_t *dev_status) {
  s.abort = 1;
  report(dev_status, MLA_ERR_DEVICE_TIMEOUT);
}

// Every lane polls, then the warp agrees.
__device__ __forceinline__ bool warp_wait(Smem &s, uint64_t *bar, uint32_t parity, int32_t *dev_status) {
  const bool ok = mbar_wait(smem_u32(bar), parity, &s.abort, kWaitBudgetNs);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0) set_abort(s, dev_status);
  return false;
}

// The block of token t, and the pool's row of t in it: 0 if it is none (reported).
__device__ __forceinline__ int32_t block_of(const Params &p, const Walk &w, int32_t t) {
  const int32_t page = t >> p.page_log2;
  return t < w.ch->shared ? p.shared_table[page] : p.block_table[(int64_t)w.chain * p.max_blocks_per_seq + page];
}
__device__ __forceinline__ int32_t pool_row(const Params &p, int32_t blk, int32_t t) {
  if (blk < 0 || blk >= p.num_blocks) {
    report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    return 0;
  }
  return (blk << p.page_log2) + (t & (p.block_size - 1));
}

// kBox: rows of a box of K, min(block_size, 128).
template <int kBox>
__global__ void __launch_bounds__(kThreads, 1) shared_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem &s = *reinterpret_cast<Smem *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int32_t pair = (int32_t)cluster_id();
  const bool first_block = rank == 0;

  if (tid == 0) {
    auto init = [](uint64_t *bar, int count) { mbar_init(smem_u32(bar), count); };
    for (int i = 0; i < kSlotsK; ++i) init(&s.k_full[i], 1), init(&s.k_empty[i], 1);
    for (int i = 0; i < kSlotsV; ++i) init(&s.v_full[i], 1), init(&s.v_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      init(&s.s_full[i], 1);
      init(&s.s_free[i], 2 * kSoftmaxWarps);
      init(&s.max_full[0][i], 4);
      init(&s.max_full[1][i], 4);
      init(&s.sum_full[i], 4);
      init(&s.p_full[i], 5);
      init(&s.p_here[i], 4);
      init(&s.p_free[i], 1);
      init(&s.q_full[i], 1);
      init(&s.q_free[i], 1);
      init(&s.pv_done[i], 1);
    }
    init(&s.o_free, 2 * kSoftmaxWarps);
    init(&s.mma_end, 2);
    init(&s.tail_full, 1);
    s.abort = 0;
    fence_mbarrier_init_cluster();
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.q_few);
  }
  if (warp == 3) {
    tmem_alloc_pair(smem_u32(&s.tmem_base), kCols);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_arrive();  // barriers and tensor memory, to both blocks
  griddep_wait();
  // The merge's launch is over with before this grid's end; its blocks come as this grid's leave (384 threads of 168
  // registers, two of them spilled, leave none for a warp of 90).
  griddep_launch_dependents();

  // ---------------------------------------------------------------- the deal
  const int32_t shared_blocks = *p.shared_blocks, my_length = tid < p.batch ? p.seq_lens[tid] : 0;
  const Chains ch(p, shared_blocks, blockIdx.x == 0 && tid == 0);
  {
    // costs of a block's worth of requests, and the sum over those before each
    int64_t before = ch.cost_a(), mine = 0, start = 0;
    auto sum_up = [&](int32_t b0, int32_t L) {
      if (blockIdx.x == 0 && L != ch.length(L)) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
      mine = b0 + tid < p.batch ? ch.cost(ch.units(ch.length(L))) : 0;
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
    sum_up(0, my_length);
    for (int32_t b0 = kThreads; b0 < p.batch; b0 += kThreads) {
      __syncthreads();
      sum_up(b0, b0 + tid < p.batch ? p.seq_lens[b0 + tid] : 0);
    }
    const int64_t C = before, each = ch.cost(ch.units_a());
    const int32_t n = pairs_for(C, p.pairs);
    const int64_t x0 = pair < n ? bound(C, n, pair) : C;
    if (tid == 0) {
      s.total = C;
      s.share[0] = x0;
      s.share[1] = pair < n ? bound(C, n, pair + 1) : C;
      const bool in_a = ch.packed > 0 && x0 < ch.cost_a();
      s.start_chain = in_a ? (int32_t)quotient(x0, each) : ch.packed + p.batch;
      s.start_cost = in_a ? s.start_chain * each : C;
    }
    __syncthreads();
    auto find = [&](int32_t b0) {
      if (mine > 0 && start <= x0 && x0 < start + mine) {
        s.start_chain = ch.packed + b0 + tid;
        s.start_cost = start;
      }
    };
    if (p.batch <= kThreads) {
      find(0);
    } else {
      before = ch.cost_a();
      for (int32_t b0 = 0; b0 < p.batch; b0 += kThreads) {
        sum_up(b0, b0 + tid < p.batch ? p.seq_lens[b0 + tid] : 0);
        find(b0);
        __syncthreads();
      }
    }
  }
  __syncthreads();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  Walk walk(p, ch, s);

  // The issuing roles are one thread each.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (mbar_wait(smem_u32(bar), parity, &s.abort, kWaitBudgetNs)) return true;
    set_abort(s, p.dev_status);
    return false;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- Q and K
    if (elect_one_sync()) {
      constexpr int kBoxes = kOwn / kBox;
      const uint32_t q_bar = cluster_addr(smem_u32(&s.q_full[0]), 0), k_bar = cluster_addr(smem_u32(&s.k_full[0]), 0);
      uint32_t sl = 0, turn = 1, items = 0, piece = 0;
      bool ok = true, was_few = false, have = walk.next();
      // This block's tokens of a tile (both blocks load at least a box of every item, so that neither falls
      // behind the rings' rounds: where the second has none of its own, the tile's first, for masked columns).
      auto own_of = [&](const Walk &w, int32_t tt) { return tt + (int)rank * kOwn < w.t1 ? tt + (int)rank * kOwn : tt; };
      auto boxes_of = [](int32_t tokens) { return max(1, (min(tokens, kOwn) + kBox - 1) / kBox); };
      int32_t blk[kBoxes], y[kBoxes];
      auto look_up = [&](const Walk &w, int32_t tt) {
        const int32_t own = own_of(w, tt);
#pragma unroll
        for (int i = 0; i < kBoxes; ++i) blk[i] = own + i * kBox < w.t1 ? block_of(p, w, own + i * kBox) : 0;
      };
      auto settle = [&](const Walk &w, int32_t tt) {
        const int32_t own = own_of(w, tt);
#pragma unroll
        for (int i = 0; i < kBoxes; ++i) y[i] = own + i * kBox < w.t1 ? pool_row(p, blk[i], own + i * kBox) : 0;
      };
      if (have) {
        look_up(walk, walk.t0);
        settle(walk, walk.t0);
      }
      while (ok && have) {
        Walk ahead = walk;
        const bool more = ahead.next();
        // the last piece's queries stay where they are read while these come, if neither takes all the room
        if (piece >= 2 && !(ok = wait(&s.q_free[piece & 1u], ((piece >> 1) - 1) & 1u))) break;
        const bool few = walk.few(), beside = few && was_few;
        if (piece >= 1 && !beside && !(ok = wait(&s.q_free[(piece - 1) & 1u], ((piece - 1) >> 1) & 1u))) break;
        was_few = few;
        const uint32_t bar = q_bar + 8 * (piece & 1u);
        if (few) {
          if (first_block) {
            mbar_arrive_expect_tx(smem_u32(&s.q_full[piece & 1u]), kChunks * kFewChunkBytes);
            tma_load_3d_pair(smem_u32(s.q[0]) + (piece & 1u) * kFewBytes, &maps.q_few, 0, walk.row(), 0, bar);
          }
        } else {
          if (first_block) mbar_arrive_expect_tx(smem_u32(&s.q_full[piece & 1u]), 2 * kChunks * kChunkBytes);
          for (int c = 0; c < kChunks; c += 3) tma_load_3d_pair(smem_u32(s.q[c]), &maps.q, 0, walk.row() + (int)rank * kHalf, c, bar);
        }
        ++piece;
        for (int32_t tt = walk.t0; ok && tt < walk.t1; tt += kTile) {
          const int32_t n = min(kTile, walk.t1 - tt);
          const int32_t boxes = boxes_of(rank == 0 || n <= kOwn ? n : n - kOwn);
          const int32_t others = boxes_of(rank == 1 || n <= kOwn ? n : n - kOwn);
          const uint32_t bytes = (uint32_t)((boxes + others) * kBox * 128);
          // what comes next: its table entries are read while this tile's loads are issued ...
          const bool last = tt + kTile >= walk.t1;
          if (!last) look_up(walk, tt + kTile);
          else if (more) look_up(ahead, ahead.t0);
          for (int c = 0; c < kChunks; ++c) {
            if (!(ok = wait(&s.k_empty[sl], turn))) break;
            if (first_block) mbar_arrive_expect_tx(smem_u32(&s.k_full[sl]), bytes);
            const uint32_t dst = smem_u32(s.k[0]) + sl * kItemBytes, full = k_bar + 8 * sl;
#pragma unroll
            for (int i = 0; i < kBoxes; ++i)
              if (i < boxes) tma_load_2d_pair(dst + i * kBox * 128, &maps.k, 64 * c, y[i], full);
            ++items;
            if (++sl == kSlotsK) sl = 0, turn ^= 1u;
          }
          // ... and looked at when they are
          if (!last) settle(walk, tt + kTile);
          else if (more) settle(ahead, ahead.t0);
        }
        walk = ahead;
        have = more;
      }
      if (s.abort && first_block) {  // let the loads in flight land in both blocks
        for (uint32_t i = items > kSlotsK ? items - kSlotsK : 0; i < items; ++i)
          (void)mbar_wait(smem_u32(&s.k_full[i % kSlotsK]), (i / kSlotsK) & 1u, nullptr, kDrainBudgetNs);
        for (uint32_t i = piece > 2 ? piece - 2 : 0; i < piece; ++i)
          (void)mbar_wait(smem_u32(&s.q_full[i & 1u]), (i >> 1) & 1u, nullptr, kDrainBudgetNs);
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- V
    constexpr int kBoxV = kBox < kGroup ? kBox : kGroup, kBoxes = kGroup / kBoxV;
    const uint32_t v_bar = cluster_addr(smem_u32(&s.v_full[0]), 0), tail_bar = cluster_addr(smem_u32(&s.tail_full), 0);
    uint32_t sl = 0, turn = 1, items = 0;
    auto advance = [&]() {
      ++items;
      if (++sl == kSlotsV) sl = 0, turn ^= 1u;
    };
    bool ok = true;
    while (ok && walk.next()) {
      int32_t blk[kBoxes];
      auto look_up = [&](int32_t tt) {
#pragma unroll
        for (int i = 0; i < kBoxes; ++i) blk[i] = tt + i * kBoxV < walk.t1 ? block_of(p, walk, tt + i * kBoxV) : 0;
      };
      look_up(walk.t0);
      for (int32_t tt = walk.t0; ok && tt < walk.t1; tt += kGroup) {
        const int cnt = min(kGroup, walk.t1 - tt), boxes = (cnt + kBoxV - 1) / kBoxV;
        int32_t y[kBoxes];
#pragma unroll
        for (int i = 0; i < kBoxes; ++i) y[i] = i < boxes ? pool_row(p, blk[i], tt + i * kBoxV) : 0;
        if (cnt & 15) {
          // the chain's last tokens: the warp's threads copy, with zeros up to the next multiple of 16
          const uint32_t slots[2] = {sl, sl + 1 == kSlotsV ? 0 : sl + 1};
          const int rows = (cnt + 15) & ~15, r0 = lane >> 4, c = lane & 15;  // 16 bytes c of a row's 256, every other row
          for (int j = 0; ok && j < 2; ++j) {
            if (!(ok = warp_wait(s, &s.v_empty[sl], turn, p.dev_status))) break;
            const uint32_t ring = smem_u32(s.v[sl]) + (c >> 3) * kChunkBytes;
            const __nv_bfloat16 *src = p.cache + 64 * (4 * j + 2 * (int)rank) + 8 * c;
#pragma unroll
            for (int i = 0; i < kBoxes; ++i)
              for (int r = i * kBoxV + r0; r < min(rows, (i + 1) * kBoxV); r += 2)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ring + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                             "l"(src + (r < cnt ? (int64_t)y[i] + (r - i * kBoxV) : 0) * kRow), "r"(r < cnt ? 16 : 0)
                             : "memory");
            advance();
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_proxy_async_shared();
          __syncwarp();
          if (ok && lane == 0) {
            if (first_block) {
              mbar_arrive(smem_u32(&s.v_full[slots[0]]));
              mbar_arrive(smem_u32(&s.v_full[slots[1]]));
            } else {
              mbar_arrive_release_cluster(tail_bar);
            }
          }
          break;
        }
        const uint32_t bytes = (uint32_t)(2 * 2 * boxes * kBoxV * 128);  // two chunks, two blocks
        if (tt + kGroup < walk.t1) look_up(tt + kGroup);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (!(ok = warp_wait(s, &s.v_empty[sl], turn, p.dev_status))) break;
          if (elect_one_sync()) {
            if (first_block) mbar_arrive_expect_tx(smem_u32(&s.v_full[sl]), bytes);
            const int chunk = 4 * j + 2 * (int)rank;
            const uint32_t dst = smem_u32(s.v[0]) + sl * kItemBytes, bar = v_bar + 8 * sl;
            if (kBox >= kGroup) {
              tma_load_3d_pair(dst, &maps.v, 0, y[0], chunk, bar);
            } else {
#pragma unroll
              for (int i = 0; i < kBoxes; ++i) {
                if (i >= boxes) break;
                tma_load_2d_pair(dst + i * kBoxV * 128, &maps.k, 64 * chunk, y[i], bar);
                tma_load_2d_pair(dst + kChunkBytes + i * kBoxV * 128, &maps.k, 64 * (chunk + 1), y[i], bar);
              }
            }
          }
          __syncwarp();
          advance();
        }
      }
    }
    if (s.abort && first_block && lane == 0)
      for (uint32_t i = items > kSlotsV ? items - kSlotsV : 0; i < items; ++i)
        (void)mbar_wait(smem_u32(&s.v_full[i % kSlotsV]), (i / kSlotsV) & 1u, nullptr, kDrainBudgetNs);
  } else if (warp == 1) {
    if (elect_one_sync()) {
      if (first_block) {
        // -------------------------------------------------------------- S = Q K^T
        constexpr uint32_t id = idesc_bf16_f32(kRows, kTile, 0);
        const uint32_t a0 = desc_low(s.q[0], 16), b0 = desc_low(s.k[0], 16);
        uint32_t sl = 0, turn = 0, g = 0, piece = 0;
        bool ok = true;
        while (ok && walk.next()) {
          if (!(ok = wait(&s.q_full[piece & 1u], (piece >> 1) & 1u))) break;
          const uint32_t chunk = (walk.few() ? kFewChunkBytes : kChunkBytes) >> 4;
          const uint32_t q0 = a0 + (walk.few() ? (piece & 1u) * (kFewBytes >> 4) : 0);
          for (int32_t tt = walk.t0; ok && tt < walk.t1; tt += kTile, ++g) {
            if (g >= 2 && !(ok = wait(&s.s_free[g & 1u], ((g >> 1) - 1) & 1u))) break;
            const uint32_t d = tmem + kColS + 128 * (g & 1u);
            for (int c = 0; c < kChunks; ++c) {
              if (!(ok = wait(&s.k_full[sl], turn))) break;
              tc_fence_after();
              const uint32_t a = q0 + c * chunk, b = b0 + sl * (kItemBytes >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ss_pair_low(d, a + 2 * k, b + 2 * k, id, (c | k) ? 1u : 0u);
              mma_commit_pair(smem_u32(&s.k_empty[sl]));
              if (++sl == kSlotsK) sl = 0, turn ^= 1u;
            }
            mma_commit_pair(smem_u32(&s.s_full[g & 1u]));
          }
          mma_commit_pair(smem_u32(&s.q_free[piece++ & 1u]));
        }
        mma_commit_pair(smem_u32(&s.mma_end));
      } else {
        // The other block's P, said to the first when both warps of a half have written it.
        const uint32_t bar = cluster_addr(smem_u32(&s.p_full[0]), 0);
        uint32_t g = 0;
        bool ok = true;
        while (ok && walk.next())
          for (int32_t tt = walk.t0; ok && tt < walk.t1; tt += kTile, ++g)
            for (int h = 0; ok && h < 2; ++h)
              if ((ok = wait(&s.p_here[h], g & 1u))) mbar_arrive_release_cluster(bar + 8 * h);
      }
      // Both blocks stay until the end of all MMAs has been said to both: that is the last arrival of the MMAs at
      // a block's barriers, and the meeting at the end does not wait for them.
      if (!mbar_wait(smem_u32(&s.mma_end), 0, nullptr, kWaitBudgetNs)) report(p.dev_status, MLA_ERR_DEVICE_TIMEOUT);
    }
  } else if (warp == 3) {
    // ---------------------------------------------------------------- O += P V
    if (first_block && elect_one_sync()) {
      constexpr uint32_t id = idesc_bf16_f32(kRows, 256, 1);
      const uint32_t a0 = desc_low(s.p[0], 16), b0 = desc_low(s.v[0], kChunkBytes);
      uint32_t sl = 0, turn = 0, g = 0, piece = 0, tails = 0;
      bool ok = true;
      while (ok && walk.next()) {
        if (piece > 0 && !(ok = wait(&s.o_free, (piece - 1) & 1u))) break;  // the last piece's O is out
        ++piece;
        uint32_t more = 0;
        for (int32_t tt = walk.t0; ok && tt < walk.t1; tt += kTile, ++g) {
          const int32_t n = min(kTile, walk.t1 - tt);
          if (!(ok = wait(&s.s_free[g & 1u], (g >> 1) & 1u))) break;  // O is at this tile's scale
          for (int h = 0; h < 2; ++h) {
            if (!(ok = wait(&s.p_full[h], g & 1u))) break;
            for (int gr = 2 * h; ok && gr < min(2 * h + 2, groups_of(n)); ++gr) {
              const int cnt = min(kGroup, n - gr * kGroup), steps = (cnt + 15) >> 4;
              if ((cnt & 15) && !(ok = wait(&s.tail_full, tails++ & 1u))) break;
              for (int j = 0; j < 2; ++j) {
                if (!(ok = wait(&s.v_full[sl], turn))) break;
                tc_fence_after();
                const uint32_t a = a0 + gr * (kChunkBytes >> 4), b = b0 + sl * (kItemBytes >> 4);
                const uint32_t d = tmem + kColO + 128 * j;
                if (steps == 4) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) mma_ss_pair_low(d, a + 2 * k, b + 128 * k, id, k > 0 ? 1u : more);
                } else {
                  for (int k = 0; k < steps; ++k) mma_ss_pair_low(d, a + 2 * k, b + 128 * k, id, k > 0 ? 1u : more);
                }
                mma_commit_pair(smem_u32(&s.v_empty[sl]));
                if (++sl == kSlotsV) sl = 0, turn ^= 1u;
              }
              more = 1;
            }
            if (!ok) break;
            mma_commit_pair(smem_u32(&s.p_free[h]));
          }
          if (ok) mma_commit_pair(smem_u32(&s.pv_done[g & 1u]));
        }
      }
      mma_commit_pair(smem_u32(&s.mma_end));
      if (!mbar_wait(smem_u32(&s.mma_end), 0, nullptr, kWaitBudgetNs)) report(p.dev_status, MLA_ERR_DEVICE_TIMEOUT);
    } else if (!first_block) {
      if (pair == 0) write_pieces(p, ch, s.total);
    }
  } else {
    // ---------------------------------------------------------------- softmax, results
    // Thread = a row and a quarter of the tile's tokens (64), or of the 512 dims: tensor memory's lanes
    // hold 64 rows x the two halves of N, and two warps share a lane's columns.
    const int quad = warp & 3, half = quad >> 1, part = (warp - kSoftmaxWarp0) >> 2;
    const int rows32 = quad & 1, r = rows32 * 32 + lane;  // this block's row
    const int place = 2 * half + part;                    // which 64 tokens
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t s_bar = cluster_addr(smem_u32(&s.s_free[0]), 0), o_bar = cluster_addr(smem_u32(&s.o_free), 0);
    const uint32_t p_bar = smem_u32(first_block ? &s.p_full[half] : &s.p_here[half]);
    const float c = p.scale_log2;
    uint32_t g = 0, tops = 0, sums = 0;  // tiles, and those with a maximum and pieces with a sum of this warp's
    bool ok = true;
    while (ok && walk.next()) {
      float m_used = -INFINITY, l = 0.f;
      // this warp's rows that are queries; one without any only hands on
      const int real_rows = min(32, (walk.packed ? kRows : p.heads) - (int)rank * kHalf - rows32 * 32);
      for (int32_t tt = walk.t0; tt < walk.t1; tt += kTile, ++g) {
        const int32_t mine = walk.t1 - tt - place * 64;  // real tokens of this quarter, if below 64
        if (!(ok = warp_wait(s, &s.s_full[g & 1u], (g >> 1) & 1u, p.dev_status))) break;
        tc_fence_after();
        if (real_rows <= 0) {
          if (g > 0 && !(ok = warp_wait(s, &s.p_free[half], (g - 1) & 1u, p.dev_status))) break;
          if (lane == 0) {
            mbar_arrive_cluster(s_bar + 8 * (g & 1u));
            mbar_arrive(p_bar);
          }
          continue;
        }
        uint32_t x[64];
        const uint32_t src = lanes + kColS + 128 * (g & 1u) + 64 * part;
        tmem_ld32(src, x);
        tmem_ld32(src + 32, x + 32);
        tmem_wait_ld();
        tmem_loaded32(x);
        tmem_loaded32(x + 32);
        tc_fence_before();
        if (mine < 64) {
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (k >= mine) x[k] = 0xff800000u;  // -inf
        }
        float t0 = __uint_as_float(x[0]), t1 = __uint_as_float(x[1]);
#pragma unroll
        for (int k = 2; k < 64; k += 2) {
          t0 = fmaxf(t0, __uint_as_float(x[k]));
          t1 = fmaxf(t1, __uint_as_float(x[k + 1]));
        }
        s.max[tops & 1u][r][place] = fmaxf(t0, t1);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.max_full[tops & 1u][rows32]));
        if (!(ok = warp_wait(s, &s.max_full[tops & 1u][rows32], (tops >> 1) & 1u, p.dev_status))) break;
        const float4 four = *reinterpret_cast<const float4 *>(s.max[tops & 1u][r]);
        ++tops;
        const float top = fmaxf(fmaxf(four.x, four.y), fmaxf(four.z, four.w)) * c;
        float alpha = 1.f;
        if (top > m_used + kRescaleThreshold || tt == walk.t0) {
          alpha = m_used == -INFINITY ? 0.f : ex2_approx(m_used - top);
          m_used = top;
        }
        const float shift = m_used == -INFINITY ? 0.f : m_used;
        if (tt > walk.t0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O is free once the P V of the tile before is done
          if (!(ok = warp_wait(s, &s.pv_done[(g - 1) & 1u], ((g - 1) >> 1) & 1u, p.dev_status))) break;
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            uint32_t o[32];
            tmem_ld32(lanes + kColO + 128 * part + 32 * i, o);
            tmem_wait_ld();
            tmem_loaded32(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(lanes + kColO + 128 * part + 32 * i, o);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(s_bar + 8 * (g & 1u));  // S is read, O at this tile's scale
        uint32_t w[32];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float a = ex2_approx(fmaf(__uint_as_float(x[2 * k]), c, -shift)), b = ex2_approx(fmaf(__uint_as_float(x[2 * k + 1]), c, -shift));
          s0 += a;
          s1 += b;
          __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
          w[k] = *reinterpret_cast<uint32_t *>(&two);
        }
        l = l * alpha + (s0 + s1);
        // this half of P was last read by the P V of the tile before
        if (g > 0 && !(ok = warp_wait(s, &s.p_free[half], (g - 1) & 1u, p.dev_status))) break;
#pragma unroll
        for (int u = 0; u < 8; ++u)
          *reinterpret_cast<uint4 *>(s.p[place] + r * 128 + ((u ^ (r & 7)) << 4)) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_bar);
      }
      if (!ok) break;
      // ---- O / l
      if (real_rows > 0) {
        s.sum[r][place] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.sum_full[rows32]));
        if (!warp_wait(s, &s.sum_full[rows32], sums++ & 1u, p.dev_status)) break;
        const float4 four = *reinterpret_cast<const float4 *>(s.sum[r]);
        l = (four.x + four.y) + (four.z + four.w);
      }
      if (!warp_wait(s, &s.pv_done[(g - 1) & 1u], ((g - 1) >> 1) & 1u, p.dev_status)) break;
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse = l == 0.f ? -INFINITY : (m_used + log2f(l)) * 0.69314718055994531f;
      if (real_rows > 0) {
        const int row0 = (int)rank * kHalf + rows32 * 32;  // of the chain
        const bool whole = walk.whole;
        const int unit_rows = walk.packed ? kRows : p.heads;
        uint16_t *dst;  // bf16 of a whole request, f16 of a piece
        float *lse_dst, *unit_dst = nullptr;
        if (whole) {
          const int64_t at = (int64_t)walk.chain * p.heads + row0;
          dst = (uint16_t *)p.out + at * kVDim;
          lse_dst = p.lse ? p.lse + at : nullptr;
        } else {
          const int64_t slot = ((int64_t)walk.chain + pair) * unit_rows;
          dst = (uint16_t *)(walk.packed ? p.o_a : p.o_b) + (slot + row0) * kVDim;
          lse_dst = (walk.packed ? p.lse_a : p.lse_b) + slot + row0;
          unit_dst = (walk.packed ? p.unit_a : p.unit_b) + slot * 8 + (4 * part + 2 * half) * unit_rows + row0 + lane;
        }
        dst += 256 * part + 128 * half + 8 * (lane & 7);
        // 64 dims at a time by way of this warp's part of P, so that 8 threads store a row's 128 bytes
        uint8_t *stage = s.p[place] + rows32 * 32 * 128;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          uint32_t o[64];
          tmem_ld32(lanes + kColO + 128 * part + 64 * i, o);
          tmem_ld32(lanes + kColO + 128 * part + 64 * i + 32, o + 32);
          tmem_wait_ld();
          tmem_loaded32(o);
          tmem_loaded32(o + 32);
          if (whole) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
              o[k] = *reinterpret_cast<uint32_t *>(&two);
            }
          } else {
            // f16 in units of a power of two that takes the largest of the 64 to [2^14, 2^15): a rounding of
            // 2^-12 of it at most, where bf16's 2^-9 of each was as large as all other errors of `out` together
            float top0 = 0.f, top1 = 0.f;
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
              top0 = fmaxf(top0, fabsf(__uint_as_float(o[k])));
              top1 = fmaxf(top1, fabsf(__uint_as_float(o[k + 1])));
            }
            const float top = fmaxf(top0, top1) * inv;
            const uint32_t e = top < INFINITY ? max(__float_as_uint(top) >> 23, 15u) : 141u;  // (141: as they are)
            const float by = inv * __uint_as_float((268u - e) << 23);
            if (lane < real_rows) unit_dst[i * unit_rows] = __uint_as_float((e - 14u) << 23);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              __half2 two = __floats2half2_rn(__uint_as_float(o[2 * k]) * by, __uint_as_float(o[2 * k + 1]) * by);
              o[k] = *reinterpret_cast<uint32_t *>(&two);
            }
          }
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rr = 4 * k + (lane >> 3);
            if (rr < real_rows)
              *reinterpret_cast<uint4 *>(dst + (int64_t)rr * kVDim + 64 * i) =
                  *reinterpret_cast<const uint4 *>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
          }
        }
        __syncwarp();
        if (lane < real_rows && place == 0 && lse_dst) lse_dst[lane] = lse;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(o_bar);
    }
  }

  // ---------------------------------------------------------------- the end
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // nobody arrives at a block that has left
  tc_fence_after();
  if (warp == 3) tmem_dealloc_pair(tmem, kCols);
}

// ---------------------------------------------------------------------------- merge

// A warp joins the pieces of a query row: those of its packed chain on the shared tokens and those of
// its request's own.  out = sum_i e^(lse_i - M) o_i / sum_i e^(lse_i - M), in fp32.
constexpr int kMergeThreads = 256, kMergeFlight = 4;

__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const Params p) {
  const int lane = threadIdx.x & 31;
  const uint32_t row = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);  // (below 2^27)
  const uint32_t b = row / (uint32_t)p.heads, h = row - b * p.heads, in_a = row % kRows;
  griddep_wait();
  if (b >= (uint32_t)p.batch) return;
  // all at once: what is not there is not looked at
  const int32_t shared_blocks = *p.shared_blocks, length = p.seq_lens[b];
  const Pieces all_own = p.pieces_b[b], all_com = p.pieces_a[row / kRows], none = {0, -1};
  const Chains ch(p, shared_blocks, false);
  const int32_t L = ch.length(length);
  const Pieces own = ch.units(L) > 0 ? all_own : none;
  const Pieces com = ch.packed > 0 && L >= ch.shared ? all_com : none;
  const int na = com.last - com.first + 1, nb = own.last - own.first + 1;
  if (ch.from(L) == 0 && nb == 1) return;  // written at once
  // the first piece of either kind: its rows, its units (of this lane's 8 dims of each half) and its lse
  const int64_t slot_a = (int64_t)(row / kRows) + com.first, slot_b = (int64_t)b + own.first;
  const uint4 *oa = reinterpret_cast<const uint4 *>(p.o_a + (slot_a * kRows + in_a) * kVDim) + lane;
  const uint4 *ob = reinterpret_cast<const uint4 *>(p.o_b + (slot_b * p.heads + h) * kVDim) + lane;
  const float *ua = p.unit_a + (slot_a * 8 + (lane >> 3)) * kRows + in_a, *ub = p.unit_b + (slot_b * 8 + (lane >> 3)) * p.heads + h;
  const float *la = p.lse_a + slot_a * kRows + in_a, *lb = p.lse_b + slot_b * p.heads + h;
  float m = -INFINITY, z = 0.f, acc[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
  for (int i0 = 0; i0 < na + nb; i0 += kMergeFlight) {
    float l[kMergeFlight], unit[kMergeFlight][2];
    uint4 x[kMergeFlight][2];
#pragma unroll
    for (int u = 0; u < kMergeFlight; ++u) {
      const int i = i0 + u, j = i - na;
      l[u] = -INFINITY;
      unit[u][0] = unit[u][1] = 0.f;
      x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
      if (j < nb) {
        const bool a = j < 0;
        const int step = a ? i : j, rows = a ? kRows : p.heads;
        const uint4 *o = (a ? oa : ob) + (int64_t)step * rows * (kVDim / 8);
        const float *units = (a ? ua : ub) + (int64_t)step * rows * 8;
        l[u] = (a ? la : lb)[(int64_t)step * rows];
        unit[u][0] = units[0];
        unit[u][1] = units[4 * rows];
        x[u][0] = o[0];
        x[u][1] = o[32];
      }
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < kMergeFlight; ++u) top = fmaxf(top, l[u]);
    const float keep = m == -INFINITY ? 0.f : ex2_approx((m - top) * 1.4426950408889634f);
    m = top;
    z *= keep;
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] *= keep;
#pragma unroll
    for (int u = 0; u < kMergeFlight; ++u) {
      const float w = l[u] == -INFINITY ? 0.f : ex2_approx((l[u] - (m == -INFINITY ? 0.f : m)) * 1.4426950408889634f);
      z += w;
      const uint32_t v[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
      if (w != 0.f) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 two = __half22float2(*reinterpret_cast<const __half2 *>(&v[k]));
          const float f = w * unit[u][k >> 2];
          acc[2 * k] += f * two.x;
          acc[2 * k + 1] += f * two.y;
        }
      }
    }
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  uint4 o[2];
  uint32_t *ow = reinterpret_cast<uint32_t *>(o);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    __nv_bfloat162 two = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    ow[k] = *reinterpret_cast<uint32_t *>(&two);
  }
  uint4 *dst = reinterpret_cast<uint4 *>(p.out + (int64_t)row * kVDim);
  dst[lane] = o[0];
  dst[32 + lane] = o[1];
  if (lane == 0 && p.lse) p.lse[row] = z == 0.f ? -INFINITY : m + logf(z);
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

// Pairs of SMs of the current device that run at once, 0 if it cannot be asked.
int pairs_current() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_acquire);
  if (n > 0) return n;
  const int smem = (int)sizeof(Smem) + 1024;
  if (cudaFuncSetAttribute(shared_kernel<16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(shared_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(shared_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(shared_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return 0;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms / 2 * 2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, shared_kernel<64>, &cfg) != cudaSuccess || n < 1) return 0;
  n = std::min(n, kMaxPairs);
  known[dev].store(n, std::memory_order_release);
  return n;
}

struct Layout {
  size_t pieces_a, pieces_b, lse_a, lse_b, unit_a, unit_b, o_a, o_b, total;
};

Layout layout(int64_t batch, int64_t heads, int64_t pairs) {
  const int64_t packed = (batch * heads + kRows - 1) / kRows;
  Layout l;
  size_t o = 0;
  l.pieces_a = o; o = align256(o + sizeof(Pieces) * packed);
  l.pieces_b = o; o = align256(o + sizeof(Pieces) * batch);
  l.lse_a = o;    o = align256(o + sizeof(float) * (packed + pairs) * kRows);
  l.lse_b = o;    o = align256(o + sizeof(float) * (batch + pairs) * heads);
  l.unit_a = o;   o = align256(o + sizeof(float) * (packed + pairs) * kRows * 8);
  l.unit_b = o;   o = align256(o + sizeof(float) * (batch + pairs) * heads * 8);
  l.o_a = o;      o = align256(o + sizeof(__half) * (packed + pairs) * kRows * kVDim);
  l.o_b = o;      o = align256(o + sizeof(__half) * (batch + pairs) * heads * kVDim);
  l.total = o;
  return l;
}

}  // namespace shared
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_decode_shared_workspace_size(int32_t batch, int32_t num_heads) {
  if (batch < 0 || batch > 1 << 20 || num_heads < 1 || num_heads > kHeads) return 0;
  const int pairs = shared::pairs_current();
  return pairs > 0 ? shared::layout(batch, num_heads, pairs).total : 0;
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
  if (num_blocks <= 0 || num_blocks > INT32_MAX || num_blocks * block_size > INT32_MAX || max_blocks_per_seq <= 0 ||
      (int64_t)max_blocks_per_seq * block_size > 1 << 30 || (int64_t)max_shared_blocks * block_size > 1 << 30)
    return invalid("num_blocks, max_blocks_per_seq or max_shared_blocks out of range");
  if (batch > 1 << 20) return invalid("batch > 2^20");
  if (batch == 0) return MLA_OK;
  if (!q || !cache || !shared_blocks || (max_shared_blocks > 0 && !shared_table) || !block_table || !seq_lens || !out || !workspace)
    return invalid("null pointer");
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16)) return invalid("q, cache and out must be 16-byte aligned");
  if (!aligned(shared_table, 4) || !aligned(shared_blocks, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4))
    return invalid("shared_table, shared_blocks, block_table, seq_lens and lse must be 4-byte aligned");
  if (!aligned(workspace, 256)) return invalid("workspace must be 256-byte aligned");
  const int pairs = pairs_current();
  if (pairs < 1) return status_of(cudaErrorInvalidDevice);
  const Layout l = layout(batch, num_heads, pairs);
  if (workspace_bytes < l.total) {
    set_error_detail("workspace is smaller than mla_decode_shared_workspace_size()");
    return MLA_ERR_WORKSPACE_TOO_SMALL;
  }
  Maps maps;
  const int64_t rows = num_blocks * block_size;
  if (!tmap::encode_2d(&maps.k, cache, rows, (uint32_t)std::min(block_size, kOwn)) ||
      !tmap::encode_3d(&maps.v, cache, rows, kGroup, 2) ||
      !tmap::encode_3d(&maps.q, q, (int64_t)batch * num_heads, kHalf, 3) ||
      !tmap::encode_3d(&maps.q_few, q, (int64_t)batch * num_heads, kFew, kChunks)) {
    set_error_detail("cannot describe q or the cache to TMA");
    return MLA_ERR_CUDA;
  }
  char *ws = (char *)workspace;
  Params p;
  p.cache = (const __nv_bfloat16 *)cache;
  p.shared_table = shared_table;
  p.shared_blocks = shared_blocks;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.out = (__nv_bfloat16 *)out;
  p.lse = lse;
  p.dev_status = dev_status;
  p.pieces_a = (Pieces *)(ws + l.pieces_a);
  p.pieces_b = (Pieces *)(ws + l.pieces_b);
  p.lse_a = (float *)(ws + l.lse_a);
  p.lse_b = (float *)(ws + l.lse_b);
  p.unit_a = (float *)(ws + l.unit_a);
  p.unit_b = (float *)(ws + l.unit_b);
  p.o_a = (__half *)(ws + l.o_a);
  p.o_b = (__half *)(ws + l.o_b);
  p.num_blocks = (int32_t)num_blocks;
  p.block_size = block_size;
  for (p.page_log2 = 4; 1 << p.page_log2 < block_size;) ++p.page_log2;
  p.max_shared_blocks = max_shared_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.batch = batch;
  p.heads = num_heads;
  p.pairs = pairs;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem) + 1024;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = block_size == 16   ? cudaLaunchKernelEx(&cfg, shared_kernel<16>, maps, p)
                  : block_size == 32 ? cudaLaunchKernelEx(&cfg, shared_kernel<32>, maps, p)
                  : block_size == 64 ? cudaLaunchKernelEx(&cfg, shared_kernel<64>, maps, p)
                                     : cudaLaunchKernelEx(&cfg, shared_kernel<128>, maps, p);
  if (e != cudaSuccess) return status_of(e);
  const int64_t warps = kMergeThreads / 32;
  cfg.gridDim = dim3((unsigned)(((int64_t)batch * num_heads + warps - 1) / warps));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return status_of(cudaLaunchKernelEx(&cfg, merge_kernel, p));
}

}  // extern "C"
