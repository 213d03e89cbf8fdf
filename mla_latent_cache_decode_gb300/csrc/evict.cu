// Thinning out a full latent cache (sm_103a): which tokens of a request stay
// (select_kernel) and the move of their rows to the front of the request's
// pages (compact_kernel).  What each token's weight is, mass.cu computes.
//
// Select.  Request b of L tokens keeps K at most.  L <= K: all of them.  Else
// the first `sink` and the last `recent` ones, and of the M = L - sink - recent
// between them the r = K - sink - recent of the largest weight, the earlier one
// first where weights are equal.  That is a threshold: the r-th largest weight
// T, and of the tokens with weight T the first ones.  A weight becomes a 32-bit
// key of the same order (-0 as +0, NaN below everything), and T is found from
// its top bits down, 11, 11 and 10 of them: a histogram of the keys that agree
// with what is known of T, and the bin in which the r-th lies.  Then one pass in
// order of position writes what stays.  A request is one cluster's: each block
// takes a contiguous part, the histograms and counts are added up through
// distributed shared memory, and nothing depends on the order of atomics.
//
// What bounds it: latency.  131,072 + 7 x 1,024 tokens take 23 us on eight blocks a
// request: 10 without the three passes (loads, counts, the places), and 3.3 to 5 a
// pass, of which the histograms' atomics are nothing measurable and two meetings
// of the cluster with three trips through distributed shared memory most.  (Every
// block adding up all bins of all blocks took 32 us; keys in registers 23, and 9.8
// instead of 5.2 for four short requests by the code's size; equal digits counted
// once for a warp 35.)  20 x 4,096 tokens: 7.9 us, a block each.
//
// Compact.  keep[b][0..n) ascends strictly, so token j comes from keep[j] >= j
// and a row's target is never behind its source: in order of j, writing rows
// below J touches no source of rows from J on.  A phase loads a run of rows into
// registers, waits until every block of the cluster has (the targets are sources
// of the same phase at most), and stores them; nothing waits between phases.
// Columns do not depend on each other, so a row is cut into nine slices (128
// bytes of a bf16 row, 64 of an E4M3 one) and a cluster moves one slice of one
// request of one layer.  A row's two pages are looked up once, by one thread, a
// phase ahead.
//
// What bounds it: memory, by the bytes in flight.  20 x 4,096 tokens cut to 2,048: 94 MB
// in 18.8 us (5.0 TB/s, 74% of the copy rate); eight E4M3 layers: 138 MB in 27.5 us.
// Before the blocks met without ordering memory: 20.5 and 32 us.  From there: eight
// units a thread 22.7 and 35.7 us, sixteen 26 and 44; three slices a row 25 and 36,
// whole rows 40; two blocks an SM asked for instead of four 26 us; registers for eight
// to an SM 20.9, by spilling (for six, as it is, 40 registers and one or two spilled).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "cluster.cuh"
#include "common.cuh"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace evict {

using namespace sm100;

// What block `rank` of the cluster holds at this block's address p.
__device__ __forceinline__ uint32_t remote_u32(const uint32_t *p, uint32_t rank) {
  return cluster_load_u32(cluster_addr(smem_u32(p), rank));
}

// ---------------------------------------------------------------------------- select

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelKeys = 16384;  // keys of a block's part that shared memory holds; longer parts are read again

struct SelectParams {
  const float *mass;
  int64_t mass_stride;
  const int32_t *seq_lens;
  int32_t *keep;
  int32_t *new_lens;
  int32_t *dev_status;
  int32_t max_tokens, budget, sink, recent, blocks;
};

struct SelectSmem {
  uint32_t hist[3][kBins];
  uint32_t warp_sum[kSelWarps];
  uint32_t warp_more[kSelWarps], warp_same[kSelWarps];
  uint32_t totals[2];  // of this block: tokens that stay without asking, tokens of weight T
  uint32_t found, above;
  uint32_t bins[kBins / 2], bins_total;  // of a cluster's block: its share of the bins, over all blocks
  uint32_t keys[kSelKeys];
};

// Order as the weights', equal where they are; NaN lowest.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Of a number of each thread, the sum over the threads before.
__device__ __forceinline__ uint32_t sum_before(SelectSmem &s, uint32_t mine) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // the last call's sums are read
  if (lane == 31) s.warp_sum[warp] = incl;
  __syncthreads();
  return incl - mine + __reduce_add_sync(0xffffffffu, lane < warp ? s.warp_sum[lane] : 0);
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  SelectSmem &s = *reinterpret_cast<SelectSmem *>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = p.blocks, b = blockIdx.x / nb;
  const int rank = nb > 1 ? (int)cluster_rank() : 0;
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&s.hist[0][0])[i] = 0;
  griddep_wait();
  int32_t L = p.seq_lens[b];
  if (L < 0 || L > p.max_tokens) {
    if (tid == 0 && rank == 0) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    L = L < 0 ? 0 : p.max_tokens;
  }
  const int32_t K = p.budget;
  int32_t *keep = p.keep + (int64_t)b * K;
  if (tid == 0 && rank == 0) p.new_lens[b] = min(L, K);
  if (L <= K) {  // (the same for every block of the cluster)
    for (int64_t j = rank * kSelThreads + tid; j < K; j += nb * kSelThreads) keep[j] = j < L ? (int32_t)j : -1;
    return;
  }
  // this block's tokens, and each warp's
  const int32_t wpart = ((L + nb * kSelWarps - 1) / (nb * kSelWarps) + 31) & ~31;
  const int32_t part = wpart * kSelWarps;
  const int32_t first = min((int64_t)L, (int64_t)rank * part), last = min((int64_t)L, (int64_t)first + part);
  const bool held = last - first <= kSelKeys;
  const float *mass = p.mass + (int64_t)b * p.mass_stride;
  const int32_t lo = p.sink, hi = L - p.recent;  // the tokens that are asked about
  auto key_at = [&](int32_t t) { return held ? s.keys[t - first] : key_of(mass[t]); };
  if (held) {
    for (int32_t t0 = first + tid; t0 < last; t0 += 16 * kSelThreads) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = t0 + i * kSelThreads < last ? mass[t0 + i * kSelThreads] : 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t0 + i * kSelThreads < last) s.keys[t0 + i * kSelThreads - first] = key_of(x[i]);
    }
  }
  __syncthreads();
  uint32_t known = 0, need = (uint32_t)(K - p.sink - p.recent);
  const int shifts[4] = {21, 10, 0, 0};
#pragma unroll 1
  for (int pass = 0; pass < 3 && need > 0; ++pass) {
    const int shift = shifts[pass], above_shift = pass == 0 ? 32 : shifts[pass - 1];
    const uint32_t mask = (1u << (pass == 2 ? 10 : 11)) - 1;
    uint32_t *hist = s.hist[pass];
    for (int32_t t = max(first, lo) + tid; t < min(last, hi); t += kSelThreads) {
      const uint32_t k = key_at(t);
      if (pass == 0 || (k >> above_shift) == known) atomicAdd(&hist[(k >> shift) & mask], 1u);
    }
    // the bin, from the top down, that holds the need-th largest
    if (nb == 1) {
      __syncthreads();
      const int bin = kBins - 1 - 2 * tid;
      const uint32_t n0 = hist[bin], n1 = hist[bin - 1], excl = sum_before(s, n0 + n1);
      if (excl < need && need <= excl + n0 + n1) {
        const bool second = excl + n0 < need;
        s.found = (uint32_t)(second ? bin - 1 : bin);
        s.above = second ? excl + n0 : excl;
      }
    } else {
      // each block adds up its share of the bins over the blocks, and says what they hold together
      cluster_sync();
      const int per = kBins / nb, bin = kBins - 1 - (rank * per + tid);
      uint32_t n[8], sum = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) n[r] = tid < per && r < nb ? remote_u32(&hist[bin], r) : 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) sum += n[r];
      if (tid < per) s.bins[tid] = sum;
      const uint32_t before = sum_before(s, sum);
      if (tid == kSelThreads - 1) s.bins_total = before + sum;
      cluster_sync();
      uint32_t total[8], above = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) total[r] = r < nb ? remote_u32(&s.bins_total, r) : 0;
      int owner = 0;  // of the bin; the shares lie from the top down in order of rank
#pragma unroll
      for (int r = 0; r < 7; ++r) {
        if (owner == r && above + total[r] < need) {
          above += total[r];
          owner = r + 1;
        }
      }
      const uint32_t mine = tid < per ? remote_u32(&s.bins[tid], owner) : 0, excl = above + sum_before(s, mine);
      if (excl < need && need <= excl + mine) {
        s.found = (uint32_t)(kBins - 1 - (owner * per + tid));
        s.above = excl;
      }
    }
    __syncthreads();
    known = pass == 0 ? s.found : (known << (pass == 2 ? 10 : 11)) | s.found;
    need -= s.above;
    __syncthreads();
  }
  // With need = 0 from the start no weight is asked for; else every token above T = known stays and
  // the first `need` of those with weight T.
  const bool none = K == p.sink + p.recent;
  const int32_t w0 = min(last, first + warp * wpart), w1 = min(last, w0 + wpart);
  uint32_t more = 0, same = 0;
  for (int32_t t0 = w0; t0 < w1; t0 += 32) {
    const int32_t t = t0 + lane;
    const bool in = t < w1, middle = in && t >= lo && t < hi;
    const uint32_t k = middle && !none ? key_at(t) : 0;
    more += __popc(__ballot_sync(0xffffffffu, in && (!middle || (!none && k > known))));
    same += __popc(__ballot_sync(0xffffffffu, middle && !none && k == known));
  }
  if (lane == 0) s.warp_more[warp] = more, s.warp_same[warp] = same;
  __syncthreads();
  uint32_t my_more = s.warp_more[lane], my_same = s.warp_same[lane];
  const uint32_t total_more = __reduce_add_sync(0xffffffffu, my_more), total_same = __reduce_add_sync(0xffffffffu, my_same);
  uint32_t at_more = __reduce_add_sync(0xffffffffu, lane < warp ? my_more : 0);
  uint32_t at_same = __reduce_add_sync(0xffffffffu, lane < warp ? my_same : 0);
  if (nb > 1) {
    if (tid == 0) s.totals[0] = total_more, s.totals[1] = total_same;
    cluster_sync();
    for (int r = 0; r < rank; ++r) at_more += remote_u32(&s.totals[0], r), at_same += remote_u32(&s.totals[1], r);
  }
  // place of a token: the sure ones before it and the taken ones of weight T before it
  for (int32_t t0 = w0; t0 < w1; t0 += 32) {
    const int32_t t = t0 + lane;
    const bool in = t < w1, middle = in && t >= lo && t < hi;
    const uint32_t k = middle && !none ? key_at(t) : 0;
    const bool sure = in && (!middle || (!none && k > known)), tie = middle && !none && k == known;
    const uint32_t sures = __ballot_sync(0xffffffffu, sure), ties = __ballot_sync(0xffffffffu, tie);
    const uint32_t below = (1u << lane) - 1;
    const uint32_t ties_before = at_same + __popc(ties & below);
    const bool stays = sure || (tie && ties_before < need);
    const uint32_t place = at_more + __popc(sures & below) + min(ties_before, need);
    if (stays && place < (uint32_t)K) keep[place] = t;
    at_more += __popc(sures);
    at_same += __popc(ties);
  }
  if (nb > 1) cluster_sync();  // the others may still read this block's shared memory
}

// ---------------------------------------------------------------------------- compact

constexpr int kSlices = 9;
constexpr int kMoveThreads = 256, kMoveBlocks = 6;
constexpr int kMoveUnits = 4;  // 16-byte (4-byte: a weight) units that a thread holds in a phase

struct CompactParams {
  uint8_t *cache;
  int64_t layer_bytes;
  const int32_t *block_table;
  const int32_t *keep;
  const int32_t *seq_lens;
  const int32_t *new_lens;
  float *mass;
  int64_t mass_stride;
  int32_t *dev_status;
  int32_t batch, layers, num_blocks, block_size, max_blocks_per_seq, budget, max_tokens, blocks;
};

// The source of token j, or -1: it stays where it is, or its entry is no ascending one of the
// request's (reported).
__device__ __forceinline__ int32_t source_of(const CompactParams &p, const int32_t *keep, int32_t j, int32_t L) {
  const int32_t t = keep[j], before = j > 0 ? keep[j - 1] : -1;
  if (t < j || t >= L || before >= t) {
    report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    return -1;
  }
  return t == j ? -1 : t;
}

// Pool rows of token j's source and target, or -1: nothing to move (a block outside the pool is reported).
__device__ __forceinline__ int2 rows_of(const CompactParams &p, const int32_t *table, const int32_t *keep, int32_t j, int32_t L) {
  const int32_t t = source_of(p, keep, j, L);
  if (t < 0) return make_int2(-1, -1);
  const int32_t from_page = t / p.block_size, to_page = j / p.block_size;
  const int32_t from = table[from_page], to = table[to_page];
  if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks) {
    report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    return make_int2(-1, -1);
  }
  return make_int2(from * p.block_size + (t - from_page * p.block_size), to * p.block_size + (j - to_page * p.block_size));
}

// kLanes units of 16 bytes make a slice of a row: 8 (bf16) or 4 (E4M3).
template <int kLanes>
__global__ void __launch_bounds__(kMoveThreads, kMoveBlocks) compact_kernel(const CompactParams p) {
  static_assert(kMoveThreads % kLanes == 0, "whole rows");
  constexpr int kPass = kMoveThreads / kLanes, kRows = kPass * kMoveUnits;  // rows of one unit a thread; of a phase
  __shared__ int2 s_rows[2][kRows];  // sources and targets of a phase's rows
  const int tid = threadIdx.x, nb = p.blocks;
  const int rank = nb > 1 ? (int)cluster_rank() : 0;
  const int64_t job = blockIdx.x / nb;
  const int64_t moves = (int64_t)p.batch * p.layers * kSlices;
  const bool weights = job >= moves;  // the jobs behind the rows' are the weights' of one request
  const int32_t b = weights ? (int32_t)(job - moves) : (int32_t)(job / kSlices % p.batch);
  griddep_wait();
  int32_t L = p.seq_lens[b], n = p.new_lens[b];
  const int64_t pages = (int64_t)p.max_blocks_per_seq * p.block_size;
  const int32_t most = p.mass ? (int32_t)min(pages, (int64_t)p.max_tokens) : (int32_t)pages;
  if (L < 0 || L > most || n < 0 || n > min(L, p.budget)) {
    if (tid == 0) report(p.dev_status, MLA_ERR_DEVICE_RANGE);
    L = min(max(L, 0), most);
    n = min(max(n, 0), min(L, p.budget));
  }
  const int32_t *keep = p.keep + (int64_t)b * p.budget;
  // Every block of the cluster has this phase's values in registers.  That is all that has to be so before
  // the stores: no block reads what another writes, and a load whose value is here cannot see a later store.
  // So the blocks meet without ordering memory, which would wait for the last phase's stores to arrive.  The
  // block's own barrier takes in every word that was loaded (`seen`), so that no thread passes it with a load under way.
  auto meet = [&](uint32_t seen) {
    if (__syncthreads_or(seen == 0x9e3779b9u)) __threadfence_block();  // (the answer is used, or the question would go)
    if (nb > 1) cluster_meet();
  };
  if (weights) {
    float *mass = p.mass + (int64_t)b * p.mass_stride;
    for (int64_t base = 0; base < n; base += (int64_t)nb * kMoveThreads * kMoveUnits) {
      float x[kMoveUnits];
      bool put[kMoveUnits];
      const int64_t j0 = base + (int64_t)rank * kMoveThreads * kMoveUnits + tid;
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u) {
        const int64_t j = j0 + u * kMoveThreads;
        const int32_t t = j < n ? source_of(p, keep, (int32_t)j, L) : -1;
        put[u] = t >= 0;
        if (put[u]) x[u] = __ldcg(mass + t);
      }
      uint32_t seen = 0;
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u)
        if (put[u]) seen ^= __float_as_uint(x[u]);
      meet(seen);
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u)
        if (put[u]) mass[j0 + u * kMoveThreads] = x[u];
    }
    // every block has loaded its last weights: what is behind the new end starts over
    for (int64_t j = n + (int64_t)rank * kMoveThreads + tid; j < L; j += (int64_t)nb * kMoveThreads) mass[j] = 0.f;
    return;
  }
  const int slice = (int)(job % kSlices), layer = (int)(job / kSlices / p.batch);
  constexpr int64_t kRowBytes = kSlices * kLanes * 16;
  uint8_t *cache = p.cache + (int64_t)layer * p.layer_bytes + (slice * kLanes + tid % kLanes) * 16;
  const int32_t *table = p.block_table + (int64_t)b * p.max_blocks_per_seq;
  auto look_up = [&](int64_t base, int2 *to) {
    for (int r = tid; r < kRows; r += kMoveThreads) {
      const int64_t j = base + (int64_t)rank * kRows + r;
      to[r] = j < n ? rows_of(p, table, keep, (int32_t)j, L) : make_int2(-1, -1);
    }
  };
  look_up(0, s_rows[0]);
  __syncthreads();
  int turn = 0;
  for (int64_t base = 0; base < n; base += (int64_t)nb * kRows, turn ^= 1) {
    uint4 x[kMoveUnits];
    int32_t to[kMoveUnits];
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) {
      const int2 row = s_rows[turn][u * kPass + tid / kLanes];
      to[u] = row.y;
      if (row.y >= 0) x[u] = __ldcg(reinterpret_cast<const uint4 *>(cache + row.x * kRowBytes));
    }
    look_up(base + (int64_t)nb * kRows, s_rows[turn ^ 1]);  // the next phase's, while these load
    uint32_t seen = 0;
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u)
      if (to[u] >= 0) seen ^= x[u].x ^ x[u].y ^ x[u].z ^ x[u].w;
    meet(seen);
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u)
      if (to[u] >= 0) *reinterpret_cast<uint4 *>(cache + to[u] * kRowBytes) = x[u];
  }
}

// ---------------------------------------------------------------------------- host

mla_status_t invalid(const char *why) {
  set_error_detail(why);
  return MLA_ERR_INVALID_ARGUMENT;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool overlap(const int32_t *a, int64_t na, const int32_t *b, int64_t nb) {
  return (uintptr_t)a < (uintptr_t)(b + nb) && (uintptr_t)b < (uintptr_t)(a + na);
}

mla_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  set_error_detail(cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

template <typename Kernel, typename Params>
cudaError_t launch(Kernel kernel, int64_t grid, int threads, size_t smem, int cluster, cudaStream_t stream, const Params &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

int device_sms(cudaError_t *e) {
  int dev = 0, sms = 0;
  *e = cudaGetDevice(&dev);
  if (*e == cudaSuccess) *e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

cudaError_t allow_select_smem() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SelectSmem));
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

// Blocks of a cluster: what its longest part asks for, as long as there are fewer blocks than `enough`.
int cluster_for(int64_t wanted, int64_t clusters, int64_t enough) {
  int c = 1;
  while (c < 8 && c < wanted && clusters * c < enough) c *= 2;
  return c;
}

mla_status_t run_compact(CompactParams p, int64_t num_blocks, int row_bytes, int64_t layers, void *stream) {
  set_error_detail("");
  if (p.batch < 0 || p.budget < 0) return invalid("batch < 0 or max_keep < 0");
  if (layers < 0 || layers > INT32_MAX) return invalid("num_layers outside [0, 2^31)");
  if (p.block_size <= 0 || num_blocks <= 0 || num_blocks > INT32_MAX || num_blocks * p.block_size > INT32_MAX ||
      p.max_blocks_per_seq <= 0)
    return invalid("block_size, num_blocks and max_blocks_per_seq must be > 0, num_blocks * block_size below 2^31");
  if ((int64_t)p.max_blocks_per_seq * p.block_size > 1 << 30) return invalid("max_blocks_per_seq * block_size > 2^30");
  if ((int64_t)p.batch * layers > INT32_MAX) return invalid("batch * num_layers too large");
  if (p.batch == 0) return MLA_OK;
  if (!p.block_table || !p.seq_lens || !p.new_lens || (p.budget > 0 && !p.keep) || (layers > 0 && !p.cache)) return invalid("null pointer");
  if (!aligned(p.cache, 16)) return invalid("cache must be 16-byte aligned");
  if (!aligned(p.block_table, 4) || !aligned(p.keep, 4) || !aligned(p.seq_lens, 4) || !aligned(p.new_lens, 4) || !aligned(p.mass, 4))
    return invalid("block_table, keep, seq_lens, new_lens and mass must be 4-byte aligned");
  if (p.mass && (p.max_tokens < 0 || (p.batch > 1 && p.mass_stride < p.max_tokens)))
    return invalid("mass_stride is below max_tokens, or max_tokens < 0");
  p.layers = (int32_t)layers;
  p.num_blocks = (int32_t)num_blocks;
  p.layer_bytes = num_blocks * p.block_size * row_bytes;
  const int64_t jobs = (int64_t)p.batch * layers * kSlices + (p.mass ? p.batch : 0);
  if (jobs == 0) return MLA_OK;
  cudaError_t e;
  const int sms = device_sms(&e);
  if (e != cudaSuccess) return status_of(e);
  const int lanes = row_bytes / kSlices / 16;
  const int64_t rows = std::min<int64_t>(p.budget, (int64_t)p.max_blocks_per_seq * p.block_size);
  p.blocks = cluster_for((rows + kMoveUnits * kMoveThreads / lanes - 1) / (kMoveUnits * kMoveThreads / lanes), jobs, 4 * (int64_t)sms);
  if (jobs * p.blocks > INT32_MAX) return invalid("batch * num_layers too large");
  e = row_bytes == kRow * 2 ? launch(compact_kernel<kRow * 2 / 16 / kSlices>, jobs * p.blocks, kMoveThreads, 0, p.blocks, (cudaStream_t)stream, p)
                            : launch(compact_kernel<kRow / 16 / kSlices>, jobs * p.blocks, kMoveThreads, 0, p.blocks, (cudaStream_t)stream, p);
  return status_of(e);
}

CompactParams compact_params(void *cache, int32_t block_size, const int32_t *block_table, int32_t max_blocks_per_seq, int32_t batch,
                             const int32_t *keep, int32_t max_keep, const int32_t *seq_lens, const int32_t *new_lens, float *mass,
                             int64_t mass_stride, int32_t max_tokens, int32_t *dev_status) {
  CompactParams p = {};
  p.cache = (uint8_t *)cache;
  p.block_size = block_size;
  p.block_table = block_table;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.batch = batch;
  p.keep = keep;
  p.budget = max_keep;
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.mass = mass;
  p.mass_stride = mass_stride;
  p.max_tokens = max_tokens;
  p.dev_status = dev_status;
  return p;
}

}  // namespace evict
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_evict_select(const float *mass, int64_t mass_stride, int32_t max_tokens, const int32_t *seq_lens, int32_t batch,
                              int32_t sink, int32_t recent, int32_t *keep, int32_t max_keep, int32_t *new_lens,
                              int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_evict_select");
  set_error_detail("");
  if (batch < 0 || max_tokens < 0 || max_tokens > 1 << 30) return evict::invalid("batch < 0 or max_tokens outside [0, 2^30]");
  if (sink < 0 || recent < 0 || max_keep < 1 || (int64_t)sink + recent > max_keep)
    return evict::invalid("need max_keep >= 1, sink >= 0, recent >= 0 and sink + recent <= max_keep");
  if (batch == 0) return MLA_OK;
  if ((max_tokens > 0 && !mass) || !seq_lens || !keep || !new_lens) return evict::invalid("null pointer");
  if (!evict::aligned(mass, 4) || !evict::aligned(seq_lens, 4) || !evict::aligned(keep, 4) || !evict::aligned(new_lens, 4))
    return evict::invalid("mass, seq_lens, keep and new_lens must be 4-byte aligned");
  // (blocks of a request read its length each for itself: written over, some would go through the passes
  // without the others)
  if (evict::overlap(seq_lens, batch, new_lens, batch) || evict::overlap(seq_lens, batch, keep, (int64_t)batch * max_keep))
    return evict::invalid("keep and new_lens must not overlap seq_lens");
  if (batch > 1 && mass_stride < max_tokens) return evict::invalid("mass_stride is below max_tokens");
  cudaError_t e;
  const int sms = evict::device_sms(&e);
  if (e == cudaSuccess) e = evict::allow_select_smem();
  if (e != cudaSuccess) return evict::status_of(e);
  evict::SelectParams p;
  p.mass = mass;
  p.mass_stride = mass_stride;
  p.seq_lens = seq_lens;
  p.keep = keep;
  p.new_lens = new_lens;
  p.dev_status = dev_status;
  p.max_tokens = max_tokens;
  p.budget = max_keep;
  p.sink = sink;
  p.recent = recent;
  p.blocks = evict::cluster_for((max_tokens + 8191) / 8192, batch, sms);
  if ((int64_t)batch * p.blocks > INT32_MAX) return evict::invalid("batch too large");
  return evict::status_of(evict::launch(evict::select_kernel, (int64_t)batch * p.blocks, evict::kSelThreads, sizeof(evict::SelectSmem),
                                        p.blocks, (cudaStream_t)stream, p));
}

mla_status_t mla_cache_compact(void *cache, int64_t num_layers, int64_t num_blocks, int32_t block_size, const int32_t *block_table,
                               int32_t max_blocks_per_seq, int32_t batch, const int32_t *keep, int32_t max_keep,
                               const int32_t *seq_lens, const int32_t *new_lens, float *mass, int64_t mass_stride,
                               int32_t max_tokens, int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_cache_compact");
  return evict::run_compact(evict::compact_params(cache, block_size, block_table, max_blocks_per_seq, batch, keep, max_keep, seq_lens,
                                                  new_lens, mass, mass_stride, max_tokens, dev_status),
                            num_blocks, kRow * 2, num_layers, stream);
}

mla_status_t mla_cache_compact_fp8(void *cache8, int64_t num_layers, int64_t num_blocks, int32_t block_size,
                                   const int32_t *block_table, int32_t max_blocks_per_seq, int32_t batch, const int32_t *keep,
                                   int32_t max_keep, const int32_t *seq_lens, const int32_t *new_lens, float *mass,
                                   int64_t mass_stride, int32_t max_tokens, int32_t *dev_status, void *stream) {
  TraceRange trace_range("mla_cache_compact_fp8");
  return evict::run_compact(evict::compact_params(cache8, block_size, block_table, max_blocks_per_seq, batch, keep, max_keep, seq_lens,
                                                  new_lens, mass, mass_stride, max_tokens, dev_status),
                            num_blocks, kRow, num_layers, stream);
}

}  // extern "C"
