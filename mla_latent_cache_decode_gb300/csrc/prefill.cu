// mla_prefill kernel: attention of prompt tokens over expanded keys and values.
// Request b owns query rows [q_offsets[b], q_offsets[b+1]) and key rows
// [kv_offsets[b], kv_offsets[b+1]); with i, j counted inside the request,
//   s_ij = softmax_scale * (q_nope_i . k_nope_j + q_pe_i . k_pe_j)
//   j visible to i: j < nk, and when causal also j <= nk - nq + i
//   out_i = sum_j softmax(s_i)_j v_j,   lse_i = log sum_j exp(s_ij)
// A row that sees no key gets out = 0 and lse = -inf, one that sees keys but has
// no score above -inf NaN in both.
//
// Work.  An item is up to 256 query rows of one request and head: two tiles (A,
// B) of 128 rows that share every key and value tile of 128 rows.  Per key tile
// and query tile the tensor cores run S = Q K^T (12 MMAs of 128 x 128 x 16) and
// O += P V (8 of them): 1,280 cycles of their dense rate, against which the
// softmax of the other tile runs.  A request's last 128 rows or fewer would
// leave one of the tiles idle: there the two tiles are two heads, or the odd and
// the even key tiles of one (see Mode).  Items come in the order of requests
// (longest context first), groups of heads whose keys and values fit L2
// together, and tiles, a request's last (the longest when causal) first, so that
// the SMs that run at one time read few heads' keys and values, mostly from L2.
// The grid has a block an item; running blocks claim those of blocks that have
// not started.  With a workspace and fewer items than half the SMs, an item's
// keys are cut into parts, a block each, and join_kernel adds them up.
//
// Memory.  Shared: Q of both tiles (96 KB), keys in a ring of four 64-dim
// chunks of 16 KB (a key tile has three; each is handed back as soon as both
// tiles' MMAs on it are issued and done), values in two stages of 32 KB.
// Tensor memory: S of A and B (128 columns each; P overwrites its S as bf16),
// O of A and B (128 columns each).
//
// Warp roles: warps 0-3 softmax and epilogue of tile A, warps 4-7 of tile B
// (one thread per row; O is rescaled only when the running maximum grows by
// more than 2^8), warp 8 issues all MMAs in the order PV_A(j-1) S_A(j)
// PV_B(j-1) S_B(j), across items too, warp 9 issues the TMA loads, warp 10
// claims the items, warp 11 checks the offsets.  Every MMA is issued by one
// thread, so S_A(j) complete means PV_A(j-1) complete: O may be rescaled then
// without a further wait.  The weights are rounded to bf16 (the MMA's type, half
// a step 2^-8 each, independent from key to key); their sum, the maxima and O
// are fp32.
//
// What bounds it.  8,192 causal tokens of 128 heads, 1,736-1,796 us: 1.53-1.58
// PFLOP/s, 80-83% of the measured bf16 rate; every key visible 1.72-1.85 PFLOP/s.
// The tensor cores are busy 72% of the cycles of a 4,096-token prompt; the rest
// is the fill and the drain of each item (a claim, Q, the first S without a
// softmax beside it, O's way out) and the GPU's power limit.  Short prompts are
// bound by that latency: 4 prompts of 1 to 200 tokens 18 us, of which 6 are
// bytes (18.0 in a captured graph too: the GPU's time, not the call's); 9 queries
// on 18,097 keys of 16 heads 39.1 us (38.6 in a graph), 3.9 TB/s.
//
// What its parts gave, us (8,192 causal tokens of 128 heads; 3,992 queries of 16
// heads in four prompts, every key visible): two tiles an item, blocks by number 3,421 / 166; claimed items, the
// register split, packed fp32 arithmetic 1,896 / 84; odd and even key tiles,
// longest context first 1,799 / 77; pairs of heads, the claim near an item's end
// 1,771 / 69; 96 score registers a row instead of 128 and one pass over O 1,760 /
// 66.  Slower were: O by way of shared memory and TMA stores, a warpgroup of its
// own for the epilogue, MMAs issued from a loop or by the whole warp in step.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "ragged.cuh"
#include "sm100_issue.cuh"
#include "tmap.h"
#include "trace.h"

namespace mla {
void set_error_detail(const char *msg);

namespace prefill {
using namespace sm100;

constexpr int kNope = 128, kRope = MLA_ROPE_DIM, kV = 128;
constexpr int kTile = 128;                // query rows and key rows of a tile
constexpr int kChunk = kTile * 128;       // 64 dims of 128 rows, 128-byte swizzle: 16 KB
constexpr int kQChunks = 3, kVChunks = 2; // 64-dim chunks of a query (key) and of a value tile
constexpr int kKSlots = 4, kVSlots = 2;
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);  // the last warp completes a warpgroup
// Registers a thread: 384 x 168 at launch; the softmax warpgroups, which hold
// a row of S, take over what the third one gives up.
constexpr int kSoftmaxRegs = 192, kOtherRegs = 120;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register split");
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;  // tile t at + 128 t
// The longest legal wait is for another role's whole item: 2^26 keys, at half
// a million tiles of 1.3 us, 0.7 s.
constexpr int64_t kMaxKv = 1 << 26;
constexpr uint64_t kWaitNs = 3000000000ull;
constexpr uint64_t kDrainNs = 10000000ull;
constexpr float kRescale = 8.0f;  // log2
constexpr int32_t kGroupKeys = (48 << 20) / (2 * (kNope + kV));  // key rows of all heads walked together: 48 MB of 129 MB of L2
constexpr int kAskTiles = 4;               // key tiles ahead of an item's last load
constexpr int kMinPart = 4;                // key tiles of a part, at least

struct Strided {
  const __nv_bfloat16 *p;
  int64_t token, head;  // elements
};

struct Maps {
  CUtensorMap q_nope, q_pe, k_nope, k_pe, v;
};

struct Params {
  const int32_t *q_offsets, *kv_offsets;
  int32_t batch, heads, total_q, total_kv, causal, two_heads;
  float scale_log2;
  __nv_bfloat16 *out;
  float *lse;
  float *partial, *partial_lse;  // split form: [blocks][256][128], [blocks][256]; else null
  int4 *parts;                   // split form: two words a block, see join_kernel
  int32_t *dev_status;
};

// One item: rows [q0, q0 + rows) of head h over key tiles [kt, kt + .) of key
// rows [k0, k0 + nk).  Row r of the item sees keys [0, min(nk, see + r)).
// Query tile t runs n[t] key tiles.
enum Mode : int32_t {
  // More than 128 rows: query tile t holds rows 128 t ..; both run the same key
  // tiles (n[0] <= n[1]).
  kTwoTiles,
  // Up to 128 rows: both query tiles hold them, tile t runs key tiles kt + t,
  // kt + t + 2, ...: two chains of softmax and MMA instead of one, joined in
  // the epilogue.
  kOddEven,
  // Up to 128 rows, with items enough: query tile t holds head h + t, each with
  // its own keys and values.
  kTwoHeads,
};
struct Work {
  int32_t h, q0, rows, k0, nk, see, kt, n[2], mode;
  int32_t part, parts, slot, slot_step;  // parts > 1: a part of the keys, joined later
  // key tiles loaded: of the only head, or of both in turn
  __device__ __forceinline__ int32_t loads() const { return mode == kTwoTiles ? n[1] : n[0] + n[1]; }
};

struct __align__(1024) Smem {
  uint8_t q[2][kQChunks][kChunk];
  uint8_t k[kKSlots][kChunk];
  uint8_t v[kVSlots][kVChunks][kChunk];
  uint64_t q_full[2], q_empty[2], k_full[kKSlots], k_empty[kKSlots], v_full[kVSlots], v_empty[kVSlots];
  uint64_t s_full[2], p_full[2], o_full[2];
  // an odd-even item: tile 1's maxima and sums, then both tiles' factors
  float2 join[kTile];
  uint64_t join_sums, join_factors, join_end;
  uint64_t work_full[2], work_empty[2];
  uint64_t fin, roles_done, claim_full, near_end;
  uint4 claim;  // the answer of cluster launch control
  Work work[2];  // rows = 0: no more items
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory of one SM");

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

__device__ __forceinline__ void set_abort(Smem &s, int32_t *dev_status) {
  s.abort = 1;
  report(dev_status, MLA_ERR_DEVICE_TIMEOUT);
}

// A wait by one thread; on giving up the other roles are told.
__device__ __forceinline__ bool wait_or_abort(Smem &s, const Params &p, uint64_t &bar, uint32_t parity) {
  if (mbar_wait(smem_u32(&bar), parity, &s.abort, kWaitNs)) return true;
  if (!*(volatile int *)&s.abort) set_abort(s, p.dev_status);
  return false;
}

// The same by every lane of a warp, which then agrees.
__device__ __forceinline__ bool warp_wait(Smem &s, const Params &p, uint64_t &bar, uint32_t parity) {
  const bool ok = mbar_wait(smem_u32(&bar), parity, &s.abort, kWaitNs);
  if (__all_sync(0xffffffffu, ok)) return true;
  if ((threadIdx.x & 31) == 0 && !*(volatile int *)&s.abort) set_abort(s, p.dev_status);
  return false;
}

// ---------------------------------------------------------------- items

__device__ __forceinline__ int32_t rows_of(const int32_t *o, int32_t b, int32_t total) {
  return max(ragged::cut(o[b + 1], total) - ragged::cut(o[b], total), 0);
}

// A lane's request.
struct Request {
  int32_t q0, nq, k0, nk, tiles;  // tiles of 256 queries
};

__device__ __forceinline__ Request request(const Params &p, int32_t b) {
  Request r = {};
  if (b >= p.batch) return r;
  r.q0 = ragged::cut(p.q_offsets[b], p.total_q);
  r.nq = rows_of(p.q_offsets, b, p.total_q);
  r.k0 = ragged::cut(p.kv_offsets[b], p.total_kv);
  r.nk = rows_of(p.kv_offsets, b, p.total_kv);
  r.tiles = (r.nq + 2 * kTile - 1) / (2 * kTile);
  return r;
}

__device__ __forceinline__ Request shuffle(const Request &r, int src) {
  Request o;
  o.q0 = __shfl_sync(0xffffffffu, r.q0, src);
  o.nq = __shfl_sync(0xffffffffu, r.nq, src);
  o.k0 = __shfl_sync(0xffffffffu, r.k0, src);
  o.nk = __shfl_sync(0xffffffffu, r.nk, src);
  o.tiles = __shfl_sync(0xffffffffu, r.tiles, src);
  return o;
}

// Up to 32 requests in the order of their contexts, longest first, so that
// the longest items start first and short ones fill the end.
__device__ __forceinline__ Request sorted(const Request &r, int32_t batch, int lane) {
  if (batch <= 1) return r;
  int rank = 0, src = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int32_t nk = __shfl_sync(0xffffffffu, r.nk, i);
    rank += nk > r.nk || (nk == r.nk && i < lane);
  }
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (__shfl_sync(0xffffffffu, rank, i) == lane) src = i;
  return shuffle(r, src);
}

template <typename T>
__device__ __forceinline__ T prefix(T x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Key tiles that rows [first, first + rows) of a request run over.
__device__ __forceinline__ int32_t key_tiles(const Params &p, const Request &r, int32_t first, int32_t rows) {
  const int32_t keys = p.causal ? min(r.nk, r.nk - r.nq + first + rows) : r.nk;
  return rows > 0 && keys > 0 ? (keys + kTile - 1) / kTile : 0;
}

// Tile `tile` (from the request's start) of head h, key tiles
// [n part / parts, n (part + 1) / parts) of its n; `two_heads`: up to 128 rows
// are taken together with the next head's.
__device__ __forceinline__ Work make_work(const Params &p, const Request &r, int32_t tile, int32_t h, int32_t part,
                                          int32_t parts, bool two_heads) {
  Work w = {};
  const int32_t first = tile * 2 * kTile;
  w.h = h;
  w.q0 = r.q0 + first;
  w.rows = min(2 * kTile, r.nq - first);
  w.k0 = r.k0;
  w.nk = r.nk;
  w.see = p.causal ? r.nk - r.nq + first + 1 : r.nk;
  w.part = part;
  w.parts = parts;
  const int32_t n = key_tiles(p, r, first, w.rows);
  int32_t end = n;
  if (parts > 1) {
    w.kt = (int32_t)((int64_t)n * part / parts);
    end = (int32_t)((int64_t)n * (part + 1) / parts);
  }
  if (w.rows <= kTile && two_heads) {
    w.mode = kTwoHeads;
    w.n[0] = w.n[1] = end - w.kt;
  } else if (w.rows <= kTile) {
    w.mode = kOddEven;
    w.n[0] = (end - w.kt + 1) / 2;
    w.n[1] = (end - w.kt) / 2;
  } else {
    w.mode = kTwoTiles;
    w.n[0] = max(min(key_tiles(p, r, first, kTile), end) - w.kt, 0);
    w.n[1] = end - w.kt;
  }
  return w;
}

// A request's last tile, when it has up to 128 rows and pairs of heads share
// an item.
__device__ __forceinline__ int32_t thin_tile(const Params &p, const Request &r) {
  return p.two_heads && r.tiles > 0 && r.nq - (r.tiles - 1) * 2 * kTile <= kTile ? 1 : 0;
}

// Item `at` in the order: requests (up to 32: longest context first), groups of
// heads whose keys and values fit L2 together, tiles from the request's last
// (the longest when causal) to its first, heads of the group.  By one warp;
// rows = 0 behind the last.  A walk over many requests resumes where the last
// one ended: a block's items come in rising order.
struct Walk {
  int32_t b0, before;  // first of 32 requests, and the items of those before
};
__device__ __forceinline__ Work find_work(const Params &p, const Request &few, Walk &walk, int32_t at, int lane) {
  if (at < walk.before) walk = Walk{0, 0};
  int32_t &before = walk.before;
  for (int32_t &b0 = walk.b0; b0 < p.batch; b0 += 32) {
    const Request mine = p.batch <= 32 ? few : request(p, b0 + lane);
    const int32_t thin = thin_tile(p, mine);
    const int32_t items = (mine.tiles - thin) * p.heads + thin * ((p.heads + 1) / 2);
    const int32_t upto = before + prefix(items, lane);
    const uint32_t hit = __ballot_sync(0xffffffffu, at >= upto - items && at < upto);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const Request r = shuffle(mine, src);
      int32_t i = at - __shfl_sync(0xffffffffu, upto - items, src);
      const int32_t rt = thin_tile(p, r);
      // an even number of heads, or all
      const int32_t group = min(p.heads, max(2, kGroupKeys / max(r.nk, 1) & ~1));
      const int32_t of_group = (r.tiles - rt) * group + rt * ((group + 1) / 2);
      const int32_t first = i / of_group * group;
      const int32_t heads = min(group, p.heads - first);
      i -= i / of_group * of_group;
      if (rt && i < (heads + 1) / 2) {
        const int32_t h = first + 2 * i;
        return make_work(p, r, r.tiles - 1, h, 0, 1, h + 1 < p.heads);
      }
      i -= rt * ((heads + 1) / 2);
      return make_work(p, r, r.tiles - 1 - rt - i / heads, first + i % heads, 0, 1, false);
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
  return Work{};
}

// Split form: few items on long contexts.  Every item is cut into parts of at
// most `most` key tiles, such that the parts are no more than the blocks; part
// `at` leaves its output in slot `at` of the workspace.  By one warp; rows = 0
// behind the last.  (At most half as many items as blocks, so everything here
// counts in 32 bits and in few rounds of 32 requests.)
__device__ __forceinline__ Work find_part(const Params &p, int32_t at, int32_t blocks, int lane) {
  int32_t items = 0, total = 0;
  Request mine = request(p, lane);
  auto tiles_of = [&](const Request &r, int32_t t) {
    return key_tiles(p, r, t * 2 * kTile, min(2 * kTile, r.nq - t * 2 * kTile));
  };
  for (int32_t b0 = 0; b0 < p.batch; b0 += 32) {
    const Request r = p.batch <= 32 ? mine : request(p, b0 + lane);
    items += r.tiles;
    for (int32_t t = 0; t < r.tiles; ++t) total += tiles_of(r, t);
  }
  items = __reduce_add_sync(0xffffffffu, items) * p.heads;
  total = __reduce_add_sync(0xffffffffu, total) * p.heads;
  // sum of ceil(n / most) <= total / most + items <= blocks
  const int32_t spare = max(1, blocks - items), most = max(kMinPart, (total + spare - 1) / spare);
  int32_t before = 0;
  for (int32_t b0 = 0; b0 < p.batch; b0 += 32) {
    if (p.batch > 32) mine = request(p, b0 + lane);
    int32_t parts = 0;
    for (int32_t t = 0; t < mine.tiles; ++t) parts += max(1, (tiles_of(mine, t) + most - 1) / most);
    parts *= p.heads;
    const int32_t upto = before + prefix(parts, lane);
    const uint32_t hit = __ballot_sync(0xffffffffu, at >= upto - parts && at < upto);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const Request r = shuffle(mine, src);
      int32_t first = __shfl_sync(0xffffffffu, upto - parts, src);
      for (int32_t t = 0; t < r.tiles; ++t) {
        const int32_t cut = max(1, (tiles_of(r, t) + most - 1) / most);
        if (at < first + cut * p.heads) {
          const int32_t i = at - first;
          Work w = make_work(p, r, t, i % p.heads, i / p.heads, cut, false);
          w.slot = at;
          w.slot_step = p.heads;
          return w;
        }
        first += cut * p.heads;
      }
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
  return Work{};
}

// A role's view of the items: next() waits for one and copies it, done()
// hands its slot back.
struct Items {
  uint32_t i = 0;
  __device__ __forceinline__ bool ready(Smem &s, const Params &p) {
    return wait_or_abort(s, p, s.work_full[i & 1], (i >> 1) & 1);
  }
  __device__ __forceinline__ Work get(Smem &s) const { return s.work[i & 1]; }
  __device__ __forceinline__ void done(Smem &s) {
    mbar_arrive(smem_u32(&s.work_empty[i & 1]));
    ++i;
  }
};

// ---------------------------------------------------------------- softmax

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two fp32 in one 64-bit register pair: one instruction for two operations.
__device__ __forceinline__ void fma2(float &x, float &y, float a, float b) {  // x, y = x * a + b, y * a + b
  asm("{\n .reg .b64 v, m, n;\n mov.b64 v, {%0, %1};\n mov.b64 m, {%2, %2};\n mov.b64 n, {%3, %3};\n"
      " fma.rn.f32x2 v, v, m, n;\n mov.b64 {%0, %1}, v;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float &x, float &y, float a, float b) {  // x, y += a, b
  asm("{\n .reg .b64 v, m;\n mov.b64 v, {%0, %1};\n mov.b64 m, {%2, %3};\n"
      " add.rn.f32x2 v, v, m;\n mov.b64 {%0, %1}, v;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// Columns c0 .. c0 + 31 of a row of S; keys from `lim` on are not seen.
__device__ __forceinline__ void mask32(float *x, int c0, int lim) {
#pragma unroll
  for (int k = 0; k < 32; ++k) x[k] = c0 + k < lim ? x[k] : -INFINITY;
}

__device__ __forceinline__ void max32(const float *x, float (&mx)[4]) {
#pragma unroll
  for (int k = 0; k < 32; k += 2) mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], x[k], x[k + 1]);
}

// 32 weights 2^(x scale_log2 + nm) as bf16 into 16 columns of tensor memory,
// their sum in fp32 into ps.
__device__ __forceinline__ void weights32(const float *x, float scale_log2, float nm, float (&ps)[4], uint32_t p_addr) {
  uint32_t pk[16];
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    float a = x[k], b = x[k + 1];
    fma2(a, b, scale_log2, nm);
    a = ex2_approx(a);
    b = ex2_approx(b);
    add2(ps[k & 2], ps[(k & 2) + 1], a, b);
    pk[k / 2] = pack2(a, b);
  }
  tmem_st16(p_addr, pk);
}

// One key tile of one row: S from tensor memory, its maximum and the sum of the
// weights, and the weights back over S as bf16.  The row sees `lim` keys of the
// tile (may be <= 0 or >= 128), the warp's rows at least `lo` and at most `hi`.
//   kLong: straight-line code on registers.  The last chunk of S, which the
//     weights do not overwrite, is read twice, so that 96 values live at a time
//     leave the registers for the rest of the loop.
//   else: loops over the four 32-key chunks, each read again for its weights, in
//     a quarter of the code; chunks that no row sees are left out of the maximum,
//     those behind the request's last key (`keys` are there) altogether.
// The instruction cache decides: an item of few key tiles pays for its code, not
// for its arithmetic (see use_long).
template <bool kLong>
__device__ __forceinline__ void softmax_tile(uint32_t s_addr, uint32_t o_addr, float scale_log2, int keys, int lim, int lo,
                                             int hi, bool first, float &m, float &l) {
  float x[96];
  uint32_t *xr = reinterpret_cast<uint32_t *>(x);
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  if (kLong) {
    tmem_ld32(s_addr + 96, xr + 64);
    tmem_ld32(s_addr, xr);
    tmem_ld32(s_addr + 32, xr + 32);
    tmem_wait_ld();
    tmem_loaded32(xr);
    tmem_loaded32(xr + 32);
    tmem_loaded32(xr + 64);
    if (lo < kTile) {
      mask32(x + 64, 96, lim);
      mask32(x, 0, lim);
      mask32(x + 32, 32, lim);
    }
    max32(x + 64, mx);
    tmem_ld32(s_addr + 64, xr + 64);
    max32(x, mx);
    max32(x + 32, mx);
    tmem_wait_ld();
    tmem_loaded32(xr + 64);
    if (lo < kTile) mask32(x + 64, 64, lim);
    max32(x + 64, mx);
  } else {
#pragma unroll 1
    for (int c = 0; c < min(hi, kTile); c += 32) {
      tmem_ld32(s_addr + c, xr);
      tmem_wait_ld();
      tmem_loaded32(xr);
      if (lo < c + 32) mask32(x, 0, lim - c);
      max32(x, mx);
    }
  }
  const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale_log2;
  const bool grow = top > m + kRescale || (m == -INFINITY && top > -INFINITY);
  if (__any_sync(0xffffffffu, grow)) {
    const float alpha = grow ? ex2_approx(m - top) : 1.f;  // 0 when nothing was seen before
    if (grow) m = top;
    l *= alpha;
    if (!first) {
#pragma unroll 1
      for (int c = 0; c < kV; c += 16) {
        uint32_t o[16];
        tmem_ld16(o_addr + c, o);
        tmem_wait_ld();
        tmem_loaded16(o);
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
        tmem_st16(o_addr + c, o);
      }
    }
  }
  const float nm = m == -INFINITY ? 0.f : -m;  // a row that has seen nothing: every weight is 0
  float ps[4] = {0.f, 0.f, 0.f, 0.f};
  if (kLong) {
    weights32(x, scale_log2, nm, ps, s_addr);
    tmem_ld32(s_addr + 96, xr);
    weights32(x + 32, scale_log2, nm, ps, s_addr + 16);
    weights32(x + 64, scale_log2, nm, ps, s_addr + 32);
    tmem_wait_ld();
    tmem_loaded32(xr);
    if (lo < kTile) mask32(x, 96, lim);
    weights32(x, scale_log2, nm, ps, s_addr + 48);
  } else {
#pragma unroll 1
    for (int c = 0; c < min(keys, kTile); c += 32) {
      tmem_ld32(s_addr + c, xr);
      tmem_wait_ld();
      tmem_loaded32(xr);
      if (lo < c + 32) mask32(x, 0, lim - c);
      weights32(x, scale_log2, nm, ps, s_addr + c / 2);
    }
  }
  l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
}

// 16 outputs of a row, 16 bytes a store.  No 32-byte stores: in a function that both
// kernels below call, not inlined, they wrote only their first 4 or 8 bytes in one of
// the two, written as PTX or as a 32-byte vector type (nvcc 13.0).  They took 65.2 us
// where these take 66.9-67.7 (3,992 queries of 16 heads, every key visible), 38.8 / 39.2
// (9 queries on 18,097 keys), the same elsewhere.
__device__ __forceinline__ void store16(__nv_bfloat16 *dst, const float *x) {
  uint32_t u[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = pack2(x[2 * k], x[2 * k + 1]);
  reinterpret_cast<uint4 *>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
  reinterpret_cast<uint4 *>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
}

// A tcgen05 instruction is the whole warp's: every lane comes to it, and together.
// Lanes without a row (the last of a tile) leave out the stores, not the loop, and
// where lanes part (a store, a loop of unequal length) a __syncwarp joins them again
// ahead of the next one.

// A whole row of output: O / l.  Not inlined: the softmax loop around it needs
// the registers.
__device__ __noinline__ void store_out(uint32_t o, float inv, bool real, __nv_bfloat16 *out) {
#pragma unroll 1
  for (int c = 0; c < kV; c += 32) {
    float x[32];
    uint32_t *xr = reinterpret_cast<uint32_t *>(x);
    __syncwarp();
    tmem_ld32(o + c, xr);
    tmem_wait_ld();
    tmem_loaded32(xr);
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] *= inv;
    if (real) {
      store16(out + c, x);
      store16(out + c + 16, x + 16);
    }
  }
}

// Columns [c0, c1) of a row's output: a * O_a (+ b * O_b with `two`), to `out`
// as bf16 or, for a part of the keys, to `partial` as fp32.  `any`: O holds
// something.  Not inlined, like store_out.
__device__ __noinline__ void store_row(uint32_t oa, float a, uint32_t ob, float b, bool two, bool any, int c0, int c1,
                                       bool real, __nv_bfloat16 *out, float *partial) {
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    float x[32];
    uint32_t *xr = reinterpret_cast<uint32_t *>(x);
    __syncwarp();
    if (any) {
      tmem_ld32(oa + c, xr);
      tmem_wait_ld();
      tmem_loaded32(xr);
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = a != 0.f ? x[k] * a : 0.f;
    if (two) {
      uint32_t y[32];
      tmem_ld32(ob + c, y);
      tmem_wait_ld();
      tmem_loaded32(y);
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] += b != 0.f ? __uint_as_float(y[k]) * b : 0.f;
    }
    if (real && partial) {
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        *reinterpret_cast<float4 *>(partial + c + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
    } else if (real) {
      store16(out + c, x);
      store16(out + c + 16, x + 16);
    }
  }
}

template <bool kLong>
__device__ __forceinline__ void softmax_role(Smem &s, const Params &p, int warp, int lane, uint32_t tmem) {
  const int t = warp >> 2, q4 = warp & 3;
  const int row = q4 * 32 + lane;  // of the tile: TMEM lane
  const uint32_t lanes = tmem + ((uint32_t)(q4 * 32) << 16);
  const uint32_t s_addr = lanes + kColS + 128 * t;
  Items items;
  // key tiles of this query tile, key tiles loaded, outputs of either query tile, odd-even items
  uint32_t g = 0, vg = 0, outs0 = 0, outs1 = 0, joins = 0;
  while (true) {
    if (!warp_wait(s, p, s.work_full[items.i & 1], (items.i >> 1) & 1)) return;
    // read from shared memory where it is needed: the registers are S's
    const Work &w = s.work[items.i & 1];
    if (w.rows == 0) return;
    const int n = t ? w.n[1] : w.n[0];
    const int at = w.mode == kTwoTiles ? t * kTile + row : row;  // row of the item
    float m = -INFINITY, l = 0.f;
    {
      // of this query tile's first key tile: the keys the row sees from there
      // on, the keys there are, and its number among all tiles loaded
      const int key = (w.kt + (w.mode == kOddEven ? t : 0)) * kTile;
      int lim = min(w.nk, p.causal ? w.see + at : w.nk) - key;
      int lo = __reduce_min_sync(0xffffffffu, lim), hi = __reduce_max_sync(0xffffffffu, lim);
      const int step = w.mode == kOddEven ? 2 * kTile : kTile;
      for (int j = 0; j < n; ++j, ++g, lim -= step, lo -= step, hi -= step) {
        if (!warp_wait(s, p, s.s_full[t], g & 1)) return;
        tc_fence_after();
        softmax_tile<kLong>(s_addr, s_addr + (kColO - kColS), p.scale_log2, w.nk - key - j * step, lim, lo, hi, j == 0, m, l);
        if (j == n - 1) {
          // A last key tile's P V reads value rows up to a multiple of 16: those
          // behind the request's last key hold anything (0 * NaN = NaN), so they
          // are zeroed first, by both query tiles alike.
          const int valid = w.nk - key - j * step;
          if (valid < kTile && (valid & 15)) {
            const uint32_t vi = vg + (w.mode == kTwoTiles ? j : 2 * j + t);
            if (!warp_wait(s, p, s.v_full[vi % kVSlots], (vi / kVSlots) & 1)) return;
            const int pad = 16 - (valid & 15);
            for (int k = q4 * 32 + lane; k < pad * 16; k += 128) {
              const int r = valid + (k >> 4), c = (k >> 3) & 1;
              *reinterpret_cast<uint4 *>(&s.v[vi % kVSlots][c][r * 128 + (k & 7) * 16]) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_shared();
            __syncwarp();
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&s.p_full[t]));
      }
    }
    vg += w.loads();
    // ---- epilogue: O / l.  A row that sees no key has l = 0, and so has one whose
    // scores are all -inf (a key or query that is not finite): it becomes NaN, like
    // those with a score of NaN or +inf.  (A part of the keys leaves that to the join.)
    const bool real = at < w.rows;
    const bool nan = w.parts == 1 && (p.causal ? w.see + at : w.nk) > 0;  // if l = 0
    const int64_t out_row = ((int64_t)w.q0 + at) * p.heads + w.h + (w.mode == kTwoHeads ? t : 0);
    __nv_bfloat16 *out = p.out + out_row * kV;
    float *partial = nullptr, *lse = p.lse ? p.lse + out_row : nullptr;
    if (w.parts > 1) {
      partial = p.partial + ((int64_t)w.slot * 2 * kTile + at) * kV;
      lse = p.partial_lse + (int64_t)w.slot * 2 * kTile + at;
    }
    if (w.mode != kOddEven) {
      if (n > 0) {
        if (!warp_wait(s, p, s.o_full[t], (t ? outs1 : outs0) & 1)) return;
        tc_fence_after();
      }
      if (n > 0 && !partial)
        store_out(s_addr + (kColO - kColS), l != 0.f ? 1.f / l : nan ? NAN : 0.f, real, out);
      else
        store_row(s_addr + (kColO - kColS), l != 0.f ? 1.f / l : 0.f, 0, 0.f, false, n > 0, 0, kV, real, out, partial);
      if (real && lse) *lse = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : nan ? NAN : -INFINITY;
      tc_fence_before();
    } else {
      // tile 1 tells its maxima and sums, tile 0 answers with the factors of
      // both O, and tile t writes dims 64 t .. 64 t + 63 of the rows
      float2 f;
      if (t == 1) {
        s.join[row] = make_float2(m, l);
        mbar_arrive(smem_u32(&s.join_sums));
        if (!warp_wait(s, p, s.join_factors, joins & 1)) return;
        f = s.join[row];
      } else {
        if (!warp_wait(s, p, s.join_sums, joins & 1)) return;
        const float2 other = s.join[row];
        const float top = fmaxf(m, other.x);
        f.x = l != 0.f ? ex2_approx(m - top) : 0.f;
        f.y = other.y != 0.f ? ex2_approx(other.x - top) : 0.f;
        const float sum = f.x * l + f.y * other.y, inv = sum != 0.f ? 1.f / sum : nan ? NAN : 0.f;
        f.x *= inv;
        f.y *= inv;
        s.join[row] = f;
        mbar_arrive(smem_u32(&s.join_factors));
        if (real && lse) *lse = sum != 0.f ? (top + log2f(sum)) * 0.69314718055994531f : nan ? NAN : -INFINITY;
      }
      if ((w.n[0] > 0 && !warp_wait(s, p, s.o_full[0], outs0 & 1)) ||
          (w.n[1] > 0 && !warp_wait(s, p, s.o_full[1], outs1 & 1)))
        return;
      tc_fence_after();
      store_row(lanes + kColO, f.x, lanes + kColO + 128, f.y, w.n[1] > 0, w.n[0] > 0, 64 * t, 64 * t + 64, real, out,
                partial);
      tc_fence_before();
      // neither O nor the meeting place is reused before both have read it
      mbar_arrive(smem_u32(&s.join_end));
      if (!warp_wait(s, p, s.join_end, joins & 1)) return;
      ++joins;
    }
    outs0 += w.n[0] > 0;
    outs1 += w.n[1] > 0;
    __syncwarp();
    if (lane == 0) items.done(s); else ++items.i;
  }
}

// ---------------------------------------------------------------- MMA issuer

// P V of a query tile's latest key tile, issued once its softmax is done.
struct Pending {
  bool on, first, last, free_v;
  uint32_t v;  // key tile, among all loaded
  int ksteps;
};

// Kept small and free of run-time choices in the loops: the time between a
// softmax's end and the first MMA behind it is on every tile's path.
struct MmaRole {
  Smem &s;
  const Params &p;
  uint32_t tmem;
  uint32_t d_q, d_k, d_v;  // descriptors (low words) of q[0][0], k[0], v[0]
  Pending pend[2];
  uint32_t g[2], q_used[2];  // key tiles and items of each query tile
  uint32_t kv;               // key tiles of the items before

  template <int t>
  __device__ __forceinline__ bool run_pv() {
    Pending &a = pend[t];
    const uint32_t slot = a.v % kVSlots;
    if (!wait_or_abort(s, p, s.v_full[slot], (a.v / kVSlots) & 1) ||
        !wait_or_abort(s, p, s.p_full[t], (g[t] - 1) & 1))
      return false;
    tc_fence_after();
    constexpr uint32_t id = idesc_bf16_f32(kTile, kV, 1);
    const uint32_t dv = d_v + slot * (kVChunks * kChunk >> 4);
    const uint32_t d = tmem + kColO + 128 * t, pa = tmem + kColS + 128 * t;
    if (a.ksteps == kTile / 16) {
      mma_ts_low(d, pa, dv, id, a.first ? 0u : 1u);
#pragma unroll
      for (int k = 1; k < kTile / 16; ++k) mma_ts_low(d, pa + 8 * k, dv + 128 * k, id, 1u);
    } else {
#pragma unroll 1
      for (int k = 0; k < a.ksteps; ++k)
        mma_ts_low(d, pa + 8 * k, dv + 128 * k, id, (a.first && k == 0) ? 0u : 1u);
    }
    if (a.free_v) mma_commit(smem_u32(&s.v_empty[slot]));
    if (a.last) mma_commit(smem_u32(&s.o_full[t]));
    a.on = false;
    return true;
  }

  // S of query tile t (its Q in tile tq's place) and a key tile, of which `keys`
  // are the request's: as many columns, to a multiple of 16 (100 prompts of 3
  // queries on 40 keys 147.5 -> 144.6 us).
  template <int t, int tq, bool kFreeK>
  __device__ __forceinline__ bool run_s(uint32_t tile, int keys) {
    const uint32_t id = idesc_bf16_f32(kTile, min((keys + 15) & ~15, kTile), 0);
    const uint32_t d = tmem + kColS + 128 * t;
#pragma unroll
    for (int c = 0; c < kQChunks; ++c) {
      const uint32_t chunk = tile * kQChunks + c, slot = chunk % kKSlots;
      if (!wait_or_abort(s, p, s.k_full[slot], (chunk / kKSlots) & 1)) return false;
      tc_fence_after();
      const uint32_t a = d_q + (tq * kQChunks + c) * (kChunk >> 4), b = d_k + slot * (kChunk >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_ss_low(d, a + 2 * k, b + 2 * k, id, (c > 0 || k > 0) ? 1u : 0u);
      if (kFreeK) mma_commit(smem_u32(&s.k_empty[slot]));
    }
    mma_commit(smem_u32(&s.s_full[t]));
    ++g[t];
    return true;
  }

  template <int t, Mode kMode>
  __device__ __forceinline__ bool step(int j, int n, int loads, int tail_keys) {
    if (pend[t].on && !run_pv<t>()) return false;
    if (j >= n) return true;
    constexpr bool kOwnTiles = kMode != kTwoTiles;        // key tiles of its own
    constexpr int tq = kMode == kOddEven ? 0 : t;         // place of its Q
    if (j == 0 && tq == t && !wait_or_abort(s, p, s.q_full[t], q_used[t]++ & 1)) return false;
    const int jt = kOwnTiles ? 2 * j + t : j;             // among the item's loads
    const int keys = tail_keys - (kMode == kOddEven ? jt : j) * kTile;  // from this tile on
    if (!run_s<t, tq, kOwnTiles || t == 1>(kv + jt, keys)) return false;
    if (kMode == kOddEven ? jt == loads - 1 : j == n - 1) mma_commit(smem_u32(&s.q_empty[tq]));
    pend[t] = Pending{true, j == 0, j == n - 1, kOwnTiles || t == 1, kv + jt, keys >= kTile ? kTile / 16 : (keys + 15) >> 4};
    return true;
  }

  template <Mode kMode>
  __device__ __forceinline__ bool item(int n0, int n1, int loads, int tail_keys) {
    const int rounds = max(n0, n1);
#pragma unroll 1
    for (int j = 0; j < rounds; ++j)
      if (!step<0, kMode>(j, n0, loads, tail_keys) || !step<1, kMode>(j, n1, loads, tail_keys)) return false;
    kv += loads;
    return true;
  }

  __device__ __forceinline__ void run() {
    Items items;
    bool ok = true;
    while (ok && items.ready(s, p)) {
      const Work &w = s.work[items.i & 1];
      const int rows = w.rows, n0 = w.n[0], n1 = w.n[1], tail_keys = w.nk - w.kt * kTile;
      const int mode = w.mode, loads = w.loads();
      items.done(s);
      if (max(n0, n1) == 0) {  // no key to see, or no more items: what is pending has no S to wait behind
        ok = (!pend[0].on || run_pv<0>()) && (!pend[1].on || run_pv<1>());
        if (rows == 0) break;
      } else {
        ok = mode == kTwoTiles  ? item<kTwoTiles>(n0, n1, loads, tail_keys)
             : mode == kOddEven ? item<kOddEven>(n0, n1, loads, tail_keys)
                                : item<kTwoHeads>(n0, n1, loads, tail_keys);
      }
    }
    // every MMA issued is finished before the tensor memory is given back
    mma_commit(smem_u32(&s.fin));
    if (!mbar_wait(smem_u32(&s.fin), 0, nullptr, kWaitNs)) report(p.dev_status, MLA_ERR_DEVICE_TIMEOUT);
  }
};

__device__ __forceinline__ void mma_role(Smem &s, const Params &p, uint32_t tmem) {
  MmaRole r{s,
            p,
            tmem,
            desc_low(s.q[0][0], 16),
            desc_low(s.k[0], 16),
            desc_low(s.v[0][0], kChunk),
            {},
            {0, 0},
            {0, 0},
            0};
  r.run();
}

// ---------------------------------------------------------------- TMA producer

__device__ __forceinline__ void load_role(Smem &s, const Params &p, const Maps &maps) {
  Items items;
  uint32_t nq[2] = {0, 0}, nk = 0, nv = 0;  // loads issued: query tiles, key chunks, value tiles
  const uint64_t hint = policy_evict_normal();
  bool ok = true;
  auto load_q = [&](const Work &w, int t) -> bool {
    if ((t ? w.n[1] : w.n[0]) == 0 || (t == 1 && w.mode == kOddEven)) return true;
    if (!wait_or_abort(s, p, s.q_empty[t], (nq[t] & 1) ^ 1)) return false;
    const uint32_t bar = smem_u32(&s.q_full[t]);
    mbar_arrive_expect_tx(bar, kQChunks * kChunk);
    const int32_t y = w.q0 + (w.mode == kTwoTiles ? t * kTile : 0), h = w.h + (w.mode == kTwoHeads ? t : 0);
    tma_load_3d_hint(smem_u32(s.q[t][0]), &maps.q_nope, 0, h, y, bar, hint);
    tma_load_3d_hint(smem_u32(s.q[t][1]), &maps.q_nope, 64, h, y, bar, hint);
    tma_load_3d_hint(smem_u32(s.q[t][2]), &maps.q_pe, 0, h, y, bar, hint);
    ++nq[t];
    return true;
  };
  // key rows from y on, of head h
  auto load_k = [&](int32_t h, int32_t y) -> bool {
    for (int c = 0; c < kQChunks; ++c, ++nk) {
      const uint32_t slot = nk % kKSlots;
      if (!wait_or_abort(s, p, s.k_empty[slot], ((nk / kKSlots) & 1) ^ 1)) return false;
      const uint32_t bar = smem_u32(&s.k_full[slot]);
      mbar_arrive_expect_tx(bar, kChunk);
      if (c < 2) tma_load_3d_hint(smem_u32(s.k[slot]), &maps.k_nope, 64 * c, h, y, bar, hint);
      else tma_load_3d_hint(smem_u32(s.k[slot]), &maps.k_pe, 0, 0, y, bar, hint);
    }
    return true;
  };
  auto load_v = [&](int32_t h, int32_t y) -> bool {
    const uint32_t slot = nv % kVSlots;
    if (!wait_or_abort(s, p, s.v_empty[slot], ((nv / kVSlots) & 1) ^ 1)) return false;
    const uint32_t bar = smem_u32(&s.v_full[slot]);
    mbar_arrive_expect_tx(bar, kVChunks * kChunk);
    for (int c = 0; c < kVChunks; ++c)
      tma_load_3d_hint(smem_u32(s.v[slot][c]), &maps.v, 64 * c, h, y, bar, hint);
    ++nv;
    return true;
  };
  while (ok && items.ready(s, p)) {
    const Work w = items.get(s);
    items.done(s);
    if (w.rows == 0) break;
    const int loads = w.loads();
    const bool heads = w.mode == kTwoHeads;
    // Only now may the next item be claimed: a block that claims while its
    // item has long to run would keep it from those that run dry.
    const int ask = max(loads - kAskTiles, 0);
    if (loads == 0) mbar_arrive(smem_u32(&s.near_end));
    ok = load_q(w, 0);
    for (int j = 0; j < loads && ok; ++j) {
      if (j == ask) mbar_arrive(smem_u32(&s.near_end));
      const int32_t h = w.h + (heads ? j & 1 : 0), y = w.k0 + (w.kt + (heads ? j >> 1 : j)) * kTile;
      ok = load_k(h, y) && (j > 0 || load_q(w, 1)) && load_v(h, y);
    }
  }
  if (*(volatile int *)&s.abort) {  // no copy may still be landing when the shared memory is given up
    for (int t = 0; t < 2; ++t)
      if (nq[t]) (void)mbar_wait(smem_u32(&s.q_full[t]), (nq[t] - 1) & 1, nullptr, kDrainNs);
    for (uint32_t i = nk > kKSlots ? nk - kKSlots : 0; i < nk; ++i)
      (void)mbar_wait(smem_u32(&s.k_full[i % kKSlots]), (i / kKSlots) & 1, nullptr, kDrainNs);
    for (uint32_t i = nv > kVSlots ? nv - kVSlots : 0; i < nv; ++i)
      (void)mbar_wait(smem_u32(&s.v_full[i % kVSlots]), (i / kVSlots) & 1, nullptr, kDrainNs);
  }
}

// ---------------------------------------------------------------- scheduler

// The grid has a block for every item there may be (the host does not know
// the lengths).  A running block claims the items of blocks that have not
// started yet (cluster launch control): first come, first served, without a
// counter in memory.
struct Claims {
  uint32_t phase = 0;
  // By one warp: the next item's index, -1 when none is left (or on giving up).
  __device__ __forceinline__ int32_t next(Smem &s, const Params &p, int lane) {
    if (lane == 0) {
      fence_proxy_async_shared();  // the last answer has been read
      mbar_arrive_expect_tx(smem_u32(&s.claim_full), 16);
      asm volatile(
          "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
              smem_u32(&s.claim)),
          "r"(smem_u32(&s.claim_full))
          : "memory");
    }
    if (!warp_wait(s, p, s.claim_full, phase)) {
      // the answer must not still be landing when the shared memory is given up
      (void)mbar_wait(smem_u32(&s.claim_full), phase, nullptr, kDrainNs);
      return -1;
    }
    phase ^= 1;
    uint64_t a0, a1;
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a0), "=l"(a1) : "r"(smem_u32(&s.claim)) : "memory");
    uint32_t got, x;
    asm("{\n .reg .pred p;\n .reg .b128 a;\n mov.b128 a, {%2, %3};\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, a;\n}"
        : "=r"(got), "=r"(x)
        : "l"(a0), "l"(a1));
    __syncwarp();
    return got ? (int32_t)x : -1;
  }
};

__device__ __forceinline__ void schedule_role(Smem &s, const Params &p, int lane) {
  uint32_t i = 0;
  auto publish = [&](const Work &w) -> bool {
    if (!warp_wait(s, p, s.work_empty[i & 1], ((i >> 1) & 1) ^ 1)) return false;
    if (lane == 0) {
      s.work[i & 1] = w;
      mbar_arrive(smem_u32(&s.work_full[i & 1]));
    }
    ++i;
    return true;
  };
  if (p.partial) {  // one part a block
    const Work w = find_part(p, blockIdx.x, gridDim.x, lane);
    if (w.rows == 0 || publish(w)) (void)publish(Work{});
    if (lane == 0) {
      p.parts[2 * blockIdx.x] = make_int4(w.rows, w.parts, w.part, w.q0);
      p.parts[2 * blockIdx.x + 1] = make_int4(w.h, w.slot - w.part * w.slot_step, w.slot_step, w.see);
    }
    return;
  }
  Request few = {};
  if (p.batch <= 32) few = sorted(request(p, lane), p.batch, lane);
  Walk walk = {0, 0};
  Claims claims;
  for (int32_t at = blockIdx.x; at >= 0; at = claims.next(s, p, lane)) {
    const Work w = find_work(p, few, walk, at, lane);
    if (w.rows == 0) continue;  // a block more than there are items brings none
    if (!publish(w) || !warp_wait(s, p, s.near_end, (i - 1) & 1)) return;
  }
  (void)publish(Work{});
}

template <bool kLong>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem &s = *reinterpret_cast<Smem *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&s.q_full[t]), 1);
      mbar_init(smem_u32(&s.q_empty[t]), 1);
      mbar_init(smem_u32(&s.s_full[t]), 1);
      mbar_init(smem_u32(&s.p_full[t]), kTile);
      mbar_init(smem_u32(&s.o_full[t]), 1);
      mbar_init(smem_u32(&s.work_full[t]), 1);
      mbar_init(smem_u32(&s.work_empty[t]), kSoftmaxWarps + 2);
    }
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(smem_u32(&s.k_full[i]), 1);
      mbar_init(smem_u32(&s.k_empty[i]), 1);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(smem_u32(&s.v_full[i]), 1);
      mbar_init(smem_u32(&s.v_empty[i]), 1);
    }
    mbar_init(smem_u32(&s.join_sums), kTile);
    mbar_init(smem_u32(&s.join_factors), kTile);
    mbar_init(smem_u32(&s.join_end), 2 * kTile);
    mbar_init(smem_u32(&s.claim_full), 1);
    mbar_init(smem_u32(&s.near_end), 1);
    mbar_init(smem_u32(&s.fin), 1);
    mbar_init(smem_u32(&s.roles_done), kThreads / 32);
    s.abort = 0;
    fence_mbarrier_init_cluster();
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(smem_u32(&s.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 32 * (kSoftmaxWarps + 1)) {
    prefetch_tmap(&maps.q_nope);
    prefetch_tmap(&maps.q_pe);
    prefetch_tmap(&maps.k_nope);
    prefetch_tmap(&maps.k_pe);
    prefetch_tmap(&maps.v);
  }
  // Launched as a programmatic dependent: what is above may run while the
  // kernel before this one ends, what is below reads and writes memory.
  griddep_wait();
  griddep_launch_dependents();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<kLong>(s, p, warp, lane, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSoftmaxWarps) {
      if (elect_one_sync()) mma_role(s, p, tmem);
    } else if (warp == kSoftmaxWarps + 1) {
      if (elect_one_sync()) load_role(s, p, maps);
    } else if (warp == kSoftmaxWarps + 2) {
      schedule_role(s, p, lane);
    } else if (blockIdx.x == 0) {
      ragged::check_offsets(p.q_offsets, p.batch, p.total_q, lane, 32, p.dev_status);
      ragged::check_offsets(p.kv_offsets, p.batch, p.total_kv, lane, 32, p.dev_status);
    }
  }

  // the tensor memory is freed once every warp has reported the end of its role
  __syncwarp();
  tc_fence_before();
  if (lane == 0) mbar_arrive(smem_u32(&s.roles_done));
  if (warp == 0) {
    if (lane == 0 && !mbar_wait(smem_u32(&s.roles_done), 0, nullptr, kWaitNs))
      report(p.dev_status, MLA_ERR_DEVICE_TIMEOUT);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Split form: joins the parts of an item.  Block `at` takes every parts-th row
// of the item that part `at` belongs to, a warp per row:
//   out = sum_i e^(lse_i - top) O_i / sum_i e^(lse_i - top)
// The attention kernel's block `at` left what to do: {rows, parts, part, first
// row} and {head, first slot, slots from part to part, keys the first row sees}.
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 a = p.parts[2 * blockIdx.x], b = p.parts[2 * blockIdx.x + 1];
  const int rows = a.x, parts = a.y, part = a.z, q0 = a.w, head = b.x, first = b.y, step = b.z, see = b.w;
  // (offsets that overlap may ask for more parts than there are blocks)
  if (rows == 0 || parts == 1 || first + (parts - 1) * step >= (int)gridDim.x) return;
  for (int r = part + warp * parts; r < rows; r += kJoinThreads / 32 * parts) {
    // lane i holds part i's log-sum-exp (parts come in groups of 32)
    float top = -INFINITY;
    bool any = false;  // a part saw a key, or is NaN
    for (int i = lane; i < parts; i += 32) {
      const float x = p.partial_lse[(int64_t)(first + i * step) * 2 * kTile + r];
      top = fmaxf(top, x);
      any |= x != -INFINITY;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    if (__any_sync(0xffffffffu, any)) {
#pragma unroll 4
      for (int i = 0; i < parts; ++i) {
        const int64_t at = (int64_t)(first + i * step) * 2 * kTile + r;
        const float f = expf(p.partial_lse[at] - top);
        const float4 x = reinterpret_cast<const float4 *>(p.partial + at * kV)[lane];
        sum += f;
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
      }
    }
    // (sum = 0: no part has a score above -inf; NaN if the row sees a key)
    const bool nan = (p.causal ? see + r : see) > 0;
    const float inv = sum != 0.f ? 1.f / sum : nan ? NAN : 0.f;
    const int64_t row = ((int64_t)q0 + r) * p.heads + head;
    reinterpret_cast<uint2 *>(p.out + row * kV)[lane] = make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
    if (p.lse && lane == 0) p.lse[row] = sum != 0.f ? top + logf(sum) : nan ? NAN : -INFINITY;
  }
}

// ---------------------------------------------------------------- host

struct Args {
  Strided q_nope, q_pe, k_nope, k_pe, v;
  const int32_t *q_offsets, *kv_offsets;
  int32_t batch, heads;
  int64_t total_q, total_kv;
  int32_t causal;
  float scale;
  void *out;
  float *lse;
  int32_t *dev_status;
};

mla_status_t invalid(const char *why) {
  set_error_detail(why);
  return MLA_ERR_INVALID_ARGUMENT;
}

mla_status_t cuda_failed(cudaError_t e) {
  set_error_detail(cudaGetErrorString(e));
  return MLA_ERR_CUDA;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Strides of 16-byte multiples, at least a row's width
bool strides_ok(const Strided &s, int n) {
  return s.token % 8 == 0 && s.head % 8 == 0 && s.token >= n && s.head >= n && s.token < (1ll << 38) &&
         s.head < (1ll << 38);
}

// [tokens][heads][dims] in boxes of 128 tokens of one head, 64 dims each;
// rows behind the last read as zero.  A tensor without rows is never loaded
// from: its map names one row of `instead`.
bool encode(CUtensorMap *m, const Strided &s, int64_t tokens, int32_t heads, int dims, const void *instead) {
  tmap::EncodeTiledFn fn = tmap::encode_fn();
  if (!fn) return false;
  const bool none = tokens == 0;
  cuuint64_t size[3] = {(cuuint64_t)dims, (cuuint64_t)heads, (cuuint64_t)(none ? 1 : tokens)};
  cuuint64_t strides[2] = {(cuuint64_t)s.head * 2, (cuuint64_t)s.token * 2};
  cuuint32_t box[3] = {64, 1, kTile}, each[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(none ? instead : (const void *)s.p), size,
            strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The split form runs one part a block and at most one block an SM; a part
// leaves 256 rows of 128 fp32 and their log-sum-exps, and what to join.
constexpr size_t kPartBytes = 2 * kTile * (kV + 1) * sizeof(float) + 2 * sizeof(int4);
constexpr size_t kWorkspaceBytes = 32u << 20;
constexpr int kMaxParts = (int)(kWorkspaceBytes / kPartBytes);

// SMs of a device; the kernel's shared-memory opt-in is set on the way.
cudaError_t prepare_device(int dev, int *sms) {
  static std::atomic<int> known[64];
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  *sms = known[dev].load(std::memory_order_acquire);
  if (*sms > 0) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(prefill_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(Smem) + 1024);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(prefill_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem) + 1024);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) known[dev].store(*sms, std::memory_order_release);
  return e;
}

// A launch as a programmatic dependent (every kernel here waits for the one
// before it ahead of its first memory access).
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                   const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Which code the softmax runs, by the keys of a request in the mean (a causal
// item sees about half of them).  Straight-line code against loops, in us, 128
// heads: causal prompts of 1,024 tokens 54.1 / 51.2, 1,500 86.4 / 83.8, 2,048
// 131.6 / 131.0, 8,192 1,640 / 1,710; every key visible 2,048 229 / 236; 700
// tokens of 32 heads 51.9 / 53.0; prompts of 1, 17, 64 and 200 tokens 21.1 / 18.8
// (17.5 since the loops end with the keys).
bool use_long(const Args &a) { return a.total_kv > (a.causal ? 2048 : 512) * (int64_t)a.batch; }

mla_status_t run(const Args &a, void *workspace, size_t workspace_bytes, void *stream) {
  set_error_detail("");
  if (a.batch < 0 || a.total_q < 0 || a.total_kv < 0 || a.total_q >= 1 << 30 || a.total_kv > kMaxKv)
    return invalid("batch < 0, total_q outside [0, 2^30) or total_kv outside [0, 2^26]");
  if (a.heads < 1 || a.heads > kHeads) {
    set_error_detail("num_heads outside [1, 128]");
    return MLA_ERR_UNSUPPORTED;
  }
  if (a.causal != 0 && a.causal != 1) return invalid("causal must be 0 or 1");
  if (!std::isfinite(a.scale) || !(a.scale > 0.f)) return invalid("softmax_scale must be positive and finite");
  if (a.batch == 0 || a.total_q == 0) return MLA_OK;
  if (!a.q_nope.p || !a.q_pe.p || !a.q_offsets || !a.kv_offsets || !a.out ||
      (a.total_kv > 0 && (!a.k_nope.p || !a.k_pe.p || !a.v.p)))
    return invalid("null pointer");
  if (!aligned(a.q_nope.p, 16) || !aligned(a.q_pe.p, 16) || !aligned(a.k_nope.p, 16) || !aligned(a.k_pe.p, 16) ||
      !aligned(a.v.p, 16) || !aligned(a.out, 16))
    return invalid("queries, keys, values and out must be 16-byte aligned");
  if (!aligned(a.q_offsets, 4) || !aligned(a.kv_offsets, 4) || !aligned(a.lse, 4))
    return invalid("q_offsets, kv_offsets and lse must be 4-byte aligned");
  if (!strides_ok(a.q_nope, kNope) || !strides_ok(a.q_pe, kRope) || !strides_ok(a.k_nope, kNope) ||
      !strides_ok(a.v, kV) || !strides_ok(a.k_pe, kRope))
    return invalid("strides must be multiples of 8 elements, at least a row's width and below 2^38");
  if (workspace && (!aligned(workspace, 256) || workspace_bytes < kWorkspaceBytes)) {
    set_error_detail("workspace must be 256-byte aligned and of mla_prefill_workspace_size()");
    return aligned(workspace, 256) ? MLA_ERR_WORKSPACE_TOO_SMALL : MLA_ERR_INVALID_ARGUMENT;
  }
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = prepare_device(dev, &sms);
  if (e != cudaSuccess) return cuda_failed(e);
  Maps maps;
  if (!encode(&maps.q_nope, a.q_nope, a.total_q, a.heads, kNope, a.out) ||
      !encode(&maps.q_pe, a.q_pe, a.total_q, a.heads, kRope, a.out) ||
      !encode(&maps.k_nope, a.k_nope, a.total_kv, a.heads, kNope, a.out) ||
      !encode(&maps.k_pe, a.k_pe, a.total_kv, 1, kRope, a.out) ||
      !encode(&maps.v, a.v, a.total_kv, a.heads, kV, a.out)) {
    set_error_detail("cannot describe an operand to TMA");
    return MLA_ERR_CUDA;
  }
  Params p;
  p.q_offsets = a.q_offsets;
  p.kv_offsets = a.kv_offsets;
  p.batch = a.batch;
  p.heads = a.heads;
  p.total_q = (int32_t)a.total_q;
  p.total_kv = (int32_t)a.total_kv;
  p.causal = a.causal;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out = (__nv_bfloat16 *)a.out;
  p.lse = a.lse;
  p.dev_status = a.dev_status;
  p.partial = p.partial_lse = nullptr;
  p.parts = nullptr;
  p.two_heads = 0;
  // no more items than this, whatever the offsets say
  const int64_t most = (a.total_q / (2 * kTile) + a.batch) * (int64_t)a.heads;
  if (most > INT32_MAX) return invalid("more than 2^31 tiles of 256 queries and a head");
  const cudaStream_t st = (cudaStream_t)stream;
  const int blocks = std::min(sms, kMaxParts);
  const auto kernel = use_long(a) ? prefill_kernel<true> : prefill_kernel<false>;
  if (workspace && most <= blocks / 2) {  // see find_part
    p.partial = (float *)workspace;
    p.partial_lse = p.partial + (int64_t)blocks * 2 * kTile * kV;
    p.parts = (int4 *)(p.partial_lse + (int64_t)blocks * 2 * kTile);
    e = launch(kernel, blocks, kThreads, sizeof(Smem) + 1024, st, maps, p);
    if (e == cudaSuccess) e = launch(join_kernel, blocks, kJoinThreads, 0, st, p);
  } else {
    // two rounds of items and more: halving their number costs no SM its work
    p.two_heads = most >= 2 * sms;
    e = launch(kernel, (unsigned)most, kThreads, sizeof(Smem) + 1024, st, maps, p);
  }
  return e == cudaSuccess ? MLA_OK : cuda_failed(e);
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
  prefill::Args a;
  a.q_nope = Strided{(Bf16)q_nope, q_nope_token_stride, q_nope_head_stride};
  a.q_pe = Strided{(Bf16)q_pe, q_pe_token_stride, q_pe_head_stride};
  a.k_nope = Strided{(Bf16)k_nope, k_nope_token_stride, k_nope_head_stride};
  a.k_pe = Strided{(Bf16)k_pe, k_pe_token_stride, prefill::kRope};
  a.v = Strided{(Bf16)v, v_token_stride, v_head_stride};
  a.q_offsets = q_offsets;
  a.kv_offsets = kv_offsets;
  a.batch = batch;
  a.heads = num_heads;
  a.total_q = total_q;
  a.total_kv = total_kv;
  a.causal = causal;
  a.scale = softmax_scale;
  a.out = out;
  a.lse = lse;
  a.dev_status = dev_status;
  return prefill::run(a, workspace, workspace_bytes, stream);
}

}  // extern "C"
