// Ragged rows: request b owns rows [offsets[b], offsets[b+1]) of a packed
// tensor of `total` rows.  The offsets live on the device, so kernels cut them
// to the tensor (no access leaves it, whatever they hold) and one block
// reports those that fall or leave it.
#pragma once

#include "common.cuh"

namespace mla {
namespace ragged {

__device__ __forceinline__ int32_t cut(int32_t offset, int32_t total) {
  return min(max(offset, 0), total);
}

// Called by `threads` threads of one block, each with its own `tid`.
__device__ __forceinline__ void check_offsets(const int32_t *offsets, int32_t batch, int32_t total,
                                              int tid, int threads, int32_t *dev_status) {
  bool bad = false;
  for (int32_t b = tid; b < batch; b += threads) {
    const int32_t a = offsets[b], z = offsets[b + 1];
    bad |= a < 0 || a > z || z > total;
  }
  if (bad) report(dev_status, MLA_ERR_DEVICE_RANGE);
}

struct Place {
  int32_t request, offset;  // and its first row
};

// The request that owns each lane's row t, by a whole warp: the last one with
// offsets[b] <= t (0 when there is none).  Up to 1,024 requests 32 offsets are
// compared at a time, one load's latency each; more are searched by halves.
__device__ __forceinline__ Place place_of(const int32_t *offsets, int32_t batch, int32_t t) {
  Place at = {0, 0};
  if (batch <= 1024) {
    const int lane = threadIdx.x & 31;
    for (int32_t b0 = 0; b0 < batch; b0 += 32) {
      const int32_t mine = b0 + lane < batch ? offsets[b0 + lane] : INT32_MAX;
      const int n = min(32, batch - b0);
      for (int i = 0; i < n; ++i) {
        const int32_t o = __shfl_sync(0xffffffffu, mine, i);
        if (o <= t || b0 + i == 0) at = Place{b0 + i, o};
      }
    }
    return at;
  }
  int32_t lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (offsets[mid] <= t) lo = mid; else hi = mid;
  }
  return Place{lo, offsets[lo]};
}

}  // namespace ragged
}  // namespace mla
