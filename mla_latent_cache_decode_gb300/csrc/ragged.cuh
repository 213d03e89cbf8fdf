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

// The request that owns row t, given offsets[0] <= t < offsets[batch].
__device__ __forceinline__ int32_t request_of(const int32_t *offsets, int32_t batch, int32_t t) {
  int32_t lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (offsets[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace ragged
}  // namespace mla
