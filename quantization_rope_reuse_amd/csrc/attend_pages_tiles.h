// The tiles of cached tokens that a set of query rows walks (host and device
// code).
#pragma once

#include <hip/hip_runtime_api.h>

namespace hkv {

// Tiles of `size` tokens that a view has: [0, pre) and [lo, hi).
struct TileList {
  int pre, lo, count;
  __host__ __device__ inline int at(int i) const { return i < pre ? i : i - pre + lo; }
};

// 0 <= pre, lo, hi <= 2^31 - 1.
__host__ __device__ inline TileList tiles_of_view(int pre, int lo, int hi, int size) {
  TileList t;
  t.pre = pre / size + (pre % size != 0);
  const int end = hi / size + (hi % size != 0);
  const int first = (lo < hi ? lo : hi) / size;
  t.lo = first > t.pre ? first : t.pre;
  t.count = t.pre + (end > t.lo ? end - t.lo : 0);
  return t;
}

}  // namespace hkv
