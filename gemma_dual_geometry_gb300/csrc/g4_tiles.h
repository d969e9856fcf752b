// Which tiles of keys an interval of positions touches.  Keys may end at position 2^31 - 1 (a ring holds any
// position), so nothing is added to a key that could be the last one.
#pragma once

#include <cuda_runtime.h>

namespace g4 {

// One past the last tile of `tile` keys each that holds a key before `end`.
__host__ __device__ constexpr int tiles_before(int end, int tile) { return end > 0 ? (end - 1) / tile + 1 : 0; }

// How many of the n keys from `key` on lie before `end` (key, end >= 0).
__host__ __device__ constexpr int keys_before(int end, int key, int n) {
  return end <= key ? 0 : end - key < n ? end - key : n;
}

}  // namespace g4
