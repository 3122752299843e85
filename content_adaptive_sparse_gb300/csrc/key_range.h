// The range of 32-bit keys that holds an eviction's border (scored_cache.cu): it is cut into up to 2048 equal bins, and
// the bin with the border is the next range.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define SA_BOTH __host__ __device__ __forceinline__
#else
#define SA_BOTH inline
#endif

namespace sa {

struct KeyRange {
  static constexpr int kBins = 2048;
  uint32_t low, high;               // both inclusive

  // Keys of a bin, as a power of two: (high - low) >> shift() < kBins. For low < high.
  SA_BOTH int shift() const {
#ifdef __CUDA_ARCH__
    const int zeros = __clz((int)(high - low));
#else
    const int zeros = __builtin_clz(high - low);
#endif
    return zeros < 21 ? 21 - zeros : 0;
  }
  SA_BOTH bool holds(uint32_t k) const { return k - low <= high - low; }
  SA_BOTH uint32_t bin(uint32_t k, int shift) const { return (k - low) >> shift; }
  SA_BOTH void take(uint32_t bin, int shift) {
    low += bin << shift;
    const uint32_t width = (1u << shift) - 1u;         // low + width may lie past the largest number
    high = high - low < width ? high : low + width;
  }
};

}  // namespace sa
