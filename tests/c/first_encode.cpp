// Host threads whose first tensor maps are encoded at the same moment, with a lookup of the driver's encoder
// that takes a while: every thread has to get the encoder.
#include "tma_host.h"

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                       const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}

// in the CUDA run-time library's place
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned int, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  std::this_thread::sleep_for(std::chrono::milliseconds(100));
  *p = reinterpret_cast<void*>(encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

int main() {
  std::atomic<int> missing{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&] {
      CUtensorMap map;
      missing += !sa::encode_bhnd_map(&map, nullptr, 1, 1, 1, 64, 64, 64, 64, 64, 1, CU_TENSOR_MAP_SWIZZLE_128B);
    });
  for (auto& t : threads) t.join();
  std::printf("%d threads without the encoder\n", missing.load());
  return missing.load() != 0;
}
