// checks.cuh -- what the argument checks of the entry points share (host only).
#pragma once

#include <initializer_list>

#include "kda_common.cuh"

namespace kda {

// Sizes leave a tile's room below 2^31, so that the kernels round up in 32 bits.
constexpr int kMaxSize = 0x7fffffff - 256;

inline int sm_count() {  // of the current device
  static std::atomic<int> count[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  n = count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
    count[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}
inline bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline size_t elem(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }

// An output at the address of an input: other warps still read what one has written.
inline bool same(const void* out, std::initializer_list<const void*> in) {
  for (const void* p : in)
    if (out && out == p) return true;
  return false;
}

}  // namespace kda
