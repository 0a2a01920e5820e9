// fs_bitonic.cuh -- bitonic sort of 64-bit keys, a power of two of them, ascending.
#pragma once

#include <cstdint>

namespace fs {

constexpr int kSortBlock = 1024;   // threads of the shared-memory bitonic kernels
constexpr int kSortSmem = 2 * kSortBlock;  // keys sorted per block in shared memory

__device__ __forceinline__ void cmp_swap(uint64_t& a, uint64_t& b, bool ascending) {
  if ((a > b) == ascending) {
    const uint64_t t = a;
    a = b;
    b = t;
  }
}

// Bitonic stages with sizes k <= kSortSmem (first call: all of them; later calls: the
// strides j < kSortSmem of merge size k), in shared memory, one block per kSortSmem keys.
static __global__ void __launch_bounds__(kSortBlock) bitonic_smem_kernel(uint64_t* keys, int64_t k_merge) {
  __shared__ uint64_t s[kSortSmem];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortSmem;
  const int t = threadIdx.x;
  s[t] = keys[base + t];
  s[t + kSortBlock] = keys[base + t + kSortBlock];
  __syncthreads();
  const int64_t k_lo = k_merge > 0 ? k_merge : 2;
  const int64_t k_hi = k_merge > 0 ? k_merge : kSortSmem;
  for (int64_t k = k_lo; k <= k_hi; k <<= 1) {
    for (int64_t j = (k_merge > 0 ? kSortSmem / 2 : k / 2); j > 0; j >>= 1) {
      // thread t handles the pair (i, i + j) with i = 2t - (t mod j)
      const int i = 2 * t - (t & static_cast<int>(j - 1));
      const bool asc = ((base + i) & k) == 0;
      cmp_swap(s[i], s[i + j], asc);
      __syncthreads();
    }
  }
  keys[base + t] = s[t];
  keys[base + t + kSortBlock] = s[t + kSortBlock];
}

// One bitonic step with stride j >= kSortSmem over all n_pow2 keys.
static __global__ void __launch_bounds__(256) bitonic_global_kernel(uint64_t* keys, int64_t n_pow2,
                                                             int64_t k, int64_t j) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t >= n_pow2 / 2) return;
  const int64_t i = 2 * t - (t & (j - 1));
  const bool asc = (i & k) == 0;
  uint64_t a = keys[i], b = keys[i + j];
  if ((a > b) == asc) {
    keys[i] = b;
    keys[i + j] = a;
  }
}

}  // namespace fs
