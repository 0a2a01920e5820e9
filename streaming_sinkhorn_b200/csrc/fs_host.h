// fs_host.h -- host-side pieces that the library's translation units share: error capture,
// launch counting, and launches that turn a CUDA failure into a status.
#pragma once

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fs.h"

namespace fs {

// Defined in fs_api.cu: the text for fs_last_cuda_error, and fs_launch_count's counter.
void record_cuda_error(const char* what, cudaError_t e);
void count_launches(int64_t k);

inline fs_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return FS_OK;
  record_cuda_error(what, e);
  cudaGetLastError();  // clears a non-sticky error, so it is not reported twice
  return FS_ERR_CUDA;
}

// Device attributes a launch plan needs, of the current device.
inline int current_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  return sms > 0 ? sms : 148;
}

// Kernel attributes are set once per kernel and device (the runtime keeps them per device).
class PerDeviceOnce {
 public:
  template <typename F>
  fs_status run(const char* what, F&& set) {
    int dev = 0;
    fs_status s = cuda_status(cudaGetDevice(&dev), "cudaGetDevice");
    if (s != FS_OK) return s;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done_.load(std::memory_order_acquire) & bit)) return FS_OK;
    s = cuda_status(set(), what);
    if (s == FS_OK && dev < 64) done_.fetch_or(bit, std::memory_order_release);
    return s;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// CTAs of a kernel that an SM holds at once with this much shared memory; the last answer for each
// device is kept with its question.
class PerDeviceOccupancy {
 public:
  int get(const void* fn, int threads, size_t smem) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 64;
    if (dev < 64) {
      const uint64_t known = known_[dev].load(std::memory_order_relaxed);
      if (known != 0 && known >> 8 == smem) return static_cast<int>(known & 255);
    }
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess) {
      cudaGetLastError();
      n = 1;
    }
    if (n < 1) n = 1;
    // (an SM holds 32 CTAs at most)
    if (dev < 64 && n < 256)
      known_[dev].store(static_cast<uint64_t>(smem) << 8 | static_cast<uint64_t>(n),
                        std::memory_order_relaxed);
    return n;
  }

 private:
  std::atomic<uint64_t> known_[64] = {};
};

// Launches `kernel` (a cluster of `cluster` CTAs along x when cluster > 1; kCooperative: all
// CTAs resident at once, or an error).
constexpr int kCooperative = -1;
template <typename... P, typename... A>
fs_status launch(const char* what, void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                 cudaStream_t st, int cluster, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  if (cluster > 1) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  if (cluster == kCooperative) {
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  const fs_status s = cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...), what);
  if (s == FS_OK) count_launches(1);
  return s;
}

// A temperature: its inverse, in base 2 too, is a factor of float32 arithmetic.
inline fs_status check_eps(float eps) {
  return std::isfinite(eps) && eps > 0.0f && std::isfinite(1.5f / eps) ? FS_OK : FS_ERR_EPS;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace fs
