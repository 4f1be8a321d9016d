// Host helpers shared by the C entry points: facts about the current device
// that are looked up once, launches with programmatic stream serialization,
// tensor maps, and checks of arguments.
#pragma once

#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "spec_verify.h"

namespace sv {

// Per-device facts looked up once (SM count, kernel attributes set). Reads
// take an atomic fast path; the first lookup on a device runs under a mutex,
// so concurrent first calls from several host threads are safe. Devices past
// kMaxDevices are not cached (looked up on every call).
constexpr int kMaxDevices = 64;
inline std::mutex g_dev_cache_mu;
inline std::atomic<int> g_sm_count[kMaxDevices];

inline int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  return dev;
}

// SM count of the current device.
inline int sm_count() {
  const int dev = current_device();
  const bool cached = dev >= 0 && dev < kMaxDevices;
  if (cached) {
    const int n = g_sm_count[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
  }
  std::lock_guard<std::mutex> lock(g_dev_cache_mu);
  if (cached && g_sm_count[dev].load(std::memory_order_relaxed) > 0) return g_sm_count[dev].load();
  int n = 0;
  if (dev < 0 || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  if (cached) g_sm_count[dev].store(n, std::memory_order_release);
  return n;
}

// Largest dynamic shared memory and the largest shared-memory carveout, so
// two rings fit on one SM.
template <typename Kern>
cudaError_t set_smem_attrs(Kern kernel, int smem_bytes) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                              static_cast<int>(cudaSharedmemCarveoutMaxShared));
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

template <typename Kern, typename... Args>
cudaError_t launch(Kern kernel, int grid, int block, size_t smem, cudaStream_t stream, bool pdl,
                   const Args&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// set_smem_attrs once per kernel and device, then a PDL launch.
template <auto Kern>
struct SmemSet {
  inline static std::atomic<uint64_t> done{0};
};

// `most` bounds every later call's smem.
template <auto Kern, typename... Args>
cudaError_t launch_smem(int grid, int block, size_t smem, size_t most, cudaStream_t stream, const Args&... args) {
  const int dev = current_device();
  const bool cached = dev >= 0 && dev < kMaxDevices;
  if (!cached || !(SmemSet<Kern>::done.load(std::memory_order_acquire) >> dev & 1)) {
    const cudaError_t e = set_smem_attrs(Kern, static_cast<int>(most));
    if (e != cudaSuccess) return e;
    if (cached) SmemSet<Kern>::done.fetch_or(1ull << dev, std::memory_order_release);
  }
  return launch(Kern, grid, block, smem, stream, true, args...);
}

inline sv_status done(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

inline bool valid_rows(const sv_rows* r, int es) {
  return r && r->data && aligned(r->data, 16) && r->stride_b * es % 16 == 0 && r->stride_n * es % 16 == 0 &&
         r->stride_h * es % 16 == 0;
}

// cuTensorMapEncodeTiled of the loaded driver.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encode_tiled() {
  static std::atomic<void*> found{nullptr};
  void* f = found.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return nullptr;
    found.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

}  // namespace sv
