// Host-side helpers shared by the library's source files: error codes, alignment, per-device
// attributes, shared-memory limits and launches that may overlap the kernel before them.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "hbl.h"

namespace hbl {

// Records a CUDA error for hbl_last_cuda_error (thread-local) and returns HBL_ECUDA.
hbl_status cuda_fail(cudaError_t e);

// Reads and clears the error flag of the attention and cache kernels (synchronises `s`).
hbl_status attn_take_errors(cudaStream_t s, int* flags);

#define HBL_CHECK_LAUNCH()                          \
  do {                                              \
    const cudaError_t e_ = cudaGetLastError();      \
    if (e_ != cudaSuccess) return cuda_fail(e_);    \
  } while (0)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool is_pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }

constexpr int kMaxDevices = 64;

inline int device_sms(int dev) {
  static int cache[kMaxDevices] = {0};
  if (dev < 0 || dev >= kMaxDevices) return 148;
  if (cache[dev] == 0) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    cache[dev] = v > 0 ? v : 148;
  }
  return cache[dev];
}

// Raise a kernel's dynamic shared memory limit when a launch needs more than was allowed so far
// on the current device (the limit does not change occupancy; the launch's own size does). The
// default limit counts static shared memory too, so it is raised for any non-zero size.
struct SmemLimit {
  std::mutex mu;
  int allowed[64] = {0};
  int resident[64] = {0};  // CTAs of the kernel that fit on the device at once (see resident_ctas)
};

template <typename F>
cudaError_t allow_smem(F* kernel, int bytes, SmemLimit& lim) {
  int dev = 0;
  cudaGetDevice(&dev);
  dev &= 63;
  std::lock_guard<std::mutex> lk(lim.mu);
  if (lim.allowed[dev] >= bytes) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  // the kernels stream their data, so L1 matters less than shared memory: ask for the largest
  // carveout, so that the occupancy query (which sizes the persistent grids) and the launch agree
  // on how many CTAs share an SM
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) lim.allowed[dev] = bytes;
  return e;
}

// CTAs of a kernel that fit on the current device at once, for launches that always take the same
// threads and shared memory.
template <typename F>
int resident_ctas(F* kernel, int threads, int smem, SmemLimit& lim) {
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lk(lim.mu);
  int& n = lim.resident[dev & 63];
  if (n == 0) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1)
      per_sm = 1;
    n = per_sm * device_sms(dev);
  }
  return n;
}

inline PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Launch with programmatic stream serialization: the kernel may be scheduled while the one before
// it in the stream drains, and waits for it (pdl_wait) before it touches memory.
template <typename... KArgs, typename... Args>
hbl_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return cuda_fail(e);
  HBL_CHECK_LAUNCH();
  return HBL_OK;
}

}  // namespace hbl
