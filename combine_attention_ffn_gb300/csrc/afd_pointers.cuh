// Host helpers of the calls that take no context: checks of caller buffers,
// launches.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "afd_internal.cuh"

namespace afd {

// Sets a kernel's dynamic shared memory limit once per device (`done`: one
// bit for each, static to the caller's kernel).
template <typename K>
inline cudaError_t allow_shared(K kernel, int bytes, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// The address a kernel on the current device uses for a caller buffer: the
// buffer itself in that device's memory or in managed memory, the mapped
// device address of page-locked host memory. Pageable host memory, and
// memory of another device, are refused before anything is enqueued.
template <typename T>
inline bool device_view(T* p, T** out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  cudaPointerAttributes a = {};
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if ((a.type == cudaMemoryTypeDevice && a.device == dev) || a.type == cudaMemoryTypeManaged) {
    *out = p;
    return true;
  }
  if (a.type == cudaMemoryTypeHost && a.devicePointer) {
    *out = static_cast<T*>(a.devicePointer);
    return true;
  }
  return false;
}

// Launches a kernel as a programmatic dependent of the work before it on the
// stream: its blocks may start while that work still runs, and the kernel
// waits (pdl_wait) before it touches memory. `cluster`: blocks of a cluster,
// where the kernel leaves that to the launch.
template <typename... Params, typename... Args>
inline cudaError_t launch_clusters(void (*kernel)(Params...), int64_t grid, int block, int cluster, size_t smem,
                                   cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  take_stream_turn(stream);
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

template <typename... Params, typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(Params...), int64_t grid, int block, size_t smem, cudaStream_t stream,
                                    Args&&... args) {
  return launch_clusters(kernel, grid, block, 0, smem, stream, static_cast<Args&&>(args)...);
}

// Sizes that leave a step of any loop over rows or columns, and a tile's
// rounding up, below 2^31.
constexpr int64_t kMaxRows = INT32_MAX - (1 << 20);
constexpr int32_t kMaxFeatures = 1 << 24;

// Whether p is on an `align`-byte boundary.
inline bool aligned_to(const void* p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }

}  // namespace afd
