// Host checks of caller buffers, shared by the calls that take no context.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace afd {

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

// Whether [p, p + bytes) starts on an `align`-byte boundary.
inline bool aligned_to(const void* p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0; }

}  // namespace afd
