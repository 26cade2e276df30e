// The paged cache of an Attention source (afd_cache) as its kernels see it:
// what writes it (afd_cache.cu) and what reads it (afd_attention.cu).
#pragma once

#include <stdint.h>

#include "afd.h"
#include "afd_pointers.cuh"

namespace afd {

constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxCacheBytes = (int64_t)1 << 38;  // of keys, or values: places in units of 64 bytes in 32 bits

struct CacheParams {
  uint8_t* k;
  uint8_t* v;
  uint32_t k_page_units, v_page_units;  // of 64 bytes, from a page to the next
  float* k_scale;  // [pages][heads][page_size], E4M3 only
  float* v_scale;
  int32_t pages, page_size;
};

// The sizes, strides and alignment of a cache; its buffers may be missing where
// it has no pages.
inline afd_status check_cache(const afd_cache* c) {
  if (!c || c->num_pages < 0 || c->page_size < 1 || c->num_kv_heads < 1 || c->head_dim < 1) return AFD_ERR_ARG;
  if (c->dtype != AFD_BF16 && c->dtype != AFD_FP8_E4M3) return AFD_ERR_ARG;
  const bool fp8 = c->dtype == AFD_FP8_E4M3;
  if (!fp8 && (c->k_scale || c->v_scale)) return AFD_ERR_ARG;
  const int64_t each = fp8 ? 1 : 2;
  if (c->num_pages > 0) {
    if (!c->k || !c->v || (fp8 && (!c->k_scale || !c->v_scale)) || !aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4))
      return AFD_ERR_ARG;
    if (c->num_kv_heads <= kMaxHeads && c->head_dim <= 1024) {  // (no product below passes 64 bits)
      const int64_t page = (int64_t)c->num_kv_heads * c->page_size * c->head_dim;
      if (c->k_page_stride < page || c->v_page_stride < page) return AFD_ERR_ARG;
    }
  }
  if (c->head_dim != 64 && c->head_dim != 128) return AFD_ERR_UNSUPPORTED;
  if (c->num_kv_heads > kMaxHeads || (int64_t)c->num_pages * c->page_size > INT32_MAX) return AFD_ERR_UNSUPPORTED;
  if (c->num_pages > 0 &&
      (c->k_page_stride > kMaxCacheBytes / each / c->num_pages || c->v_page_stride > kMaxCacheBytes / each / c->num_pages ||
       c->k_page_stride * each % 64 || c->v_page_stride * each % 64 || !aligned_to(c->k, 16) || !aligned_to(c->v, 16)))
    return AFD_ERR_UNSUPPORTED;
  return AFD_OK;
}

// What the kernels use of a checked cache; false: a buffer that they cannot reach.
inline bool view_cache(const afd_cache* c, CacheParams* out) {
  const int64_t each = c->dtype == AFD_FP8_E4M3 ? 1 : 2;
  *out = {};
  out->k_page_units = (uint32_t)(c->k_page_stride * each / 64), out->v_page_units = (uint32_t)(c->v_page_stride * each / 64);
  out->pages = c->num_pages, out->page_size = c->page_size;
  if (c->num_pages == 0) return true;
  return device_view(static_cast<uint8_t*>(c->k), &out->k) && device_view(static_cast<uint8_t*>(c->v), &out->v) &&
         (each == 2 || (device_view(c->k_scale, &out->k_scale) && device_view(c->v_scale, &out->v_scale)));
}

}  // namespace afd
