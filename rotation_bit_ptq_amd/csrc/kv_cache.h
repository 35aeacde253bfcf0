// The paged key-value cache as the kernels see it.
#pragma once

#include "block_common.h"

namespace orbit {
namespace block {

struct Cache {
  char *k, *v;
  _Float16 *ks, *vs;  // INT8: one scale per (page, head, position)
  uint32_t pages, page_mask;
  int page_shift, kv_heads, head_dim;
};

inline orbit_status check_cache(const orbit_kv_cache& c) {
  if (c.format != ORBIT_KV_BF16 && c.format != ORBIT_KV_F16 && c.format != ORBIT_KV_INT8) return ORBIT_E_ARG;
  const bool coded = c.format == ORBIT_KV_INT8;  // 16-byte vectors hold 16 codes; scales are read by fours
  if (c.page_size < (coded ? 4 : 1) || c.page_size > 1024 || (c.page_size & (c.page_size - 1))) return ORBIT_E_SHAPE;
  if (c.kv_heads < 1 || c.kv_heads > 1024) return ORBIT_E_SHAPE;
  if (c.head_dim < 8 || c.head_dim > 256 || c.head_dim % (coded ? 16 : 8)) return ORBIT_E_SHAPE;
  if (c.pages < 0 || c.pages >= (1LL << 31) || c.pages * c.page_size >= (1LL << 31)) return ORBIT_E_SHAPE;
  if (c.pages > 0) {
    if (!c.k || !c.v || !aligned_to(c.k, 16) || !aligned_to(c.v, 16)) return ORBIT_E_ARG;
    if (coded && (!c.k_scale || !c.v_scale || !aligned_to(c.k_scale, 16) || !aligned_to(c.v_scale, 16)))
      return ORBIT_E_ARG;
  }
  return ORBIT_OK;
}

inline Cache cache_of(const orbit_kv_cache& c) {
  Cache d = {};
  d.k = (char*)c.k;
  d.v = (char*)c.v;
  d.ks = (_Float16*)c.k_scale;
  d.vs = (_Float16*)c.v_scale;
  d.pages = (uint32_t)c.pages;
  d.page_mask = (uint32_t)c.page_size - 1;
  while ((1 << d.page_shift) < c.page_size) ++d.page_shift;
  d.kv_heads = c.kv_heads;
  d.head_dim = c.head_dim;
  return d;
}

// Row (in units of head_dim elements, or of scales) of position `off` of
// head `h` in page `page`.
__device__ __forceinline__ long long cache_row(const Cache& c, uint32_t page, int h, uint32_t off) {
  return (((long long)page * c.kv_heads + h) << c.page_shift) + off;
}

}  // namespace block
}  // namespace orbit
