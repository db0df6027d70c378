// paged.cuh -- host-side checks shared by the calls that take strided rows or
// a paged cache.
#pragma once

#include "common.cuh"

namespace sv {
namespace paged {

inline bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Rows [token][head][D]: 16-byte aligned rows, strides that index without
// overflow (2^40 elements times 2^31 rows would not: the bound keeps the
// kernels' 64-bit offsets exact).
inline bool good_rows(const sv_rows *r, long long T) {
  if (!r || (T > 0 && !r->ptr) || !aligned(r->ptr, 16)) return false;
  const int64_t lim = (int64_t)1 << 31;
  return r->token_stride >= 0 && r->head_stride >= 0 && r->token_stride % 8 == 0 &&
         r->head_stride % 8 == 0 && r->token_stride <= lim && r->head_stride <= (lim << 8);
}

inline sv_status check_cache(const sv_paged_kv *c, int D) {
  if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return SV_ERR_INVALID_ARG;
  if (c->dtype != SV_BF16 && c->dtype != SV_E4M3) return SV_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1) return SV_ERR_INVALID_ARG;
  const int64_t unit = c->dtype == SV_E4M3 ? 16 : 8;  // elements in 16 bytes
  const int64_t lim = (int64_t)1 << 38;               // 2^39 bytes at bf16: a tensor map's bound is 2^40
  for (int64_t s : {c->page_stride, c->slot_stride, c->head_stride})
    if (s <= 0 || s % unit != 0 || s > lim) return SV_ERR_INVALID_ARG;
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return SV_ERR_INVALID_ARG;
  if (c->dtype == SV_BF16 && (c->k_scale || c->v_scale)) return SV_ERR_INVALID_ARG;
  if (c->page_size % 16 != 0 || c->page_size > 65536 || c->num_pages > 0x7fffffffLL) return SV_ERR_UNSUPPORTED;
  if (c->dtype == SV_E4M3 && D == 64) return SV_ERR_UNSUPPORTED;
  return SV_OK;
}

}  // namespace paged
}  // namespace sv
