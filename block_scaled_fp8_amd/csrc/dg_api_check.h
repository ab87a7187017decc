// Argument checks that the C ABI's files share (before any HIP call), and the kernels' form of a cache.
#pragma once

#include "../../include/dg.h"
#include "dg_kv.h"

namespace dg {

inline constexpr int64_t kMaxIndex = int64_t(1) << 30;  // tokens, rows and keys are 32-bit numbers with room to subtract

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks of a cache; `empty`: nothing will be read or written, so its pointers may be NULL.
inline int check_cache(const dg_fp8_kv_cache* c, bool empty) {
  if (!c) return api_fail(DG_ERR_NULL, "cache must not be NULL");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return api_fail(DG_ERR_UNSUPPORTED, "head_dim = %d: 64, 128 and 256 are supported", c->head_dim);
  if (c->num_heads <= 0 || c->num_heads > 65535) return api_fail(DG_ERR_SHAPE, "num_heads = %d must be in [1, 65535]", c->num_heads);
  if (c->page_size <= 0 || c->num_pages < 0) return api_fail(DG_ERR_SHAPE, "page_size = %d must be positive and num_pages = %d not negative", c->page_size, c->num_pages);
  if (int64_t(c->num_pages) * c->page_size > kMaxIndex) return api_fail(DG_ERR_SHAPE, "the cache has more than 2^30 slots");
  if (empty) return DG_OK;
  if (c->num_pages == 0) return api_fail(DG_ERR_SHAPE, "the cache has no pages");
  if (!c->k || !c->v || !c->k_sf || !c->v_sf) return api_fail(DG_ERR_NULL, "the cache's k, v, k_sf and v_sf must not be NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return api_fail(DG_ERR_LAYOUT, "the cache's k and v must be 16-byte aligned");
  if (c->page_stride % 16 || c->head_stride % 16 || c->token_stride % 16)
    return api_fail(DG_ERR_LAYOUT, "the cache's page, head and token strides must be multiples of 16 bytes");
  if (c->page_stride < 0 || c->head_stride < 0 || c->token_stride < c->head_dim)
    return api_fail(DG_ERR_LAYOUT, "the cache's strides must not be negative, and token_stride at least head_dim");
  if (c->sf_page_stride < 0 || c->sf_head_stride < 0 || c->sf_token_stride < 0)
    return api_fail(DG_ERR_LAYOUT, "the cache's scale strides must not be negative");
  // (an offset within a head's page, and within 16 rows, is a 32-bit number)
  if (c->token_stride >= (1 << 24) || c->sf_token_stride >= (1 << 24) || c->token_stride * c->page_size >= (int64_t(1) << 31) ||
      c->sf_token_stride * c->page_size >= (int64_t(1) << 31))
    return api_fail(DG_ERR_LAYOUT, "the cache's token strides must be less than 2^24 bytes, and page_size times them less than 2^31");
  return DG_OK;
}

inline KvCache kernel_cache(const dg_fp8_kv_cache* c) {
  KvCache k{};
  k.k = static_cast<uint8_t*>(c->k);
  k.v = static_cast<uint8_t*>(c->v);
  k.k_sf = c->k_sf;
  k.v_sf = c->v_sf;
  k.page_stride = c->page_stride;
  k.head_stride = c->head_stride;
  k.token_stride = c->token_stride;
  k.sf_page_stride = c->sf_page_stride;
  k.sf_head_stride = c->sf_head_stride;
  k.sf_token_stride = c->sf_token_stride;
  k.num_pages = c->num_pages;
  k.num_heads = c->num_heads;
  k.page = fast_div(c->page_size);
  return k;
}

// Rows [tokens, heads, head_dim] that are read or written with 16-byte accesses.
inline int check_rows(const char* name, const void* p, int64_t token_stride, int64_t head_stride, int esz) {
  if (!p) return api_fail(DG_ERR_NULL, "%s must not be NULL", name);
  if (!aligned(p, 16) || (token_stride * esz) % 16 || (head_stride * esz) % 16)
    return api_fail(DG_ERR_LAYOUT, "%s must have 16-byte aligned rows (start, token stride and head stride)", name);
  if (token_stride < 0 || head_stride < 0) return api_fail(DG_ERR_LAYOUT, "%s's strides must not be negative", name);
  return DG_OK;
}

}  // namespace dg
