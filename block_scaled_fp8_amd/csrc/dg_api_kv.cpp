// C ABI of the FP8 key/value cache: argument validation, the split of the work, and launch.
// Validation runs before any HIP call.
#include <cmath>

#include "../../include/dg.h"
#include "dg_kv.h"

namespace {

using dg::api_fail;
using dg::api_ok;

constexpr int64_t kMaxIndex = int64_t(1) << 30;  // tokens, rows and keys are 32-bit numbers with room to subtract

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks of a cache; `empty`: nothing will be read or written, so its pointers may be NULL.
int check_cache(const dg_fp8_kv_cache* c, bool empty) {
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

dg::KvCache kernel_cache(const dg_fp8_kv_cache* c) {
  dg::KvCache k{};
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
  k.page = dg::fast_div(c->page_size);
  return k;
}

// Rows [tokens, heads, head_dim] that are read or written with 16-byte accesses.
int check_rows(const char* name, const void* p, int64_t token_stride, int64_t head_stride, int esz) {
  if (!p) return api_fail(DG_ERR_NULL, "%s must not be NULL", name);
  if (!aligned(p, 16) || (token_stride * esz) % 16 || (head_stride * esz) % 16)
    return api_fail(DG_ERR_LAYOUT, "%s must have 16-byte aligned rows (start, token stride and head stride)", name);
  if (token_stride < 0 || head_stride < 0) return api_fail(DG_ERR_LAYOUT, "%s's strides must not be negative", name);
  return DG_OK;
}

int move(bool write, const dg_fp8_kv_cache* cache, int32_t num_tokens, const void* k, int64_t k_token_stride,
         int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride, int32_t dtype,
         const int64_t* slots, hipStream_t stream) {
  if (dtype != DG_IN_BF16 && dtype != DG_IN_F32) return api_fail(DG_ERR_DTYPE, "dtype %d is not DG_IN_BF16 or DG_IN_F32", dtype);
  if (num_tokens < 0 || num_tokens > kMaxIndex) return api_fail(DG_ERR_SHAPE, "num_tokens = %d must be in [0, 2^30]", num_tokens);
  if (int s = check_cache(cache, num_tokens == 0)) return s;
  if (num_tokens == 0) return api_ok();
  const int esz = dtype == DG_IN_BF16 ? 2 : 4;
  if (int s = check_rows("k", k, k_token_stride, k_head_stride, esz)) return s;
  if (int s = check_rows("v", v, v_token_stride, v_head_stride, esz)) return s;
  if (!slots) return api_fail(DG_ERR_NULL, "slots must not be NULL");
  if (!aligned(slots, 8)) return api_fail(DG_ERR_LAYOUT, "slots must be 8-byte aligned");
  dg::KvMoveParams p{};
  p.c = kernel_cache(cache);
  p.k_token_stride = k_token_stride;
  p.k_head_stride = k_head_stride;
  p.v_token_stride = v_token_stride;
  p.v_head_stride = v_head_stride;
  // A grid has less than 2^32 threads (one of more is cut to its low 32 bits without an error), and a row takes up to 32.
  constexpr int32_t kMost = 1 << 26;
  const bool bf16 = dtype == DG_IN_BF16;
  for (int32_t from = 0; from < num_tokens; from += kMost) {
    p.k = static_cast<char*>(const_cast<void*>(k)) + from * k_token_stride * esz;
    p.v = static_cast<char*>(const_cast<void*>(v)) + from * v_token_stride * esz;
    p.slots = slots + from;
    p.num_tokens = num_tokens - from < kMost ? num_tokens - from : kMost;
    const hipError_t e = write ? dg::launch_kv_write(p, cache->head_dim, bf16, stream) : dg::launch_kv_read(p, cache->head_dim, bf16, stream);
    if (e != hipSuccess) return api_fail(DG_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  }
  return api_ok();
}

// ---------------------------------------------------------------- attention
struct AttnShape {
  int32_t batch, total_q, num_q_heads, max_seqlen_q, max_seqlen_k, window, sinks;
  bool equal;
};

int check_shape(const AttnShape& a, int32_t num_kv_heads) {
  if (a.batch < 0 || a.total_q < 0) return api_fail(DG_ERR_SHAPE, "batch = %d and total_q = %d must not be negative", a.batch, a.total_q);
  if (num_kv_heads <= 0 || a.num_q_heads <= 0 || a.num_q_heads % num_kv_heads)
    return api_fail(DG_ERR_SHAPE, "num_q_heads = %d must be a positive multiple of the cache's %d heads", a.num_q_heads, num_kv_heads);
  if (int64_t(a.total_q) * a.num_q_heads > kMaxIndex) return api_fail(DG_ERR_SHAPE, "total_q * num_q_heads must be at most 2^30");
  if (a.window < 0 || a.sinks < 0) return api_fail(DG_ERR_SHAPE, "window = %d and sinks = %d must not be negative", a.window, a.sinks);
  if (a.max_seqlen_q < 0 || a.max_seqlen_k < 0) return api_fail(DG_ERR_SHAPE, "max_seqlen_q = %d and max_seqlen_k = %d must not be negative", a.max_seqlen_q, a.max_seqlen_k);
  if (a.equal && a.batch > 0 && a.total_q % a.batch) return api_fail(DG_ERR_SHAPE, "without cu_seqlens_q, total_q = %d must be a multiple of batch = %d", a.total_q, a.batch);
  return DG_OK;
}

// The kernel, and a call's items: tiles of rows of its sequences.
struct AttnItems {
  int form;
  int64_t rows, q_tiles, items;  // rows of a sequence at most, tiles of them, tiles in all
};

AttnItems items_of(const AttnShape& a, int32_t num_kv_heads, int32_t head_dim) {
  const int64_t per_seq = a.equal ? a.total_q / a.batch : a.max_seqlen_q < a.total_q ? a.max_seqlen_q : a.total_q;
  AttnItems n;
  n.rows = per_seq * (a.num_q_heads / num_kv_heads);
  // The few-rows kernel reads the keys once for every 32 rows (from L2 after the first), the many-rows kernel
  // spends whole tiles of 128 or 256: 28 against 34 us with 4 x 30 queries over 4030 keys (120 rows), 20 against
  // 30 with 32 over 4032 (128), but 189 against 178 with 32 x 32 over up to 8032.
  n.form = n.rows <= 16 ? dg::ATTN_NARROW_16 : n.rows <= 128 ? dg::ATTN_NARROW_32 : dg::ATTN_WIDE;
  const int tile = dg::attn_tile_rows(n.form, head_dim);
  n.q_tiles = (n.rows + tile - 1) / tile;
  n.items = a.batch * n.q_tiles;
  return n;
}

// Items are 32-bit numbers to the kernels, and a grid has less than 2^32 threads (one of more is cut to its low
// 32 bits without an error).
int check_items(const AttnShape& a, int32_t num_kv_heads, int32_t head_dim) {
  const AttnItems n = items_of(a, num_kv_heads, head_dim);
  if (n.items > int64_t(UINT32_MAX) / (int64_t(num_kv_heads) * dg::attn_threads(n.form, head_dim)))
    return api_fail(DG_ERR_SHAPE, "%d sequences of up to %lld query rows a key head are more tiles than a launch holds%s", a.batch,
                    (long long)n.rows, a.equal ? "" : ": max_seqlen_q should bound the new tokens of a sequence");
  return DG_OK;
}

struct AttnPlan {
  int form = 0, q_tiles = 1, head_aim = 0, least_tiles = 1, max_cut = 1, join_rows = 1, join_few = 0, join_steps = 1, waves = 4;
  int64_t items = 0, most_parts = 0;
};

AttnPlan plan_of(const AttnShape& a, int32_t num_kv_heads, int32_t head_dim, int num_sms) {
  const AttnItems n = items_of(a, num_kv_heads, head_dim);
  const int64_t group = a.num_q_heads / num_kv_heads;
  AttnPlan pl;
  pl.form = n.form;
  const int tile = dg::attn_tile_rows(pl.form, head_dim), keys = dg::attn_tile_keys(pl.form, head_dim);
  pl.q_tiles = int(n.q_tiles);
  pl.join_rows = int(n.rows < tile ? n.rows : tile);
  pl.items = n.items;
  // Key tiles of an item at most, from the host's bound of the lengths (rounded up at both ends of a window).
  int64_t tiles = (a.max_seqlen_k + int64_t(keys) - 1) / keys;
  if (a.window) {
    const int64_t seen = (int64_t(a.window) + (tile - 1) / group + keys - 1) / keys + 1 + (int64_t(a.sinks) + keys - 1) / keys;
    if (seen < tiles) tiles = seen;
  }
  // Cutting items along the keys costs a second kernel and the parts' way through memory.  It is for items
  // that fill at most half of the chip, and for longer ones (whose lengths it also evens out) up to twice it, or
  // four times with tiles of 32 rows, whose workgroups are long (80 x 16 queries over 5016 keys, 1280 items
  // for 512 places, 315 us whole, 236 cut; single tokens of 256 sequences, 2048 for 768, 409 whole, 416 cut).
  // Few rows: 128 sequences in a window of 1024 (512 items of 35 tiles for 768 places) 32 us whole, 52 cut;
  // 64 sequences of up to 8192 keys (512 items of up to 256 tiles) 128 whole, 123 cut.  Many rows, one
  // sequence: 1024 queries over 4024 keys (128 items for 256 places) 104 whole, 78 cut; 1280 over 7424 (160
  // items) 182 whole, 209 cut, with 64 values a head 2048 over 8192 (512 items for 768 places) 167 whole,
  // 180 cut.  Several sequences: 3 x 500 queries after 1000 to 7000 keys 185 whole, 131 cut; 6 x 256 after
  // 4000 each 117 whole, 118 cut; 12 x 64 to 400 after 100 to 2000 72 whole, 78 cut.
  const int64_t with_rows = int64_t(a.total_q) * group / tile + a.batch;  // of the items, at most
  const int64_t work = (with_rows < pl.items ? with_rows : pl.items) * num_kv_heads;
  const int64_t slots = int64_t(num_sms) * dg::attn_per_cu(pl.form, head_dim);
  const bool wide = pl.form == dg::ATTN_WIDE, fills_half = 2 * work <= slots;
  const bool few = fills_half || (work < (pl.form == dg::ATTN_NARROW_32 ? 4 : 2) * slots && (wide ? a.batch > 1 && tiles >= 64 : tiles >= 128));
  pl.least_tiles = 4;
  // Short contexts of few items: eight waves instead of the second kernel, whose launch costs the host more
  // than it saves the device (1001 keys of 8 key heads: 11.6 against 9.1 us on the device, 8.5 against 12.9 on
  // the host; 2000 keys: 17.1 against 9.9).  (At 256 values a head eight waves run out of registers.)
  if (pl.form == dg::ATTN_NARROW_16 && head_dim != 256 && work <= num_sms && tiles > pl.least_tiles && tiles <= 40)
    pl.waves = 8;
  else if (few && pl.items <= (wide ? dg::MAX_SORTED : 1024) && tiles > pl.least_tiles) {
    pl.head_aim = int(slots < num_kv_heads ? 1 : slots / num_kv_heads);
    // Parts are counted to the nearest, so where there are almost as many items as places, parts of the mean size
    // would leave items half as long again whole: twice as many.  64 sequences of up to 8192 keys, 8 key heads
    // (64 items for 96 places a head) 121 -> 115 us, 90 sequences (90 for 96) 169 -> 156, 32 x 16 queries (64
    // for 64) 131 -> 106; but 20 x 16 queries (40 for 64) 73 -> 75, 32 sequences (32 for 96) 71 -> 75.
    if (!wide && 3 * (work / num_kv_heads) >= 2 * pl.head_aim) pl.head_aim *= 2;
    // One row after the other where most items may not be cut (12 x 64 to 400 queries 84 -> 78 us); where
    // few items have many parts, as many workgroups as rows give (128 queries over 8128 keys 43 us, with two
    // rows 52).
    pl.join_steps = fills_half ? 1 : 2;
    // 80 x 16 queries over 5016 keys (160 items, 128 places a head) 237 us with a workgroup for each row, 229
    // without; 32 x 4 queries, 64 values a head (32 items, 128 places) 43.6 and 40.7; but 16 single tokens (16
    // for 128) 21.4 and 23.6, 16 queries over 4016 keys (2 for 64) 18.7 and 26.6.
    pl.join_few = !wide && pl.head_aim >= 8 * (work / num_kv_heads);
    pl.max_cut = int((tiles + pl.least_tiles - 1) / pl.least_tiles);
    const int64_t by_aim = (int64_t(pl.head_aim) + pl.items) * num_kv_heads, by_cut = pl.items * num_kv_heads * pl.max_cut;
    pl.most_parts = by_aim < by_cut ? by_aim : by_cut;
  }
  return pl;
}

int64_t part_rows(const AttnPlan& pl, int32_t head_dim) { return pl.most_parts * dg::attn_tile_rows(pl.form, head_dim); }

int64_t workspace_of(const AttnPlan& pl, int32_t head_dim) {
  return pl.head_aim ? part_rows(pl, head_dim) * (head_dim + 2) * int64_t(sizeof(float)) + (pl.items + 3) / 4 * 16 : 0;
}

}  // namespace

extern "C" {

int dg_fp8_kv_cache_write(const dg_fp8_kv_cache* cache, int32_t num_tokens, const void* k, int64_t k_token_stride,
                          int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                          int32_t dtype, const int64_t* slots, hipStream_t stream) {
  return move(true, cache, num_tokens, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, dtype, slots, stream);
}

int dg_fp8_kv_cache_read(const dg_fp8_kv_cache* cache, int32_t num_tokens, void* k, int64_t k_token_stride,
                         int64_t k_head_stride, void* v, int64_t v_token_stride, int64_t v_head_stride,
                         int32_t dtype, const int64_t* slots, hipStream_t stream) {
  return move(false, cache, num_tokens, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, dtype, slots, stream);
}

int64_t dg_fp8_paged_attention_workspace(int32_t batch, int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t equal_q, int32_t max_seqlen_q, int32_t max_seqlen_k,
                                         int32_t window, int32_t sinks) {
  const AttnShape a{batch, total_q, num_q_heads, max_seqlen_q, max_seqlen_k, window, sinks, equal_q != 0};
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return api_fail(DG_ERR_UNSUPPORTED, "head_dim = %d: 64, 128 and 256 are supported", head_dim);
  if (int s = check_shape(a, num_kv_heads)) return s;
  if (batch == 0 || total_q == 0 || (!a.equal && max_seqlen_q == 0)) return 0;
  if (int s = check_items(a, num_kv_heads, head_dim)) return s;
  const int num_sms = dg::api_num_sms();
  if (num_sms <= 0) return api_fail(DG_ERR_HIP, "could not query the device's compute-unit count");
  return workspace_of(plan_of(a, num_kv_heads, head_dim, num_sms), head_dim);
}

int dg_fp8_paged_attention(const dg_fp8_kv_cache* cache, int32_t batch, int32_t total_q, int32_t num_q_heads,
                           const void* q, int64_t q_token_stride, int64_t q_head_stride,
                           const int32_t* cu_seqlens_q, int32_t max_seqlen_q,
                           const int32_t* block_table, int64_t table_stride, int32_t table_cols,
                           const int32_t* seq_lens, int32_t max_seqlen_k, float sm_scale, int32_t window, int32_t sinks,
                           void* out, int64_t o_token_stride, int64_t o_head_stride, float* lse,
                           void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const AttnShape a{batch, total_q, num_q_heads, max_seqlen_q, max_seqlen_k, window, sinks, cu_seqlens_q == nullptr};
  const bool empty = batch == 0 || total_q == 0 || (cu_seqlens_q && max_seqlen_q == 0);
  if (int s = check_cache(cache, empty)) return s;
  if (int s = check_shape(a, cache->num_heads)) return s;
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return api_fail(DG_ERR_SHAPE, "sm_scale must be positive and finite");
  // (0: one row for all sequences)
  if (table_cols < 0 || (table_stride != 0 && table_stride < table_cols))
    return api_fail(DG_ERR_LAYOUT, "table_cols = %d must not be negative, and table_stride = %lld at least as large, or 0", table_cols, (long long)table_stride);
  if (int64_t(table_cols) * cache->page_size > kMaxIndex) return api_fail(DG_ERR_SHAPE, "table_cols * page_size must be at most 2^30");
  if (empty) return api_ok();
  if (int s = check_items(a, cache->num_heads, cache->head_dim)) return s;
  if (!block_table && table_cols > 0) return api_fail(DG_ERR_NULL, "block_table must not be NULL");
  if (!seq_lens) return api_fail(DG_ERR_NULL, "seq_lens must not be NULL");
  if (int s = check_rows("q", q, q_token_stride, q_head_stride, 2)) return s;
  if (int s = check_rows("out", out, o_token_stride, o_head_stride, 2)) return s;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_seqlens_q, 4) || !aligned(lse, 4))
    return api_fail(DG_ERR_LAYOUT, "block_table, seq_lens, cu_seqlens_q and lse must be 4-byte aligned");
  const int num_sms = dg::api_num_sms();
  if (num_sms <= 0) return api_fail(DG_ERR_HIP, "could not query the device's compute-unit count");
  const AttnPlan pl = plan_of(a, cache->num_heads, cache->head_dim, num_sms);
  const int64_t need = workspace_of(pl, cache->head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return api_fail(workspace ? DG_ERR_SHAPE : DG_ERR_NULL, "this call needs a workspace of %lld bytes", (long long)need);
  if (need > 0 && !aligned(workspace, 16)) return api_fail(DG_ERR_LAYOUT, "workspace must be 16-byte aligned");

  dg::AttnParams p{};
  p.c = kernel_cache(cache);
  p.q = static_cast<const uint16_t*>(q);
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.out = static_cast<uint16_t*>(out);
  p.o_token_stride = o_token_stride;
  p.o_head_stride = o_head_stride;
  p.lse = lse;
  p.table = block_table;
  p.table_stride = table_stride;
  p.seq_lens = seq_lens;
  p.cu_q = cu_seqlens_q;
  p.table_cols = table_cols;
  p.batch = batch;
  p.total_q = total_q;
  p.q_per_seq = cu_seqlens_q ? 0 : total_q / batch;
  p.num_q_heads = num_q_heads;
  p.group = dg::fast_div(num_q_heads / cache->num_heads);
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  // (a window that holds every possible key hides nothing)
  p.window = window < int64_t(table_cols) * cache->page_size ? window : 0;
  p.sinks = p.window ? sinks : 0;
  p.q_tiles = dg::fast_div(pl.q_tiles);
  p.tile_rows = dg::attn_tile_rows(pl.form, cache->head_dim);
  p.items = int(pl.items);
  p.waves = pl.waves;
  p.head_aim = pl.head_aim;
  p.max_cut = pl.max_cut;
  p.join_rows = pl.join_rows;
  p.join_few = pl.join_few;
  p.join_steps = pl.join_steps;
  p.most_parts = int(pl.most_parts);
  p.least_tiles = pl.least_tiles;
  p.part_o = static_cast<float*>(workspace);
  p.part_mz = p.part_o + part_rows(pl, cache->head_dim) * cache->head_dim;
  p.item_end = reinterpret_cast<int32_t*>(p.part_mz + part_rows(pl, cache->head_dim) * 2);
  const hipError_t e = dg::launch_attention(p, cache->head_dim, pl.form, stream);
  if (e != hipSuccess) return api_fail(DG_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return api_ok();
}

}  // extern "C"
