// C ABI of block keys, the choice of blocks and attention over them: argument validation, the split of the work, and
// launch.  Validation runs before any HIP call.
#include <cmath>

#include "dg_api_check.h"

namespace {

using dg::aligned;
using dg::api_fail;
using dg::api_ok;
using dg::check_cache;
using dg::check_rows;
using dg::kernel_cache;
using dg::kMaxIndex;

constexpr int32_t kMaxTop = 1 << 20;
// A workgroup keeps the scores of a token's blocks in LDS (160 KiB).
constexpr int32_t kMaxColumns = 32768;

// The lists of a tile of several tokens lie in LDS: 16 KiB at most.
constexpr int64_t kMaxListed = 4096;

int check_block_keys(const dg_fp8_block_keys* b, bool empty) {
  if (!b) return api_fail(DG_ERR_NULL, "block keys must not be NULL");
  if (b->head_dim != 64 && b->head_dim != 128 && b->head_dim != 256)
    return api_fail(DG_ERR_UNSUPPORTED, "head_dim = %d: 64, 128 and 256 are supported", b->head_dim);
  if (b->num_heads <= 0 || b->num_heads > 65535) return api_fail(DG_ERR_SHAPE, "num_heads = %d must be in [1, 65535]", b->num_heads);
  if (b->num_pages < 0 || b->num_pages > kMaxIndex) return api_fail(DG_ERR_SHAPE, "num_pages = %d must be in [0, 2^30]", b->num_pages);
  if (empty) return DG_OK;
  if (b->num_pages == 0) return api_fail(DG_ERR_SHAPE, "there are no block keys");
  if (!b->codes || !b->scales) return api_fail(DG_ERR_NULL, "the block keys' codes and scales must not be NULL");
  if (!aligned(b->codes, 16) || !aligned(b->scales, 4)) return api_fail(DG_ERR_LAYOUT, "the block keys' codes must be 16-byte aligned, their scales 4-byte aligned");
  return DG_OK;
}

// The newest tokens of sequences (those of dg_fp8_paged_attention).
struct Batch {
  int32_t batch, total_q, num_q_heads, max_seqlen_q;
  bool equal;
  bool empty() const { return batch == 0 || total_q == 0 || (!equal && max_seqlen_q == 0); }
  int64_t most_tokens() const { return equal ? total_q / batch : max_seqlen_q < total_q ? max_seqlen_q : total_q; }
};

int check_batch(const Batch& a, int32_t num_kv_heads, int32_t top) {
  if (a.batch < 0 || a.total_q < 0) return api_fail(DG_ERR_SHAPE, "batch = %d and total_q = %d must not be negative", a.batch, a.total_q);
  if (num_kv_heads <= 0 || a.num_q_heads <= 0 || a.num_q_heads % num_kv_heads)
    return api_fail(DG_ERR_SHAPE, "num_q_heads = %d must be a positive multiple of the cache's %d heads", a.num_q_heads, num_kv_heads);
  if (int64_t(a.total_q) * a.num_q_heads > kMaxIndex) return api_fail(DG_ERR_SHAPE, "total_q * num_q_heads must be at most 2^30");
  if (a.max_seqlen_q < 0) return api_fail(DG_ERR_SHAPE, "max_seqlen_q = %d must not be negative", a.max_seqlen_q);
  if (a.equal && a.batch > 0 && a.total_q % a.batch) return api_fail(DG_ERR_SHAPE, "without cu_seqlens_q, total_q = %d must be a multiple of batch = %d", a.total_q, a.batch);
  if (top < 1 || top > kMaxTop) return api_fail(DG_ERR_SHAPE, "top = %d must be in [1, 2^20]", top);
  return DG_OK;
}

int check_sequences(const void* q, int64_t q_token_stride, int64_t q_head_stride, const int32_t* cu_seqlens_q, const int32_t* block_table,
                    int32_t table_cols, const int32_t* seq_lens, const int32_t* blocks) {
  if (!block_table && table_cols > 0) return api_fail(DG_ERR_NULL, "block_table must not be NULL");
  if (!seq_lens || !blocks) return api_fail(DG_ERR_NULL, "seq_lens and blocks must not be NULL");
  if (int s = check_rows("q", q, q_token_stride, q_head_stride, 2)) return s;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_seqlens_q, 4) || !aligned(blocks, 4))
    return api_fail(DG_ERR_LAYOUT, "block_table, seq_lens, cu_seqlens_q and blocks must be 4-byte aligned");
  return DG_OK;
}

int check_table(int32_t table_cols, int64_t table_stride, int32_t page_size) {
  // (0: one row for all sequences)
  if (table_cols < 0 || (table_stride != 0 && table_stride < table_cols))
    return api_fail(DG_ERR_LAYOUT, "table_cols = %d must not be negative, and table_stride = %lld at least as large, or 0", table_cols, (long long)table_stride);
  if (int64_t(table_cols) * page_size > kMaxIndex) return api_fail(DG_ERR_SHAPE, "table_cols * page_size must be at most 2^30");
  return DG_OK;
}

dg::Sequences sequences(const Batch& a, const void* q, int64_t q_token_stride, int64_t q_head_stride, const int32_t* cu_seqlens_q,
                        const int32_t* block_table, int64_t table_stride, int32_t table_cols, const int32_t* seq_lens) {
  dg::Sequences s{};
  s.q = static_cast<const uint16_t*>(q);
  s.q_token_stride = q_token_stride;
  s.q_head_stride = q_head_stride;
  s.table = block_table;
  s.table_stride = table_stride;
  s.seq_lens = seq_lens;
  s.cu_q = cu_seqlens_q;
  s.table_cols = table_cols;
  s.batch = a.batch;
  s.total_q = a.total_q;
  s.q_per_seq = cu_seqlens_q ? 0 : a.total_q / a.batch;
  s.num_q_heads = a.num_q_heads;
  return s;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A grid has less than 2^32 threads (one of more is cut to its low 32 bits without an error).
int check_grid(const Batch& a, int64_t workgroups, int threads) {
  if (workgroups > int64_t(UINT32_MAX) / threads)
    return api_fail(DG_ERR_SHAPE, "%d sequences of up to %lld tokens are more tiles than a launch holds%s", a.batch, (long long)a.most_tokens(),
                    a.equal ? "" : ": max_seqlen_q should bound the new tokens of a sequence");
  return DG_OK;
}

// Choosing: tokens of a workgroup, and workgroups that share the blocks.
struct SelectPlan {
  int64_t tile_tokens, items, row_words;
  bool one_tile;
  int parts;
};
SelectPlan select_plan(const Batch& a, int32_t num_kv_heads, int32_t head_dim, int32_t table_cols, int32_t top, int32_t first, int32_t last, int num_sms) {
  const int32_t group = a.num_q_heads / num_kv_heads;
  const int width = group > 8 ? 16 : group > 4 ? 8 : group > 2 ? 4 : group;  // columns of a token
  SelectPlan pl;
  const int64_t scored = table_cols > top ? table_cols - first - last : 1;
  pl.row_words = ceil_div(scored, 16) * 16 + 4;
  // Scores of up to 64 KiB.  Two workgroups share a compute unit's 160 KiB of LDS only where they leave room for both beside candidates and the queries'
  // codes: fewer tokens for that in sequences of eight tiles and more, whose tiles share the keys in the caches, as long as none of a tile's 16 columns
  // is empty (a chunk of 2048 over 960 blocks, 32 + 8 heads of 128: 81 us, in larger tiles 112; over 2000 blocks 210 and 229, with 64 + 8 heads 251 and
  // 318; but 32 sequences of 16 new tokens over 3600 blocks 242 and 199).  (At 256 values a head registers hold one workgroup anyway.)
  // Fewer tokens, too, where they would leave compute units without a workgroup (64 tokens over 512 blocks: 10.5 us, else 19.2; with four workgroups for
  // a unit 13.2).
  const int64_t per_tile = 16 / width, tiles = dg::select_tiles(head_dim), row = 4 * pl.row_words;
  const int64_t beside = 4 * dg::SELECT_WAVES * dg::SELECT_CANDIDATES + tiles * (16 * head_dim + 64);
  const int64_t fit = 65536 / row, fit_two = head_dim == 256 ? fit : (160 * 1024 / 2 - beside) / row;
  auto larger_than_pays = [&](int64_t tokens) {
    return tokens > fit || (tokens > fit_two && tokens > per_tile && 8 * tokens <= a.most_tokens()) || tokens >= 2 * a.most_tokens() ||
           a.batch * ceil_div(a.most_tokens(), tokens) * num_kv_heads < num_sms;
  };
  pl.tile_tokens = per_tile * tiles;
  while (pl.tile_tokens > 1 && larger_than_pays(pl.tile_tokens)) pl.tile_tokens /= 2;
  pl.items = a.batch * ceil_div(a.most_tokens(), pl.tile_tokens);
  pl.one_tile = pl.tile_tokens <= per_tile;
  pl.parts = 1;
  // Few tiles of many blocks: a workgroup for each 256 blocks (2 sequences of 2048 blocks and 4 heads: 17.2 us, in one part 23.6; 500 blocks for 8 heads,
  // which stay in one, 7.6).
  const int64_t all = pl.items * num_kv_heads;
  if (pl.one_tile && scored > 512 && 4 * all <= num_sms) {
    const int64_t by_blocks = ceil_div(scored, 256), by_units = num_sms / all;
    pl.parts = int(by_blocks < by_units ? by_blocks : by_units);
  }
  return pl;
}
int64_t select_workspace(const SelectPlan& pl, int32_t num_kv_heads) {
  return pl.parts > 1 ? pl.items * num_kv_heads * pl.tile_tokens * pl.row_words * int64_t(sizeof(uint32_t)) : 0;
}
int check_choice(int32_t top, int32_t first, int32_t last) {
  if (first < 0 || last < 1 || first > top || last > top - first)
    return api_fail(DG_ERR_SHAPE, "first = %d must not be negative, last = %d at least 1, and both together at most top = %d", first, last, top);
  return DG_OK;
}
int check_columns(int32_t table_cols) {
  if (table_cols > kMaxColumns) return api_fail(DG_ERR_UNSUPPORTED, "table_cols = %d: sequences of up to %d blocks are supported", table_cols, kMaxColumns);
  return DG_OK;
}

// Attention: tokens of a tile, and workgroups that share its keys.
struct SparsePlan {
  int64_t tile_tokens, head_tiles, items, parts;
  int waves;
};
// Segments of a list are 32-bit numbers to the kernel.
int check_lists(int32_t top, int32_t page_size) {
  if (top * ceil_div(page_size, 64) > kMaxIndex) return api_fail(DG_ERR_SHAPE, "top = %d blocks of %d tokens are more than 2^30 segments of 64", top, page_size);
  return DG_OK;
}

// Whether offsets into the cache's keys (values) or scales pass 32 bits.
bool is_far(const dg_fp8_kv_cache* c) {
  auto end = [&](int64_t page, int64_t head, int64_t token, int64_t row) {
    return double(c->num_pages - 1) * double(page) + double(c->num_heads - 1) * double(head) + double(c->page_size - 1) * double(token) + double(row);
  };
  return end(c->page_stride, c->head_stride, c->token_stride, c->head_dim) >= 4294967295.0 ||
         end(c->sf_page_stride, c->sf_head_stride, c->sf_token_stride, 1) >= 4294967295.0;
}

SparsePlan sparse_plan(const Batch& a, int32_t num_kv_heads, int32_t head_dim, int32_t page_size, int32_t top, int num_sms) {
  const int32_t group = a.num_q_heads / num_kv_heads;
  SparsePlan pl;
  pl.tile_tokens = group > 16 ? 1 : 16 / group;
  if (pl.tile_tokens > a.most_tokens()) pl.tile_tokens = a.most_tokens();
  if (pl.tile_tokens * top > kMaxListed) pl.tile_tokens = top < kMaxListed ? kMaxListed / top : 1;
  const int64_t list = top * ceil_div(page_size, 64);  // segments of a token's list: at most 2^30, as all of a tile's have to be
  if (pl.tile_tokens * list > kMaxIndex) pl.tile_tokens = kMaxIndex / list;
  pl.head_tiles = ceil_div(group, 16);
  pl.items = a.batch * ceil_div(a.most_tokens(), pl.tile_tokens);
  const int64_t with_rows = a.total_q / pl.tile_tokens + a.batch;  // of the items, at most
  const int64_t work = (with_rows < pl.items ? with_rows : pl.items) * num_kv_heads * pl.head_tiles;
  const int64_t segments = pl.tile_tokens * list, slots = num_sms;
  pl.parts = 1;
  pl.waves = 4;
  // Short lists of few tiles: eight waves instead of parts, whose second kernel costs the host more than it saves the device (one token of 8 key
  // heads over 16 blocks of 64: choice and attention 21 us a call with the host, in parts 31; on the device alone 10.3 and 9.6; over 32 blocks
  // 14.6 and 9.6).  (At 256 values a head eight waves run out of registers.)
  if (head_dim != 256 && work <= num_sms && segments > 4 && segments <= 20) {
    pl.waves = 8;
    return pl;
  }
  // Parts until there is a workgroup for each compute unit (8 sequences, 8 key heads, 64 blocks: 19.0 us, in one part 34.6; with three for a unit
  // 20.3), of eight segments at least, two for a wave (1 sequence: 9.9 us, in one part 33).
  while (pl.parts < 64 && 2 * pl.parts * work <= slots && 8 * pl.parts <= segments) pl.parts *= 2;
  return pl;
}
int64_t part_rows(const SparsePlan& pl, int32_t num_kv_heads) { return pl.items * num_kv_heads * pl.head_tiles * pl.parts * 16; }
int64_t workspace_of(const SparsePlan& pl, int32_t num_kv_heads, int32_t head_dim) {
  return pl.parts > 1 ? part_rows(pl, num_kv_heads) * (head_dim + 2) * int64_t(sizeof(float)) : 0;
}

}  // namespace

extern "C" {

int dg_fp8_kv_block_keys_update(const dg_fp8_kv_cache* cache, const dg_fp8_block_keys* keys, int32_t num_entries, const int32_t* pages,
                                hipStream_t stream) {
  if (!cache) return api_fail(DG_ERR_NULL, "cache must not be NULL");
  if (num_entries < 0 || num_entries > kMaxIndex) return api_fail(DG_ERR_SHAPE, "num_entries = %d must be in [0, 2^30]", num_entries);
  dg_fp8_kv_cache c = *cache;  // (values are not read)
  c.v = c.k;
  c.v_sf = c.k_sf;
  if (int s = check_cache(&c, num_entries == 0)) return s;
  if (int s = check_block_keys(keys, num_entries == 0)) return s;
  if (keys->num_pages != c.num_pages || keys->num_heads != c.num_heads || keys->head_dim != c.head_dim)
    return api_fail(DG_ERR_SHAPE, "block keys of %d pages, %d heads of %d do not fit the cache's %d, %d of %d", keys->num_pages, keys->num_heads,
                    keys->head_dim, c.num_pages, c.num_heads, c.head_dim);
  if (num_entries == 0) return api_ok();
  if (!pages) return api_fail(DG_ERR_NULL, "pages must not be NULL");
  if (!aligned(pages, 4)) return api_fail(DG_ERR_LAYOUT, "pages must be 4-byte aligned");
  dg::BlockKeysParams p{};
  p.c = kernel_cache(&c);
  p.b = {keys->codes, keys->scales};
  // (64 threads for a page and head; a grid has less than 2^32)
  const int32_t most = (1 << 25) / c.num_heads;
  for (int32_t from = 0; from < num_entries; from += most) {
    p.pages = pages + from;
    p.num_pages = num_entries - from < most ? num_entries - from : most;
    const hipError_t e = dg::launch_block_keys(p, c.head_dim, stream);
    if (e != hipSuccess) return api_fail(DG_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  }
  return api_ok();
}

int64_t dg_fp8_kv_select_blocks_workspace(int32_t batch, int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                          int32_t equal_q, int32_t max_seqlen_q, int32_t table_cols, int32_t top, int32_t first, int32_t last) {
  const Batch a{batch, total_q, num_q_heads, max_seqlen_q, equal_q != 0};
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return api_fail(DG_ERR_UNSUPPORTED, "head_dim = %d: 64, 128 and 256 are supported", head_dim);
  if (int s = check_batch(a, num_kv_heads, top)) return s;
  if (table_cols < 0) return api_fail(DG_ERR_LAYOUT, "table_cols = %d must not be negative", table_cols);
  if (int s = check_choice(top, first, last)) return s;
  if (int s = check_columns(table_cols)) return s;
  if (a.empty()) return 0;
  const int num_sms = dg::api_num_sms();
  if (num_sms <= 0) return api_fail(DG_ERR_HIP, "could not query the device's compute-unit count");
  return select_workspace(select_plan(a, num_kv_heads, head_dim, table_cols, top, first, last, num_sms), num_kv_heads);
}

int dg_fp8_kv_select_blocks(const dg_fp8_block_keys* keys, int32_t page_size, int32_t batch, int32_t total_q, int32_t num_q_heads,
                            const void* q, int64_t q_token_stride, int64_t q_head_stride, const int32_t* cu_seqlens_q, int32_t max_seqlen_q,
                            const int32_t* block_table, int64_t table_stride, int32_t table_cols, const int32_t* seq_lens, int32_t top,
                            int32_t first, int32_t last, int32_t* blocks, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const Batch a{batch, total_q, num_q_heads, max_seqlen_q, cu_seqlens_q == nullptr};
  if (int s = check_block_keys(keys, a.empty())) return s;
  if (int s = check_batch(a, keys->num_heads, top)) return s;
  if (page_size <= 0) return api_fail(DG_ERR_SHAPE, "page_size = %d must be positive", page_size);
  if (int s = check_choice(top, first, last)) return s;
  if (int s = check_table(table_cols, table_stride, page_size)) return s;
  if (int s = check_columns(table_cols)) return s;
  if (a.empty()) return api_ok();
  if (int s = check_sequences(q, q_token_stride, q_head_stride, cu_seqlens_q, block_table, table_cols, seq_lens, blocks)) return s;
  const int num_sms = dg::api_num_sms();
  if (num_sms <= 0) return api_fail(DG_ERR_HIP, "could not query the device's compute-unit count");
  const SelectPlan pl = select_plan(a, keys->num_heads, keys->head_dim, table_cols, top, first, last, num_sms);
  if (int s = check_grid(a, pl.items * keys->num_heads, dg::SELECT_WAVES * 64)) return s;
  const int64_t need = select_workspace(pl, keys->num_heads);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return api_fail(workspace ? DG_ERR_SHAPE : DG_ERR_NULL, "this call needs a workspace of %lld bytes", (long long)need);
  if (need > 0 && !aligned(workspace, 16)) return api_fail(DG_ERR_LAYOUT, "workspace must be 16-byte aligned");
  dg::SelectParams p{};
  p.s = sequences(a, q, q_token_stride, q_head_stride, cu_seqlens_q, block_table, table_stride, table_cols, seq_lens);
  p.b = {keys->codes, keys->scales};
  p.num_pages = keys->num_pages;
  p.num_heads = keys->num_heads;
  p.page = dg::fast_div(page_size);
  p.top = top;
  p.first = first;
  p.last = last;
  p.group = dg::fast_div(num_q_heads / keys->num_heads);
  p.q_tiles = dg::fast_div(int32_t(pl.items / batch));
  p.tile_tokens = int32_t(pl.tile_tokens);
  p.items = int32_t(pl.items);
  p.row_words = int32_t(pl.row_words);
  p.parts = pl.parts;
  p.scores = static_cast<uint32_t*>(workspace);
  p.out = blocks;
  const hipError_t e = dg::launch_select_blocks(p, keys->head_dim, pl.one_tile, stream);
  if (e != hipSuccess) return api_fail(DG_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return api_ok();
}

int64_t dg_fp8_block_sparse_attention_workspace(int32_t batch, int32_t total_q, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                                int32_t equal_q, int32_t max_seqlen_q, int32_t page_size, int32_t top) {
  const Batch a{batch, total_q, num_q_heads, max_seqlen_q, equal_q != 0};
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return api_fail(DG_ERR_UNSUPPORTED, "head_dim = %d: 64, 128 and 256 are supported", head_dim);
  if (int s = check_batch(a, num_kv_heads, top)) return s;
  if (page_size <= 0) return api_fail(DG_ERR_SHAPE, "page_size = %d must be positive", page_size);
  if (int s = check_lists(top, page_size)) return s;
  if (a.empty()) return 0;
  const int num_sms = dg::api_num_sms();
  if (num_sms <= 0) return api_fail(DG_ERR_HIP, "could not query the device's compute-unit count");
  return workspace_of(sparse_plan(a, num_kv_heads, head_dim, page_size, top, num_sms), num_kv_heads, head_dim);
}

int dg_fp8_block_sparse_attention(const dg_fp8_kv_cache* cache, int32_t batch, int32_t total_q, int32_t num_q_heads, const void* q,
                                  int64_t q_token_stride, int64_t q_head_stride, const int32_t* cu_seqlens_q, int32_t max_seqlen_q,
                                  const int32_t* block_table, int64_t table_stride, int32_t table_cols, const int32_t* seq_lens,
                                  const int32_t* blocks, int32_t top, float sm_scale, void* out, int64_t o_token_stride,
                                  int64_t o_head_stride, float* lse, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const Batch a{batch, total_q, num_q_heads, max_seqlen_q, cu_seqlens_q == nullptr};
  if (int s = check_cache(cache, a.empty())) return s;
  if (int s = check_batch(a, cache->num_heads, top)) return s;
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return api_fail(DG_ERR_SHAPE, "sm_scale must be positive and finite");
  if (int s = check_table(table_cols, table_stride, cache->page_size)) return s;
  if (int s = check_lists(top, cache->page_size)) return s;
  if (a.empty()) return api_ok();
  if (int s = check_sequences(q, q_token_stride, q_head_stride, cu_seqlens_q, block_table, table_cols, seq_lens, blocks)) return s;
  if (int s = check_rows("out", out, o_token_stride, o_head_stride, 2)) return s;
  if (!aligned(lse, 4)) return api_fail(DG_ERR_LAYOUT, "lse must be 4-byte aligned");
  const int num_sms = dg::api_num_sms();
  if (num_sms <= 0) return api_fail(DG_ERR_HIP, "could not query the device's compute-unit count");
  const SparsePlan pl = sparse_plan(a, cache->num_heads, cache->head_dim, cache->page_size, top, num_sms);
  const int64_t tiles = pl.items * cache->num_heads * pl.head_tiles;
  const bool far = is_far(cache);
  const int waves = far ? 4 : pl.waves;
  if (int s = check_grid(a, tiles * pl.parts, waves * 64)) return s;
  // (the join, which only parts have, gives each of a tile's 16 rows a workgroup)
  if (pl.parts > 1) {
    if (int s = check_grid(a, tiles * 16, 256)) return s;
  }
  const int64_t need = workspace_of(pl, cache->num_heads, cache->head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return api_fail(workspace ? DG_ERR_SHAPE : DG_ERR_NULL, "this call needs a workspace of %lld bytes", (long long)need);
  if (need > 0 && !aligned(workspace, 16)) return api_fail(DG_ERR_LAYOUT, "workspace must be 16-byte aligned");
  dg::SparseParams p{};
  p.s = sequences(a, q, q_token_stride, q_head_stride, cu_seqlens_q, block_table, table_stride, table_cols, seq_lens);
  p.c = kernel_cache(cache);
  p.blocks = blocks;
  p.out = static_cast<uint16_t*>(out);
  p.o_token_stride = o_token_stride;
  p.o_head_stride = o_head_stride;
  p.lse = lse;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.top = top;
  p.list = dg::fast_div(top);
  p.segments = dg::fast_div(int32_t(ceil_div(cache->page_size, 64)));
  p.group = dg::fast_div(num_q_heads / cache->num_heads);
  p.q_tiles = dg::fast_div(int32_t(pl.items / batch));
  p.tile_tokens = int32_t(pl.tile_tokens);
  p.head_tiles = int32_t(pl.head_tiles);
  p.items = int32_t(pl.items);
  p.far = far;
  p.waves = waves;
  p.parts = int32_t(pl.parts);
  p.part_o = static_cast<float*>(workspace);
  p.part_mz = p.part_o + (pl.parts > 1 ? part_rows(pl, cache->num_heads) * cache->head_dim : 0);
  const hipError_t e = dg::launch_sparse_attention(p, cache->head_dim, stream);
  if (e != hipSuccess) return api_fail(DG_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return api_ok();
}

}  // extern "C"
