// Internal interface between the host library and the kernels of the FP8 key/value cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

// Shared by the host files: record a failure (returns `code`), record success (returns DG_OK),
// and the persistent grid size in force (negative if the device cannot be queried).
int api_fail(int code, const char* fmt, ...);
int api_ok();
int api_num_sms();

// Division of 0 <= n < 2^31 by a fixed d >= 1: n / d = (n * mul) >> shr.
struct FastDiv {
  uint32_t mul;
  int32_t shr;
  int32_t d;
};
inline FastDiv fast_div(int32_t d) {
  // With l = ceil(log2 d) and mul = floor(2^(31+l) / d) + 1 the quotient's error is below n / 2^(31+l) < 1 / d.
  int l = 0;
  while ((int64_t(1) << l) < d) ++l;
  return {uint32_t((uint64_t(1) << (31 + l)) / uint32_t(d) + 1), 31 + l, d};
}
__device__ __forceinline__ int32_t div(int32_t n, const FastDiv& f) {
  return int32_t(((uint64_t)(uint32_t)n * f.mul) >> f.shr);
}

// The cache as the kernels see it: E4M3 codes [pages, heads, page size, head dim] and UE8M0 scale
// codes [pages, heads, page size], strides in bytes, the same for keys and values.
struct KvCache {
  uint8_t *k, *v, *k_sf, *v_sf;
  int64_t page_stride, head_stride, token_stride;
  int64_t sf_page_stride, sf_head_stride, sf_token_stride;
  int32_t num_pages, num_heads;
  FastDiv page;  // the page size
};

struct KvMoveParams {  // write and read
  KvCache c;
  void *k, *v;  // tokens' rows [num_tokens, heads, head dim] (write: read from; read: written to)
  int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;  // elements
  const int64_t* slots;
  int32_t num_tokens;
};
hipError_t launch_kv_write(const KvMoveParams& p, int head_dim, bool bf16, hipStream_t stream);
hipError_t launch_kv_read(const KvMoveParams& p, int head_dim, bool bf16, hipStream_t stream);

// Rows [tokens, heads, head dim], strides in elements.
struct Rows {
  void* p;
  int64_t token_stride, head_stride;
};

// Norm and rotation of queries' and keys' rows: forward (q, k -> q_out, k_out), with the keys, and the values v, going to
// the cache instead (slots), or backward (and dq, dk, the gradients of the results; q_out and k_out are those of q and k).
struct RopeParams {
  Rows q, k, v, dq, dk, q_out, k_out;
  const void *q_weight, *k_weight;  // [head dim]
  const float* cos_sin;             // [num_positions, rot]
  int64_t cos_sin_stride;
  const int64_t* positions;         // [num_tokens]
  int64_t num_positions;
  int32_t rot, num_tokens, q_heads, kv_heads;
  float eps;
  int32_t weights_bf16;
  KvCache c;
  const int64_t* slots;
  FastDiv pieces;                   // waves that share a token (forward)
  int32_t q_pieces, kv_pieces;      // those of its queries, and of its keys (forward: and as many of its values)
  float *dq_weight, *dk_weight;     // [head dim]
  float* parts;                     // [workgroups, 2, head dim] sums of the weights' gradients (workgroups > 1)
  int32_t workgroups;               // backward only
};
hipError_t launch_norm_rope(const RopeParams& p, int head_dim, bool bf16, bool interleaved, bool write, hipStream_t stream);
hipError_t launch_norm_rope_backward(const RopeParams& p, int head_dim, bool bf16, bool interleaved, hipStream_t stream);
// heads of a token that a wave takes at once
inline int rope_heads(int head_dim) { return 1024 / head_dim; }

struct AttnParams {
  KvCache c;
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;
  uint16_t* out;
  int64_t o_token_stride, o_head_stride;
  float* lse;                // nullptr, or [total_q, heads]
  const int32_t* table;      // [batch, table_cols]
  int64_t table_stride;
  const int32_t* seq_lens;   // [batch]
  const int32_t* cu_q;       // nullptr: every sequence has q_per_seq queries
  int32_t table_cols, batch, total_q, q_per_seq, num_q_heads;
  FastDiv group;             // query heads per key head
  float scale_log2;          // softmax scale * log2(e)
  int32_t window, sinks;     // window 0: none
  FastDiv q_tiles;           // tiles of query rows per sequence
  int32_t tile_rows;         // query rows (token, head of the group) of a tile
  int32_t items;             // batch * q_tiles
  int32_t waves;             // of a workgroup of the 16-row kernel: 4 or 8
  int32_t head_aim;          // cut items so that each key head has about so many parts; 0: one workgroup for each item and key head
  int32_t least_tiles;       // a part has at least so many key tiles (or all of its item's)
  int32_t max_cut;           // an item has at most so many parts
  int32_t most_parts;        // a bound of the number of parts
  int32_t join_rows;         // a bound of the rows of a tile
  int32_t join_few;          // few rows with many parts each: the join has a workgroup for each row
  int32_t join_steps;        // else: rows that a lane group of the many-rows join has one after the other
  // workspace (head_aim > 0)
  float* part_o;             // [most_parts, tile_rows, head dim] parts' unnormalised sums
  float* part_mz;            // [most_parts, tile_rows, 2] their running maximum (log2 units) and sum of weights
  int32_t* item_end;         // [items] a head's parts up to and with each item
};

// A page's block key, for each head: int8 codes [pages, heads, head dim] and a power of two [pages, heads].
struct BlockKeys {
  int8_t* codes;
  float* scales;
};

struct BlockKeysParams {
  KvCache c;  // (keys only)
  BlockKeys b;
  const int32_t* pages;
  int32_t num_pages;  // entries of `pages`
};
hipError_t launch_block_keys(const BlockKeysParams& p, int head_dim, hipStream_t stream);

// The newest tokens of sequences, as attention over chosen blocks sees them.
struct Sequences {
  const uint16_t* q;
  int64_t q_token_stride, q_head_stride;
  const int32_t* table;      // [batch, table_cols]
  int64_t table_stride;
  const int32_t* seq_lens;   // [batch]
  const int32_t* cu_q;       // nullptr: every sequence has q_per_seq queries
  int32_t table_cols, batch, total_q, q_per_seq, num_q_heads;
};

struct SelectParams {
  Sequences s;
  BlockKeys b;
  int32_t num_pages, num_heads;  // of the block keys
  FastDiv page;                  // tokens of a block
  int32_t top, first, last;
  FastDiv group;                 // query heads per key head
  FastDiv q_tiles;               // tiles of tokens per sequence
  int32_t tile_tokens, items;    // tokens of a tile; batch * q_tiles
  int32_t row_words;             // words of a token's scores
  int32_t parts;                 // workgroups that share a tile's blocks, with the scores in memory; 1: one kernel, scores in LDS
  uint32_t* scores;              // [items, heads, tile_tokens, row_words] (parts > 1)
  int32_t* out;                  // [total_q, heads, top]
};
constexpr int SELECT_WAVES = 8;  // of a workgroup
constexpr int SELECT_CANDIDATES = 512;  // a wave's room in LDS for scores that may be among the chosen
// tiles of 16 columns (a token's heads, rounded up to a power of two) of a workgroup: their codes stay in registers
constexpr int select_tiles(int head_dim) { return head_dim == 256 ? 2 : 4; }
// one_tile: a workgroup's tokens fit one tile of columns
hipError_t launch_select_blocks(const SelectParams& p, int head_dim, bool one_tile, hipStream_t stream);

struct SparseParams {
  Sequences s;
  KvCache c;
  const int32_t* blocks;     // [total_q, heads, top]
  uint16_t* out;
  int64_t o_token_stride, o_head_stride;
  float* lse;                // nullptr, or [total_q, query heads]
  float scale_log2;          // softmax scale * log2(e)
  int32_t top;
  FastDiv list;              // `top` as a divisor
  FastDiv segments;          // of 64 keys, of a block
  FastDiv group;             // query heads per key head
  FastDiv q_tiles;           // tiles of tokens per sequence
  int32_t tile_tokens, head_tiles, items;  // tokens of a tile, tiles of 16 heads of a token (one of the two is 1), batch * q_tiles
  int32_t waves;             // of a workgroup: 4 or 8
  int32_t far;               // 1: offsets into the cache may need more than 32 bits (4 waves)
  int32_t parts;             // workgroups that share a tile and key head (a power of two)
  float* part_o;             // [items, heads, head_tiles, parts, 16, head dim] (parts > 1)
  float* part_mz;            // [.., 16, 2]
};
hipError_t launch_sparse_attention(const SparseParams& p, int head_dim, hipStream_t stream);

// The kernels: four waves over the same 16 or 32 query rows, or waves of 32 rows each.
enum AttnForm { ATTN_NARROW_16 = 0, ATTN_NARROW_32 = 1, ATTN_WIDE = 2 };
// The many-rows kernel deals the pieces of up to so many items by size, and cuts items of such calls only: a
// lane holds four of them.
constexpr int MAX_SORTED = 256;
inline int attn_tile_rows(int form, int head_dim) {
  return form == ATTN_NARROW_16 ? 16 : form == ATTN_NARROW_32 ? 32 : head_dim == 128 ? 256 : 128;
}
inline int attn_tile_keys(int form, int head_dim) { return form != ATTN_WIDE || head_dim == 256 ? 32 : 64; }
// threads of a workgroup (of the 16-row kernel for more items than there are compute units)
inline int attn_threads(int form, int head_dim) { return form == ATTN_WIDE && head_dim != 64 ? 512 : 256; }
// workgroups that a compute unit holds at a time, by the registers of a lane: few rows of 16 102, 152 and 255 at head_dim
// 64, 128 and 256, of 32 136, 213 and all, many rows 162, 228 and 236 (of 512 for the waves of a SIMD)
inline int attn_per_cu(int form, int head_dim) {
  if (form == ATTN_WIDE) return head_dim == 64 ? 3 : 1;
  if (head_dim == 256) return 1;
  if (form == ATTN_NARROW_16) return head_dim == 64 ? 4 : 3;
  return head_dim == 64 ? 3 : 2;
}
hipError_t launch_attention(const AttnParams& p, int head_dim, int form, hipStream_t stream);

}  // namespace dg
