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
