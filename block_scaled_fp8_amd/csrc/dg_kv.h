// Internal interface between the host library and the kernels of the FP8 key/value cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

// Shared by the host files: record a failure (returns `code`), record success (returns DG_OK),
// and the persistent grid size in force (0 if the device cannot be queried).
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
  int32_t q_tiles;           // tiles of query rows per (sequence, key head)
  int32_t splits;            // parts of the key range, each its own workgroup
  float* part_o;             // [splits, total_q, heads, head dim] unnormalised sums
  float* part_ml;            // [splits, total_q, heads, 2] running maximum (log2 units) and sum
};
hipError_t launch_attention(const AttnParams& p, int head_dim, bool wide, hipStream_t stream);

// Query rows (token, head of the group) of one workgroup's tile.
inline int attn_wide_rows(int head_dim) { return head_dim == 128 ? 256 : 128; }
constexpr int kAttnNarrowRows = 32;

}  // namespace dg
