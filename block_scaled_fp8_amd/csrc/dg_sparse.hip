// Attention of new tokens over chosen blocks (pages) of the FP8 key/value cache, for gfx950 (MI355X).
//
// For a query at place x, with the keys j <= x of the blocks in its token's and key head's list:
//   s_j = scale * q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = log sum_j exp(s_j)
// by one pass with a running maximum, the products on the BF16 matrix instruction from exactly widened codes, the
// weights rounded to BF16 (2^-8 of each at most) for the second product and their sum taken before, all sums in FP32.
//
// Every token has a list of its own, so keys cannot be shared by a large tile of queries as where all see the same.
// What can: a token's query heads, and the lists of neighbouring tokens, which overlap.  A tile is the
// rows (token, head of the group) of as many tokens as fit 16 columns of a matrix instruction; it goes over the union of its
// tokens' lists, and a column's scores count where its token's list has the block.  A block that two lists
// hold is read and widened once; one that a single list holds costs what it would alone.
//
// Lane group g (lane / 16) and column lane % 16 have the roles that they have in attention of few rows over all keys: S^T in
// blocks of 16 keys, lane group g with keys 4 g + i of its column's query.
//
// The lists' blocks, in segments of 64 keys, go 64 to a wave at a time, one a lane: a lane looks its block up in the other tokens' lists (they
// ascend), and drops it where an earlier one has it.  The remaining ones are dealt in turn to the waves of the tile's workgroups, which find
// their own without asking each other, and put them into LDS as halves of 16 keys, two of which make a wave's tile.
#include <type_traits>

#include <cfloat>

#include "dg_attn_device.h"

namespace dg {
namespace sparse {

using namespace attn;

typedef int v2i __attribute__((ext_vector_type(2)));
constexpr int SEGMENT = 64;
constexpr float MOST_BF16 = 0x1.FEp127f;

// A workgroup's tile, key head and share.
struct Tile {
  int seq, kv_head, head0;     // head0: first head of the group (groups of more than 16 heads)
  int first_row, tokens;       // packed row of the first token; tokens
  int place0, key_end;         // place of the first token; one past the last place
  int rows, part;
  int64_t slot;                // number of the tile and key head, for parts
};

// Workgroup `id` of those of a launch with so many parts; false if it has no rows.
__device__ __forceinline__ bool get_tile(const SparseParams& p, Tile& t, int id, int parts) {
  // with the key head as the fastest index, and a multiple of eight heads, those of a head land on one XCD
  t.kv_head = id % p.c.num_heads;
  id /= p.c.num_heads;
  t.part = id % parts;
  id /= parts;
  const int head_tile = id % p.head_tiles;
  id /= p.head_tiles;
  t.seq = id % p.s.batch;
  const int tile = p.q_tiles.d - 1 - id / p.s.batch;
  int n;
  if (p.s.cu_q) {
    const int a = uniform(p.s.cu_q[t.seq]), b = uniform(p.s.cu_q[t.seq + 1]);
    t.first_row = min(max(a, 0), p.s.total_q);
    n = min(max(b, t.first_row), p.s.total_q) - t.first_row;
  } else {
    t.first_row = t.seq * p.s.q_per_seq;
    n = p.s.q_per_seq;
  }
  const int t0 = tile * p.tile_tokens;
  t.tokens = min(p.tile_tokens, n - t0);
  if (t.tokens <= 0) return false;
  t.first_row += t0;
  const int ctx = min(max(uniform(p.s.seq_lens[t.seq]), 0), p.s.table_cols * p.c.page.d);
  t.place0 = ctx - n + t0;
  t.key_end = max(t.place0 + t.tokens, 0);
  t.head0 = 16 * head_tile;
  t.rows = p.head_tiles > 1 ? min(16, p.group.d - t.head0) : t.tokens * p.group.d;
  t.slot = (((int64_t)(t.seq * p.q_tiles.d + tile) * p.c.num_heads + t.kv_head) * p.head_tiles + head_tile) * p.parts;
  return true;
}

// Row r of a tile: its token's number in the tile, and its query head.
struct Row {
  int token, head;
};
__device__ __forceinline__ Row row_of(const SparseParams& p, const Tile& t, int r) {
  r = min(r, t.rows - 1);
  const int token = p.head_tiles > 1 ? 0 : div(r, p.group);
  return {token, t.kv_head * p.group.d + t.head0 + r - token * p.group.d};
}

// Whether v >= 0 is one of `top` ascending numbers (negative ones, at the end, count as larger than all).  All lanes take the same steps.
__device__ __forceinline__ bool has(const int32_t* list, int top, int v) {
  int at = 0;
  for (int n = top; n > 1;) {
    const int half = n >> 1;
    at += (uint32_t)list[at + half - 1] < (uint32_t)v ? half : 0;
    n -= half;
  }
  return list[at] == v;
}

// Up to 16 keys of one block.
template <bool FAR>
struct Half {
  using Offset = std::conditional_t<FAR, int64_t, uint32_t>;
  Offset code, sf;  // of the first one, in bytes
  int key0, keys;   // place of the first one in the sequence, and how many there are
  unsigned tokens;  // whose lists have them, by bits
};
// (FAR, with offsets of 64 bits and a descriptor for each half, takes 177 to 181 us for the chunk of 2048 tokens where the other form takes 156 on pages as far
// from each other, and 47 for 46 with 64 sequences of single tokens; so caches below 4 GiB have the other one.)
// In LDS: words of one; and how many there may be, of AT_ONCE segments, of which at most every fourth is the wave's, after one that was left, and
// with the copy that makes an odd number even.  (A segment for each lane: the chunk of 2048 tokens takes 181 us, with 32 at once 188.)
template <bool FAR>
constexpr int HALF_WORDS = FAR ? 8 : 4;
constexpr int AT_ONCE = 64, MOST_HALVES = 4 * AT_ONCE / 4 + 2;

// A wave's halves.
struct Walk {
  int share, shares;     // segments of number `share` modulo `shares` (a power of two, 4 at least) are the wave's
  int from, all, before; // next segments of lists, how many there are, and the number of those that stand before them
  int at, count;         // the halves in LDS
};

// The halves of the next AT_ONCE segments of the tile's lists, one segment a lane.  SHARED: several tokens, whose lists lie one after the other in
// LDS; else the one token's list in memory.
template <bool SHARED, bool FAR>
__device__ __forceinline__ void find_halves(const SparseParams& p, const Tile& t, const int32_t* lists, uint32_t* halves, Walk& w) {
  const int lane = threadIdx.x & 63, u = w.from + lane;
  const uint64_t below = (1ull << lane) - 1;
  unsigned tokens = 0;
  int block = 0, offset = 0;
  if (u < w.all) {
    const int i = div(u, p.segments);
    offset = (u - i * p.segments.d) * SEGMENT;
    block = lists[i];
    // (keys past the tile's last token do not count)
    if (block >= 0 && block < p.s.table_cols && block * p.c.page.d + offset < t.key_end) {
      tokens = 1u;
      if (SHARED) {
        const int mine = div(i, p.list);
        tokens = 1u << mine;
        for (int i = 1, x = mine; i < t.tokens; ++i) {
          x = x + 1 == t.tokens ? 0 : x + 1;
          if (has(lists + x * p.top, p.top, block)) tokens |= 1u << x;
        }
        if (tokens & ((1u << mine) - 1)) tokens = 0;  // (an earlier token's entry stands for it)
      }
    }
  }
  const uint64_t stand = __ballot(tokens != 0);
  const int number = w.before + (int)__popcll(stand & below);
  const bool mine = tokens != 0 && (number & (w.shares - 1)) == w.share;
  const int key0 = block * p.c.page.d + offset, keys = mine ? min(min(p.c.page.d - offset, SEGMENT), t.key_end - key0) : 0;
  const int n = (keys + 15) >> 4;  // 0 to 4
  const uint64_t b0 = __ballot(n & 1), b1 = __ballot(n & 2), b2 = __ballot(n & 4);
  if (mine) {
    const int pg = p.s.table[t.seq * p.s.table_stride + block];
    const int64_t page = (unsigned)pg < (unsigned)p.c.num_pages ? pg : 0;  // (the host cannot see the table's contents)
    const int64_t code = page * p.c.page_stride + t.kv_head * p.c.head_stride + offset * p.c.token_stride;
    const int64_t sf = page * p.c.sf_page_stride + t.kv_head * p.c.sf_head_stride + offset * p.c.sf_token_stride;
    uint32_t* to = halves + (w.count + (int)__popcll(b0 & below) + 2 * (int)__popcll(b1 & below) + 4 * (int)__popcll(b2 & below)) * HALF_WORDS<FAR>;
    for (int x = 0; x < n; ++x, to += HALF_WORDS<FAR>) {
      const int64_t c = code + 16 * x * p.c.token_stride, f = sf + 16 * x * p.c.sf_token_stride;
      *(v4u*)to = (v4u){(uint32_t)c, (uint32_t)f, (uint32_t)(key0 + 16 * x), (uint32_t)min(16, keys - 16 * x) | tokens << 16};
      if (FAR) *(v2u*)(to + 4) = (v2u){(uint32_t)(c >> 32), (uint32_t)(f >> 32)};
    }
  }
  w.count += (int)__popcll(b0) + 2 * (int)__popcll(b1) + 4 * (int)__popcll(b2);
  w.before += (int)__popcll(stand);
  w.from += AT_ONCE;
}

// The wave's next 32 keys, as two halves; the second one may be a copy of the first that no query sees.  false: there are none.
// (The wave reads what its own lanes wrote: its LDS operations complete in order, so only the compiler has to keep theirs.)
template <bool SHARED, bool FAR>
__device__ __forceinline__ bool next_tile(const SparseParams& p, const Tile& t, const int32_t* lists, uint32_t* halves, Walk& w, Half<FAR> (&h)[2]) {
  constexpr int WORDS = HALF_WORDS<FAR>;
  if (w.at + 2 > w.count) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int lane = threadIdx.x & 63;
    const bool left = w.at < w.count;
    if (left && lane < WORDS) halves[lane] = halves[w.at * WORDS + lane];
    w.at = 0;
    w.count = left ? 1 : 0;
    while (w.count < 2 && w.from < w.all) find_halves<SHARED, FAR>(p, t, lists, halves, w);
    if (w.count == 0) return false;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (w.count == 1) {
      if (lane < WORDS) halves[WORDS + lane] = lane == 3 ? halves[3] & 0xFFFFu : halves[lane];
      w.count = 2;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const uint32_t* from = halves + (w.at + x) * WORDS;
    const v4u a = *(const v4u*)from;
    const uint32_t last = (uint32_t)uniform((int)a.w);
    h[x].code = (uint32_t)uniform((int)a.x);
    h[x].sf = (uint32_t)uniform((int)a.y);
    h[x].key0 = uniform((int)a.z);
    h[x].keys = (int)(last & 0xFFFFu);
    h[x].tokens = last >> 16;
    if constexpr (FAR) {
      const v2u b = *(const v2u*)(from + 4);
      h[x].code |= (int64_t)uniform((int)b.x) << 32;
      h[x].sf |= (int64_t)uniform((int)b.y) << 32;
    }
  }
  w.at += 2;
  return true;
}

// V tiles lie in LDS as codes, rows of D bytes in 16-byte chunks.  A transposing read takes the same chunk of 32 rows, 8 to a lane group, which
// are spread over all banks.
template <int D>
__device__ __forceinline__ int v_swizzle(int row) {
  return D == 64 ? row >> 2 & 3 : D == 128 ? row >> 1 & 7 : row & 15;
}

// K tiles do too: a read takes a chunk of 16 rows in each lane group, and LDS serves 8 lanes at a time.
template <int D>
__device__ __forceinline__ int k_swizzle(int row) {
  return D == 64 ? row >> 1 & 3 : row & 7;
}

// Codes that are NaN become zeros.
__device__ __forceinline__ v4u clear_nan(v4u x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] &= ~(((((x[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu);
  return x;
}

// 16 bytes a lane from `base` + `at` + `also` to LDS, the lanes' one after the other from `dst` on; or a byte, as a word.
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t base, int at, int also, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (DG_LDS void*)dst, 16, at, also, 0, 0);
}
__device__ __forceinline__ void copy_byte_to_lds(__amdgpu_buffer_rsrc_t base, int at, int also, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (DG_LDS void*)dst, 1, at, also, 0, 0);
}

// Reads of LDS that copies have filled.  In assembly, each with its own wait: before a read that it knows to be one of LDS, the compiler
// waits for all copies that are on their way to LDS, those of the next tile too.  The caller waits for the ones it reads.
//
// Two 16-byte pieces, 256 bytes apart:
__device__ __forceinline__ void read_copied(uint32_t at, v4u& a, v4u& b) {
  asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:256\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(a), "=&v"(b)
               : "v"(at)
               : "memory");
}
// Four transposing reads: in each group of 16 lanes, lane 2 r + h names an 8-byte row (r = 0..7, h = 0..1), and lane 8 h + c gets byte c of
// the rows 0..7 of its half h.
__device__ __forceinline__ void read_transposed(const uint32_t (&at)[4], v2i (&x)[4]) {
  asm volatile("ds_read_b64_tr_b8 %0, %4\n\tds_read_b64_tr_b8 %1, %5\n\tds_read_b64_tr_b8 %2, %6\n\tds_read_b64_tr_b8 %3, %7\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
               : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
               : "memory");
}
// A lane's 16 bytes of a row of each half, OFFSET bytes apart, at each of two places.
template <int OFFSET>
__device__ __forceinline__ void read_rows(uint32_t at, v4u& a, v4u& b) {
  asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(a), "=&v"(b)
               : "v"(at), "n"(OFFSET)
               : "memory");
}
template <int OFFSET>
__device__ __forceinline__ void read_rows(uint32_t at, uint32_t at2, v4u& a, v4u& b, v4u& a2, v4u& b2) {
  asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:%6\n\tds_read_b128 %2, %5\n\tds_read_b128 %3, %5 offset:%6\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(a), "=&v"(b), "=&v"(a2), "=&v"(b2)
               : "v"(at), "v"(at2), "n"(OFFSET)
               : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(const DG_LDS uint8_t*)p; }
// Wait until at most N vector-memory operations of this wave are on their way.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt is a 6-bit field");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// What bounds it.  Chunks: the issue of instructions.  A tile of 32 keys of 128 codes takes 16 matrix instructions and 218 vector ones: 64 widen codes,
// about 100 are the rest of its turn (exponentials, their test and sum 29; the values' scales and rounding 20; hiding keys 20 to 32; addresses 20; the halves'
// numbers 8), the others find the lists' halves, raise the maximum, begin and end a wave, which has 17 tiles.  On a chunk of 2048 tokens (32 query heads, 8 key heads of
// 128, 16 of 512 blocks of 64 for each token; 175 us) the vector units are busy for 79% of the time and the matrix units for 21%.  Single tokens:
// reading (64 sequences of 64 + 8 heads, 32 blocks each: 41 us, 6.5 TB/s, some of it from the last-level cache).
//   A half holds keys of one page only, so small pages leave tiles partly empty: 64 sequences of single tokens, each over 2048 keys of random blocks, take 49
// to 50 us on pages of 16 keys and more, 60 on pages of 8, 102 of 4, 188 of 2 and 364 of 1.
//   Both K and V come through LDS, by copies of whole rows: K straight into operand registers, 16 bytes of each of 16 rows to a lane group, is an
// access to the first-level cache for every lane, 256 of the 363 that a tile had then (217 us for the chunk; through LDS 188, with 170).  A wave has room for one
// tile of each: V is on its way while K is used, and the other way round.  With 39 KB for four waves, and less than 128 registers, four
// waves share a SIMD.  (The products on the FP8 matrix instruction of 128 places, with the query in two pieces, would widen nothing, but that one adds its
// products with errors of 2^-13 of the largest, where this one has those of FP32.)
template <int D, bool SHARED, int WAVES, bool FAR>
__global__ void __launch_bounds__(WAVES * 64, D == 256 ? 2 : FAR ? 3 : 4) sparse_kernel(const SparseParams p) {
  constexpr int KEYS = 32, TILE = KEYS * D;
  constexpr int CH = D / 16, PASS = 64 / CH, NP = KEYS / PASS;  // V: 16-code chunks of a row, rows of a copy, copies
  constexpr int JD = 64;                                        // values of D joined at once
  constexpr int JOIN = WAVES * 16 * (JD + 4) * 4;
  __shared__ __attribute__((aligned(256))) uint8_t lds[WAVES * 2 * TILE > JOIN ? WAVES * 2 * TILE : JOIN];
  __shared__ __attribute__((aligned(16))) uint32_t v_scales[WAVES][2][64];  // scale codes of a half's values, 16 of them, four times
  __shared__ __attribute__((aligned(16))) uint32_t halves[WAVES][MOST_HALVES * HALF_WORDS<FAR>];
  __shared__ float mz[WAVES][2][16];
  extern __shared__ int32_t tile_lists[];  // [tile_tokens][top] (SHARED)
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), g = lane >> 4, col = lane & 15;
  uint8_t *kt = lds + wave * 2 * TILE, *v = kt + TILE;
  Tile t;
  if (!get_tile(p, t, blockIdx.x, p.parts)) return;
  const Row row = row_of(p, t, col);
  const bool live = col < t.rows;
  const int place = live ? t.place0 + row.token : INT32_MIN / 2;
  v8bf q[D / 32];
  {
    const uint16_t* src = p.s.q + (t.first_row + row.token) * p.s.q_token_stride + row.head * p.s.q_head_stride + 16 * g;
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      q[2 * x] = *(const v8bf*)(src + 64 * x);
      q[2 * x + 1] = *(const v8bf*)(src + 64 * x + 8);
    }
  }
  const int64_t list_stride = (int64_t)p.c.num_heads * p.top;
  const int32_t* lists = p.blocks + t.first_row * list_stride + (int64_t)t.kv_head * p.top;
  if (SHARED) {
    for (int i = threadIdx.x; i < t.tokens * p.top; i += WAVES * 64) {
      const int x = div(i, p.list);
      tile_lists[i] = lists[x * list_stride + i - x * p.top];
    }
    __syncthreads();
    lists = tile_lists;
  }
  const unsigned every = (1u << t.tokens) - 1;
  Walk w;
  w.shares = WAVES * p.parts;
  w.share = t.part * WAVES + wave;
  w.all = t.tokens * p.top * p.segments.d;

  // whether every row sees all 16 keys of a half or none
  auto is_sharp = [&](const Half<FAR> (&h)[2]) { return h[0].keys == 16 && h[1].keys == 16 && h[0].key0 + 15 <= t.place0 && h[1].key0 + 15 <= t.place0; };

  // whether every row sees all 32 keys
  auto is_whole = [&](const Half<FAR> (&h)[2]) {
    return h[0].tokens == every && h[1].tokens == every && is_sharp(h);
  };

  // Codes go through buffer descriptors of the pages, whose addresses are scalar; lane
  // l % 32 has the scale code of key l % 32.
  uint8_t ks[2];  // (bytes until they are used: wider, they would be widened, and so waited for, where they are loaded)
  // Everything goes through buffer descriptors of the cache, with the half's offset in a scalar register.  (FAR, for caches of 4 GiB and more:
  // descriptors of the half.)  Rows past a half's keys give bytes of its last one; `some` false: all those of its first one.  (The loads are issued
  // all the same, so that as many are on their way in each turn.)
  const int ts = (int)p.c.token_stride, sts = (int)p.c.sf_token_stride;
  const int sf_row = col * sts, v_row = lane / CH;
  auto from = [&](const uint8_t* base, typename Half<FAR>::Offset at) { return rsrc(FAR ? base + at : base, -1); };
  auto also = [&](typename Half<FAR>::Offset at) { return FAR ? 0 : (int)at; };
  auto copy_k = [&](const Half<FAR> (&h)[2], bool some) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int last = some ? h[x].keys - 1 : 0;
      const __amdgpu_buffer_rsrc_t codes = from(p.c.k, h[x].code);
#pragma unroll
      for (int n = x * NP / 2; n < (x + 1) * NP / 2; ++n) {
        const int r = n * PASS + v_row;
        copy_to_lds(codes, min((r & 15) * ts + 16 * (lane % CH ^ k_swizzle<D>(r)), last * ts + D - 16), also(h[x].code), kt + n * 1024);
      }
      ks[x] = __builtin_amdgcn_raw_buffer_load_b8(from(p.c.k_sf, h[x].sf), min(sf_row, last * sts), also(h[x].sf), 0);
    }
  };
  auto copy_v = [&](const Half<FAR> (&h)[2], bool some) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int last = some ? h[x].keys - 1 : 0;
      const __amdgpu_buffer_rsrc_t codes = from(p.c.v, h[x].code);
#pragma unroll
      for (int n = x * NP / 2; n < (x + 1) * NP / 2; ++n) {
        const int r = n * PASS + v_row;
        copy_to_lds(codes, min((r & 15) * ts + 16 * (lane % CH ^ v_swizzle<D>(r)), last * ts + D - 16), also(h[x].code), v + n * 1024);
      }
      copy_byte_to_lds(from(p.c.v_sf, h[x].sf), min(sf_row, last * sts), also(h[x].sf), v_scales[wave][x]);
    }
  };

  v4f o[D / 16];
  float m, z, shift;
  // A hidden value's weight is zero, which is not enough where it is NaN (or its scale so large that weights overflow).  Nobody looks for such
  // values at first: they leave a NaN in some output.  A wave that ends with an output that is no number goes over its keys again with care: NaN among
  // the values of tiles that some row does not see in whole go to the outputs of the rows that see them, and become zeros; no weight is infinite.
#pragma unroll 1
  for (int careful = 0;; ++careful) {
    m = NEG_INF, z = 0.f, shift = FLT_MAX;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[d] = (v4f){0.f, 0.f, 0.f, 0.f};
    w.from = w.before = w.at = w.count = 0;
    // A turn takes K of a tile from LDS and issues K of the next one, takes V and issues V of the next one: what it waits for was issued half a
    // turn and more before, and the other one is on its way meanwhile.
    Half<FAR> now[2], next[2];
    bool more = next_tile<SHARED, FAR>(p, t, lists, halves[wave], w, now);
    if (more) {
      copy_k(now, true);
      __builtin_amdgcn_sched_barrier(0);
      copy_v(now, true);
      next[0] = now[0], next[1] = now[1];
    }
#pragma unroll 1
    while (more) {
      more = next_tile<SHARED, FAR>(p, t, lists, halves[wave], w, next);  // (without more, `next` is still the last tile)
      __builtin_amdgcn_sched_barrier(0);
      wait_vm<NP + 2>();  // only V may be on its way
      v4u kr[2][D / 64];
      uint32_t k_at = lds_address(kt) + col * D + 16 * (g ^ k_swizzle<D>(col));
      if constexpr (D == 64) {
        read_rows<16 * D>(k_at, kr[0][0], kr[1][0]);
      } else {
#pragma unroll
        for (int y = 0; y < D / 64; y += 2) read_rows<16 * D>(k_at ^ 64 * y, k_at ^ 64 * (y + 1), kr[0][y], kr[1][y], kr[0][y + 1], kr[1][y + 1]);
      }
      const float k_scale[2] = {__uint_as_float((uint32_t)ks[0] << 23), __uint_as_float((uint32_t)ks[1] << 23)};
      __builtin_amdgcn_sched_barrier(0);
      copy_k(next, more);
      __builtin_amdgcn_sched_barrier(0);
      v4f s[2];
      s[0] = s[1] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int y = 0; y < D / 64; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const v8bf lo = __builtin_bit_cast(v8bf, widen8(kr[x][y].x, kr[x][y].y, k_scale[x]));
          const v8bf hi = __builtin_bit_cast(v8bf, widen8(kr[x][y].z, kr[x][y].w, k_scale[x]));
          s[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, q[2 * y], s[x], 0, 0, 0);
          s[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, q[2 * y + 1], s[x], 0, 0, 0);
        }
      __builtin_amdgcn_sched_barrier(0);
      float sub[2] = {shift, shift};
      if (!is_whole(now)) {
        // keys of each half that the lane's query sees: the first ones
        int count[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) count[x] = now[x].tokens >> row.token & 1 ? min(now[x].keys, place - now[x].key0 + 1) : 0;
        // A query that sees all of a half or nothing: -inf for all its keys at once.
        if (is_sharp(now) && !careful) {
#pragma unroll
          for (int x = 0; x < 2; ++x) sub[x] = count[x] > 0 ? shift : NEG_INF;
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[x][e] = e < count[x] - 4 * g ? s[x][e] : NEG_INF;
        }
        if (__builtin_expect(careful, 0)) {
          wait_vm<NP + 2>();
          int l = lane;
          asm volatile("" : "+v"(l));  // (so that no register holds what is computed from it through the loop)
#pragma unroll 1
          for (int j = 0; j < KEYS; ++j)
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              const uint32_t four = *(const uint32_t*)(v + j * D + 16 * (d ^ v_swizzle<D>(j)) + 4 * (l >> 4));
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((j & 15) < (j < 16 ? count[0] : count[1]) && (four >> 8 * e & 0x7F) == 0x7F) o[d][e] = __builtin_nanf("");
            }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
          for (int n = 0; n < NP; ++n) {
            v4u* at = (v4u*)(v + n * 1024 + l * 16);
            *at = clear_nan(*at);
          }
        }
      }
      // Exponents against the row's largest score so far; only one that passes it by more than SLACK (compared as integers, which hold for what
      // is positive) raises it.  A row without a score has the largest number for a shift, so that its first one does.
      v4f w2[2];
      int most = 0;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w2[x][e] = __builtin_fmaf(s[x][e], p.scale_log2, sub[x]);
          most = max(most, (int)__float_as_uint(w2[x][e]));
        }
      if (__any(most > (int)__float_as_uint(SLACK))) {
        float top = NEG_INF;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, sub[x] == NEG_INF ? NEG_INF : s[x][e]);
        const float raised = fmaxf(m, groups_max(top) * p.scale_log2);  // (the scale is positive)
        const float f = raised == NEG_INF ? 1.f : exp2_hw(m - raised);
        m = raised;
        shift = m == NEG_INF ? FLT_MAX : -m;
        if (__any(z != 0.f)) {  // (else nothing has been summed)
          z *= f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) o[d] *= f;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) w2[x][e] = __builtin_fmaf(s[x][e], p.scale_log2, sub[x] == NEG_INF ? NEG_INF : shift);
      }
      // (the wave reads what its other lanes wrote: its LDS operations complete in order, so only the compiler has to keep theirs)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      v4u x4, sf[2];
      wait_vm<NP + 2>();  // only K of the next tile may be on its way
      read_copied(lds_address(&v_scales[wave][0][4 * g]), sf[0], sf[1]);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[x][e] = exp2_hw(w2[x][e]);
          z += s[x][e];
        }
      // The value's scale goes to its weight: exact, so the weight is rounded to BF16 as it would be without.
      if (__builtin_expect(careful, 0)) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float scaled = s[x][e] * __uint_as_float(sf[x][e] << 23);  // (a hidden place may hold any scale)
            s[x][e] = s[x][e] == 0.f ? 0.f : scaled > MOST_BF16 ? MOST_BF16 : scaled;
          }
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][e] *= __uint_as_float(sf[x][e] << 23);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        x4[2 * x] = pack2(s[x][0], s[x][1]);
        x4[2 * x + 1] = pack2(s[x][2], s[x][3]);
      }
      const v8bf wt = __builtin_bit_cast(v8bf, x4);
      // a transposing read takes a row of each of 8 keys in 2 lanes: those of the group's weights, 4 g.. and 16 + 4 g..
      const int rr = col >> 1, key = rr < 4 ? 4 * g + rr : 12 + 4 * g + rr;
      uint32_t at = lds_address(v) + key * D + 16 * v_swizzle<D>(key) + 8 * (lane & 1);
      asm volatile("" : "+v"(at));  // (or D / 16 addresses would be held through the loop)
#pragma unroll
      for (int d0 = 0; d0 < D / 16; d0 += 4) {
        v2i c[4];
        const uint32_t from[4] = {at ^ 16 * d0, at ^ 16 * (d0 + 1), at ^ 16 * (d0 + 2), at ^ 16 * (d0 + 3)};
        read_transposed(from, c);
#pragma unroll
        for (int d = 0; d < 4; ++d)
          o[d0 + d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, widen8((unsigned)c[d].x, (unsigned)c[d].y, 1.f)), wt, o[d0 + d], 0, 0, 0);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_sched_barrier(0);
      copy_v(next, more);
      __builtin_amdgcn_sched_barrier(0);
      now[0] = next[0], now[1] = next[1];
    }
    wait_vm<0>();  // (or a copy would still go to LDS that others write)
    if (careful) break;
    float sum = 0.f;  // (a NaN or infinity times zero is NaN)
#pragma unroll
    for (int d = 0; d < D / 16; ++d) sum += (o[d].x * 0.f + o[d].y * 0.f) + (o[d].z * 0.f + o[d].w * 0.f);
    if (__builtin_expect(!__any(sum != 0.f), 1)) break;
  }

  // join the waves: rescale to the common maximum and add up through LDS, JD values of D at a time
  z = groups_sum(z);
  if (g == 0) {
    mz[wave][0][col] = m;
    mz[wave][1][col] = z;
  }
  __syncthreads();
  float all = NEG_INF;
#pragma unroll
  for (int x = 0; x < WAVES; ++x) all = fmaxf(all, mz[x][0][col]);
  const float f = all == NEG_INF ? 1.f : exp2_hw(m - all);
  float* jo = (float*)lds;
  // this thread adds up row jr, values jd.. of JD
  const int jr = threadIdx.x >> 4, jd = 4 * (threadIdx.x & 15);
  const Row out = row_of(p, t, jr);
#pragma unroll
  for (int d0 = 0; d0 < D; d0 += JD) {
    if (d0) __syncthreads();
#pragma unroll
    for (int d = 0; d < JD / 16; ++d) *(v4f*)(jo + (wave * 16 + col) * (JD + 4) + 16 * d + 4 * g) = o[d0 / 16 + d] * f;
    __syncthreads();
    if (jr >= t.rows) continue;
    float top = NEG_INF, sum = 0.f;
#pragma unroll
    for (int x = 0; x < WAVES; ++x) top = fmaxf(top, mz[x][0][jr]);
#pragma unroll
    for (int x = 0; x < WAVES; ++x) sum += (top == NEG_INF ? 1.f : exp2_hw(mz[x][0][jr] - top)) * mz[x][1][jr];
    v4f a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < WAVES; ++x) a += *(const v4f*)(jo + (x * 16 + jr) * (JD + 4) + jd);
    if (p.parts == 1) {
      a *= inverse(sum);
      const int64_t token = t.first_row + out.token;
      *(v2u*)(p.out + token * p.o_token_stride + out.head * p.o_head_stride + d0 + jd) = (v2u){pack2(a.x, a.y), pack2(a.z, a.w)};
      if (p.lse && d0 == 0 && jd == 0) p.lse[token * p.s.num_q_heads + out.head] = log_sum(top, sum);
    } else {
      const int64_t at = (t.slot + t.part) * 16 + jr;
      *(v4f*)(p.part_o + at * D + d0 + jd) = a;
      if (d0 == 0 && jd == 0) *(v2f*)(p.part_mz + 2 * at) = (v2f){top, sum};
    }
  }
}

// out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) z_s over the parts s of a row.  A workgroup has one row: D / 4 lanes for a part, groups of
// lanes take the parts in turn, and their sums are added in their order.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const SparseParams p) {
  constexpr int L = D / 4, G = 256 / L;
  __shared__ __attribute__((aligned(16))) float sums[G][L][4];
  __shared__ float tops[G][2];
  Tile t;
  if (!get_tile(p, t, blockIdx.x >> 4, 1)) return;
  const int r = blockIdx.x & 15, lanes = threadIdx.x % L, group = threadIdx.x / L;
  if (r >= t.rows) return;
  const Row row = row_of(p, t, r);
  float m = NEG_INF, z = 0.f;
  v4f o = {0.f, 0.f, 0.f, 0.f};
  constexpr int TOGETHER = 4;  // loads that go out together
  for (int x = group; x < p.parts; x += G * TOGETHER) {
    v2f a[TOGETHER];
    v4f b[TOGETHER];
#pragma unroll
    for (int u = 0; u < TOGETHER; ++u) {
      a[u] = (v2f){NEG_INF, 0.f};
      if (x + u * G < p.parts) {
        const int64_t at = (t.slot + x + u * G) * 16 + r;
        a[u] = *(const v2f*)(p.part_mz + 2 * at);
        b[u] = *(const v4f*)(p.part_o + at * D + 4 * lanes);
      }
    }
#pragma unroll
    for (int u = 0; u < TOGETHER; ++u) {
      // no part, or one in which the row sees nothing (one whose scores are all NaN has no maximum either, but a NaN for its
      // sum, which stays)
      if (a[u].x == NEG_INF && a[u].y == 0.f) continue;
      const float top = fmaxf(m, a[u].x), f = exp2_hw(m - top), h = exp2_hw(a[u].x - top);
      z = z * f + a[u].y * h;
      o = o * f + b[u] * h;
      m = top;
    }
  }
  *(v4f*)sums[group][lanes] = o;
  if (lanes == 0) tops[group][0] = m, tops[group][1] = z;
  __syncthreads();
  if (group != 0) return;
#pragma unroll
  for (int x = 0; x < G; ++x) m = fmaxf(m, tops[x][0]);
  z = 0.f;
  o = 0.f;
#pragma unroll
  for (int x = 0; x < G; ++x) {
    // (a group without parts, or with NaN for its sum)
    const float f = tops[x][0] == NEG_INF ? 1.f : exp2_hw(tops[x][0] - m);
    z += f * tops[x][1];
    o += f * *(const v4f*)sums[x][lanes];
  }
  o *= inverse(z);
  const int64_t token = t.first_row + row.token;
  *(v2u*)(p.out + token * p.o_token_stride + row.head * p.o_head_stride + 4 * lanes) = (v2u){pack2(o.x, o.y), pack2(o.z, o.w)};
  if (p.lse && lanes == 0) p.lse[token * p.s.num_q_heads + row.head] = log_sum(m, z);
}

template <int D>
hipError_t launch(const SparseParams& p, hipStream_t stream) {
  const unsigned tiles = (unsigned)((int64_t)p.items * p.c.num_heads * p.head_tiles);
  const size_t lists = (size_t)p.tile_tokens * p.top * 4;
  const dim3 grid(tiles * p.parts), threads(p.waves * 64);
  const bool shared = p.tile_tokens > 1;
  if (p.far) {
    if (shared)
      hipLaunchKernelGGL((sparse_kernel<D, true, 4, true>), grid, threads, lists, stream, p);
    else
      hipLaunchKernelGGL((sparse_kernel<D, false, 4, true>), grid, threads, 0, stream, p);
  } else if (p.waves == 4) {
    if (shared)
      hipLaunchKernelGGL((sparse_kernel<D, true, 4, false>), grid, threads, lists, stream, p);
    else
      hipLaunchKernelGGL((sparse_kernel<D, false, 4, false>), grid, threads, 0, stream, p);
  } else if constexpr (D != 256) {
    if (shared)
      hipLaunchKernelGGL((sparse_kernel<D, true, 8, false>), grid, threads, lists, stream, p);
    else
      hipLaunchKernelGGL((sparse_kernel<D, false, 8, false>), grid, threads, 0, stream, p);
  } else {
    return hipErrorInvalidValue;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.parts == 1) return e;
  hipLaunchKernelGGL((join_kernel<D>), dim3(tiles * 16), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace sparse

hipError_t launch_sparse_attention(const SparseParams& p, int head_dim, hipStream_t stream) {
  if (head_dim == 64) return sparse::launch<64>(p, stream);
  if (head_dim == 128) return sparse::launch<128>(p, stream);
  if (head_dim == 256) return sparse::launch<256>(p, stream);
  return hipErrorInvalidValue;
}

}  // namespace dg
