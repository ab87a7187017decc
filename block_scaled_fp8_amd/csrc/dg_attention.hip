// Attention of new tokens over a paged FP8 key/value cache, for gfx950 (MI355X).
//
// For a query at place x of its sequence, with the keys j it sees (j <= x and, with a window W,
// j > x - W or j < sinks):
//   s_j = scale * q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = log sum_j exp(s_j)
// in one pass over the keys: m the running maximum of c * s (c = log2 e), z = sum 2^(c s_j - m),
// o = sum 2^(c s_j - m) v_j, all in FP32.  A query that sees no key gives zeros and lse -inf.
//
// The products run on the BF16 matrix instruction: an E4M3 code times its power-of-two scale is a
// BF16 number, so widening the cache (one conversion for two values, scale included) is exact, and
// the scales cost no arithmetic on the scores.  The weights 2^(c s - m) are rounded to BF16 for the
// second product (2^-8 relative at most, independent of m); their sum z is taken before that.
//
// Orientation: S^T = K Q^T, then O^T = V^T P^T.  A lane then owns one query (lane % 32) in both
// products: its scores, maximum, sum and outputs are its own up to one exchange between the two
// half waves, and the accumulator layout of S^T is the operand layout of P^T as long as keys are
// numbered alike in V^T: in a step of 16 keys, half wave h holds keys 4h..4h+3 and 8+4h..8+4h+3,
// and two transposing LDS reads fetch exactly those four and four keys of a V column.
//
// Query heads that share a key head are rows of the same tile: row r is query r / group, head
// r % group of the group.
#include "dg_kv.h"

namespace dg {
namespace attn {

#define DG_LDS __attribute__((address_space(3)))

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

template <int N>
struct Int {
  static constexpr int value = N;
};

constexpr float NEG_INF = -__builtin_inff();
constexpr int ROWS = 32;  // query rows of one wave: the columns of its matrix instructions
// The running maximum is raised only when a score passes it by this much (log2 units): until then
// weights stay below 2^8, which neither FP32 sums nor BF16's relative rounding notice.
constexpr float SLACK = 8.f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ unsigned pack2(float x, float y) {
  return __builtin_bit_cast(unsigned, (v2bf){(__bf16)x, (__bf16)y});
}

// Maximum and sum over the two half waves, which hold different keys of the same query.
__device__ __forceinline__ float both_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 8 codes (one row, so one scale) to 8 BF16.
__device__ __forceinline__ v4u widen8(unsigned lo, unsigned hi, float s) {
  v4u r;
  r.x = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false));
  r.y = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true));
  r.z = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false));
  r.w = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true));
  return r;
}

// LDS tiles hold BF16 rows of D values (2 D bytes) in 16-byte chunks, permuted within a row so
// that the reads below hit all banks.  K: 16 lanes read one chunk of 16 consecutive rows.  V: 16
// lanes read 4 rows x 32 bytes, and the next 16 lanes the 32 bytes beside them; the lowest bit
// keeps neighbouring rows' writes apart (a lane writes its two chunks of a row one after the other).
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
  return c ^ (D == 64 ? (row >> 1) & 7 : row & 15);
}
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
  return c ^ (D == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2) ^ (row & 1);
}

// An item: a tile of query rows of one sequence (and, for each key head, the tiles of keys that these
// rows see).
struct Work {
  int seq, kv_head;
  int q_first;           // first packed query row (token) of the sequence
  int row0, rows;        // first row of the tile; rows of the sequence in all
  int place0;            // place of the sequence's first query (negative where queries exceed the context)
  int key_end;           // one past the last key that some row of the tile sees
  int key_from;          // first key of the window of the tile's first query
  int sink_tiles, first_tile, tiles;
  int t0, t1;            // key tiles [t0, t1) of this piece of work, as list indices
  int slot;              // where a part of an item goes; -1 for a whole item

  __device__ __forceinline__ int tile_key(int i, int keys) const { return (i < sink_tiles ? i : first_tile + i - sink_tiles) * keys; }
};

// A value that is the same for all lanes, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32 | (uint32_t)uniform((int)x));
}

// The same for a piece of work: its fields come through branches that the compiler cannot tell are taken by
// all lanes, and the addresses of every tile hang on them.
__device__ __forceinline__ void make_uniform(Work& w) {
  w.seq = uniform(w.seq), w.kv_head = uniform(w.kv_head), w.q_first = uniform(w.q_first);
  w.row0 = uniform(w.row0), w.rows = uniform(w.rows), w.place0 = uniform(w.place0);
  w.key_end = uniform(w.key_end), w.key_from = uniform(w.key_from);
  w.sink_tiles = uniform(w.sink_tiles), w.first_tile = uniform(w.first_tile), w.tiles = uniform(w.tiles);
  w.t0 = uniform(w.t0), w.t1 = uniform(w.t1), w.slot = uniform(w.slot);
}

// The item's rows.  SAME: the item is the same for all lanes.  Returns the sequence's queries.
template <bool SAME>
__device__ __forceinline__ int item_rows(const AttnParams& p, int item, Work& w) {
  w.seq = p.q_tiles.d == 1 ? item : div(item, p.q_tiles);
  int n;
  if (p.cu_q) {
    int a = p.cu_q[w.seq], b = p.cu_q[w.seq + 1];
    if (SAME) a = uniform(a), b = uniform(b);
    w.q_first = min(max(a, 0), p.total_q);
    n = min(max(b, w.q_first), p.total_q) - w.q_first;
  } else {
    w.q_first = w.seq * p.q_per_seq;
    n = p.q_per_seq;
  }
  w.rows = n * p.group.d;
  w.row0 = (item - w.seq * p.q_tiles.d) * p.tile_rows;
  return n;
}

// And the keys they see, in tiles of KEYS.  Returns the item's weight: its key tiles, one where its rows see no
// key (they are still to be written), 0 without rows.
template <int KEYS, bool SAME>
__device__ __forceinline__ int describe(const AttnParams& p, int item, Work& w) {
  const int n = item_rows<SAME>(p, item, w);
  int ctx = p.seq_lens[w.seq];
  if (SAME) ctx = uniform(ctx);
  ctx = min(max(ctx, 0), p.table_cols * p.c.page.d);
  w.place0 = ctx - n;
  const int first = w.place0 + div(w.row0, p.group);
  const int last = w.place0 + div(max(min(w.row0 + p.tile_rows, w.rows) - 1, 0), p.group);
  w.key_end = max(last + 1, 0);
  w.key_from = p.window ? max(first - p.window + 1, 0) : 0;
  w.first_tile = w.key_from / KEYS;
  w.sink_tiles = min((min(p.sinks, w.key_end) + KEYS - 1) / KEYS, w.first_tile);
  w.tiles = w.key_end > 0 ? w.sink_tiles + (w.key_end + KEYS - 1) / KEYS - w.first_tile : 0;
  return w.row0 < w.rows ? max(w.tiles, 1) : 0;
}

// Lane l's item for the whole wave.
__device__ __forceinline__ void take_from_lane(Work& w, int l) {
  w.seq = __builtin_amdgcn_readlane(w.seq, l);
  w.q_first = __builtin_amdgcn_readlane(w.q_first, l);
  w.row0 = __builtin_amdgcn_readlane(w.row0, l);
  w.rows = __builtin_amdgcn_readlane(w.rows, l);
  w.place0 = __builtin_amdgcn_readlane(w.place0, l);
  w.key_end = __builtin_amdgcn_readlane(w.key_end, l);
  w.key_from = __builtin_amdgcn_readlane(w.key_from, l);
  w.first_tile = __builtin_amdgcn_readlane(w.first_tile, l);
  w.sink_tiles = __builtin_amdgcn_readlane(w.sink_tiles, l);
  w.tiles = __builtin_amdgcn_readlane(w.tiles, l);
}

// Sum over the lanes up to and with one's own.
__device__ __forceinline__ int scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // from 1, 2, 4, 8 lanes before, in rows of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // the last lane of row 0 (2) into row 1 (3)
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 into rows 2 and 3
  return x;
}

// The largest of the lanes' values, none negative.
__device__ __forceinline__ int most(int x) {
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(x, 63);
}

// How the work is dealt where items are cut: into parts of about as many key tiles, a number that follows
// from the lengths, and so is known to the device only.  A head's parts are numbered item after item, and
// heads follow each other.  A part of an item that is not cut writes the item; else it leaves its sums
// in the slot of its number, and join_kernel adds them up.
//
// With t_i the items' weights (up to 2^20: 1024 items' sum stays a 32-bit number), T their sum and
// n = head_aim, an item is cut into t_i / s parts, to the nearest, with s = max(least_tiles, ceil(T / n)), raised to a
// multiple of four (the few-rows kernel's waves), so there are at most n + items of them.
// The host's bound of the lengths, which may be wrong, enters as max_cut, the most parts of an item, alone.
//
// The many-rows kernel's workgroups take the pieces largest first, whole items of several sequences
// too: the chunks of 5 sequences, 1 to 1537 queries after 0 to 4001 keys, 159 us (183 in order of rows); 4
// sequences, 1 to 900 queries after 0 to 4000 keys, cut, 80 us (91 in order of parts; 112 whole).  Each finds
// its piece by itself, in 1 to 2 us.  One sequence's whole items are in order as they are.
struct Cut {
  unsigned size, max_cut;
  __device__ __forceinline__ int parts(int weight) const { return weight ? (int)min(max(((unsigned)weight + size / 2) / size, 1u), max_cut) : 0; }
};

__device__ __forceinline__ Cut cut_for(const AttnParams& p, int per_head) {
  return {(max((unsigned)p.least_tiles, ((unsigned)per_head + p.head_aim - 1) / (unsigned)p.head_aim) + 3) & ~3u, (unsigned)p.max_cut};
}

// Part x of n: as many key tiles as the others, or one more.
__device__ __forceinline__ void take_part(Work& w, int x, int n) {
  const int share = uniform((int)((unsigned)w.tiles / (unsigned)n)), more = w.tiles - share * n;
  w.t0 = x * share + min(x, more);
  w.t1 = w.t0 + share + (x < more ? 1 : 0);
}

// Piece number `rank` of a key head's, the largest first and equals in their order; false past the last.  For
// up to MAX_SORTED items, 64 to a register.
template <int KEYS>
__device__ __forceinline__ bool piece_by_size(const AttnParams& p, int kv_head, int rank, Work& w) {
  constexpr int MOST = MAX_SORTED / 64;
  const int lane = threadIdx.x & 63;
  int parts[MOST], size[MOST], ends[MOST];  // (parts: weights at first)
  int per_head = 0, all = 0, largest = 0;
  Work other;
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    parts[k] = 0;
    if (64 * k + lane < p.items) parts[k] = min(describe<KEYS, false>(p, 64 * k + lane, k ? other : w), 1 << 20);
    per_head += parts[k];
  }
  Cut cut{1, 1};
  if (p.head_aim) cut = cut_for(p, __builtin_amdgcn_readlane(scan(per_head), 63));
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    size[k] = parts[k];
    if (64 * k >= p.items) continue;
    parts[k] = cut.parts(size[k]);
    if (p.head_aim) {
      if (size[k]) size[k] = (size[k] + parts[k] - 1) / (unsigned)parts[k];
      ends[k] = all + scan(parts[k]);
      all = __builtin_amdgcn_readlane(ends[k], 63);
      if (blockIdx.x == 0 && threadIdx.x < 64 && 64 * k + lane < p.items) p.item_end[64 * k + lane] = ends[k];
    }
    largest = max(largest, size[k]);
  }
  auto count = [&](auto among) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < MOST; ++k) n += among(size[k]) ? parts[k] : 0;
    return __builtin_amdgcn_readlane(scan(n), 63);
  };
  // the largest threshold that more than `rank` pieces reach, bit by bit
  int t = 0;
  for (int bit = 1 << (31 - __builtin_clz(most(largest) | 1)); bit; bit >>= 1)
    if (count([&](int x) { return x >= (t | bit); }) > rank) t |= bit;
  if (t == 0) return false;
  rank -= count([&](int x) { return x > t; });
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    if (64 * k >= p.items) return false;
    const int x = scan(size[k] == t ? parts[k] : 0);
    const uint64_t later = __ballot(x > rank);
    if (later) {
      const int l = __builtin_ctzll(later), n = __builtin_amdgcn_readlane(parts[k], l);
      const int part = rank - (__builtin_amdgcn_readlane(x, l) - n);
      if (k == 0)
        take_from_lane(w, l);
      else
        describe<KEYS, true>(p, 64 * k + l, w);
      take_part(w, part, n);
      w.slot = n == 1 ? -1 : kv_head * all + __builtin_amdgcn_readlane(ends[k], l) - n + part;
      return true;
    }
    rank -= __builtin_amdgcn_readlane(x, 63);
  }
  return false;
}

// The workgroup's piece of work; false if there is none.
template <int KEYS, bool WIDE>
__device__ __forceinline__ bool get_work(const AttnParams& p, Work& w) {
  if (WIDE || p.head_aim == 0) {
    // Workgroups are dealt to the eight XCDs in turn: with the key head as the fastest index, and a multiple
    // of eight heads, those of a (sequence, key head) pair land on one XCD and share its L2.
    const int kv_head = blockIdx.x % p.c.num_heads, rank = blockIdx.x / p.c.num_heads;
    w.kv_head = kv_head;
    if (WIDE && p.items <= MAX_SORTED && (p.batch > 1 || p.head_aim)) return piece_by_size<KEYS>(p, kv_head, rank, w);
    // a sequence's later rows, which see more keys, first
    const int seq = rank % p.batch, item = seq * p.q_tiles.d + p.q_tiles.d - 1 - rank / p.batch;
    if (!describe<KEYS, true>(p, item, w)) return false;
    w.t0 = 0;
    w.t1 = w.tiles;
    w.slot = -1;
    return true;
  }
  const int lane = threadIdx.x & 63;
  auto weight = [&](int item, Work& x) { return item < p.items ? min(describe<KEYS, false>(p, item, x), 1 << 20) : 0; };
  Work other;
  const int mine = weight(lane, w);  // (the first 64 items stay in the lanes)
  int per_head = __builtin_amdgcn_readlane(scan(mine), 63);
  for (int base = 64; base < p.items; base += 64) per_head += __builtin_amdgcn_readlane(scan(weight(base + lane, other)), 63);
  // (without any row too: the join has to find that there are no parts)
  const Cut cut = cut_for(p, per_head);
  int sums = scan(cut.parts(mine)), all = __builtin_amdgcn_readlane(sums, 63);
  if (blockIdx.x == 0 && threadIdx.x < 64 && lane < p.items) p.item_end[lane] = sums;
  for (int base = 64; base < p.items; base += 64) {
    const int x = scan(cut.parts(weight(base + lane, other)));
    if (blockIdx.x == 0 && threadIdx.x < 64 && base + lane < p.items) p.item_end[base + lane] = all + x;
    all += __builtin_amdgcn_readlane(x, 63);
  }
  // renumbered, each XCD takes a contiguous run, so the parts of a (sequence, key head) pair share an L2
  const int nb = all * p.c.num_heads;
  if ((int)blockIdx.x >= nb) return false;
  const int per = nb >> 3, extra = nb & 7, xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  const int id = xcd < extra ? xcd * (per + 1) + idx : extra * (per + 1) + (xcd - extra) * per + idx;
  const int kv_head = uniform((int)((unsigned)id / (unsigned)all));
  int want = id - kv_head * all, n = 0;
  for (int base = 0;; base += 64) {
    int parts = 0;
    if (base) {
      parts = cut.parts(weight(base + lane, w));
      sums = scan(parts);
    }
    const uint64_t later = __ballot(sums > want);
    if (later) {
      const int l = __builtin_ctzll(later), before = l ? __builtin_amdgcn_readlane(sums, l - 1) : 0;
      n = __builtin_amdgcn_readlane(sums, l) - before;
      want -= before;
      take_from_lane(w, l);
      break;
    }
    want -= __builtin_amdgcn_readlane(sums, 63);
  }
  take_part(w, want, n);
  w.kv_head = kv_head;
  w.slot = n == 1 ? -1 : id;
  return true;
}

// The key whose row is loaded for key j: j itself where some row of the tile sees it, else one
// that is seen.  So nothing is read past a sequence's end or from pages that left the window;
// the weights of such places are zero (and the values finite, or cleared: see below).
__device__ __forceinline__ int key_to_load(const Work& w, int sinks, int j) {
  j = min(j, w.key_end - 1);
  return j < sinks ? j : max(j, w.key_from);
}
// A page number outside the cache reads page 0 (the host cannot see the table's contents).
__device__ __forceinline__ int page_entry(const AttnParams& p, const int32_t* row, int col) {
  const int pg = row[col];
  return (unsigned)pg < (unsigned)p.c.num_pages ? pg : 0;
}

// One lane's query row.
struct Row {
  int place;        // its place in the sequence; very low for rows that do not exist
  int token, head;  // packed query row and query head
  int r;            // number among the sequence's rows
  bool live;
};
__device__ __forceinline__ Row get_row(const AttnParams& p, const Work& w, int r) {
  Row o;
  o.r = r;
  o.live = r < w.rows;
  const int t = div(min(r, w.rows - 1), p.group);
  o.head = w.kv_head * p.group.d + min(r, w.rows - 1) - t * p.group.d;
  o.token = w.q_first + t;
  o.place = o.live ? w.place0 + t : INT32_MIN / 2;
  return o;
}

template <int D>
struct State {
  v16f o[D / 32];  // O^T: lane = query, register 16-groups of 32 values of D
  float m, z;      // running maximum (log2 units), this half wave's part of the sum
};

template <int D>
__device__ __forceinline__ void init(State<D>& st) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) st.o[i][j] = 0.f;
  st.m = NEG_INF;
  st.z = 0.f;
}

// Values that are no numbers.  The weight of a place that a query does not see is zero, which is not enough where
// the value is NaN or infinite and other rows of the tile see it.  So outside of the tiles that every row sees
// in whole, such values go to LDS as zeros, and where a wave has met one, they are added at the end, from memory,
// to the outputs of the rows that see them.  Infinite is what BF16 does not hold: codes of 240 and more under
// scales of 2^120 and more.  Scores need none of this, since mask() replaces them.  (What it costs: nothing
// for single tokens, 0 to 1% of most chunks, 3% of the shortest prompts and of some at 64 values a head: 2048 queries over 8192
// keys 228.8 -> 229.0 us, ragged chunks 155.2 -> 155.9, windowed ones 62.4 -> 63.2, 8 prompts of 512 39.1 -> 40.1, 4 x 1024
// queries at 64 values a head 106.0 -> 109.9.)
//
// The tiles of a list that rows at places lo to hi all see in whole, or all alike: n from `from` on.  (Of the first
// tokens' tiles none is counted where there is a window.)
struct WholeTiles {
  int from;
  unsigned n;
  __device__ __forceinline__ bool has(int i) const { return (unsigned)(i - from) < n; }
};
template <int KEYS>
__device__ __forceinline__ WholeTiles whole_tiles(const AttnParams& p, const Work& w, int lo, int hi) {
  if (lo == hi) return {0, UINT32_MAX};
  // key tile t, number t - first_tile + sink_tiles, lacks no keys at its end up to (t + 1) KEYS - 1 = lo, and by its
  // window none from t KEYS = hi - window + 1 on
  const int list = w.sink_tiles - w.first_tile, from = p.window ? list + (hi - p.window + KEYS) / KEYS : 0;
  return {uniform(from), (unsigned)uniform(max(list + (lo + 1) / KEYS - from, 0))};
}
// Whether one of a lane's 16 codes is NaN or may be infinite as BF16.
__device__ __forceinline__ bool may_be_odd(v4u x, uint32_t sf) {
  unsigned m = 0;  // bit 7 of a byte: its code is NaN
#pragma unroll
  for (int i = 0; i < 4; ++i) m |= (x[i] & 0x7F7F7F7Fu) + 0x01010101u;
  return (m & 0x80808080u) != 0 || sf >= 247;  // (247: 2^120)
}
// 8 BF16 that are no numbers become zeros.
__device__ __forceinline__ v4u clear_odd(v4u x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((x[i] & 0x7F80u) == 0x7F80u) x[i] &= 0xFFFF0000u;
    if ((x[i] & 0x7F800000u) == 0x7F800000u) x[i] &= 0xFFFFu;
  }
  return x;
}
// Whether a query at `place` sees key j.
__device__ __forceinline__ bool sees(const AttnParams& p, int place, int j) {
  return j <= place && (!p.window || j > place - p.window || j < p.sinks);
}
// What clear_odd has taken out of four places of a row: NaN, infinities, or nothing.
__device__ __forceinline__ v4f odd_values(unsigned codes, uint32_t sf) {
  const float s = __uint_as_float(sf << 23);
  const unsigned lo = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, false));
  const unsigned hi = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, true));
  auto odd = [](unsigned bits) { return (bits & 0x7F800000u) == 0x7F800000u ? __uint_as_float(bits) : 0.f; };
  return (v4f){odd(lo << 16), odd(lo & 0xFFFF0000u), odd(hi << 16), odd(hi & 0xFFFF0000u)};
}
// Key j's value row.
struct ValueRow {
  const uint8_t* codes;
  uint32_t sf;
};
__device__ __forceinline__ ValueRow value_row(const AttnParams& p, const Work& w, const int32_t* table, int j) {
  const int col = div(j, p.c.page), off = j - col * p.c.page.d, pg = page_entry(p, table, col);
  return {p.c.v + pg * p.c.page_stride + w.kv_head * p.c.head_stride + off * p.c.token_stride,
          p.c.v_sf[pg * p.c.sf_page_stride + w.kv_head * p.c.sf_head_stride + off * p.c.sf_token_stride]};
}

// Scores of keys that the lane's query does not see become -infinity.  key0: first key; a lane's
// register i of a block is key key0 + 4 (lane / 32) + c with c = 32 block + 8 (i / 4) + i % 4, so
// each bound is a number of the lane against constants.  late, early (uniform): whether some row of the
// wave may lack the tile's last keys, or its first ones (by its window).
template <int NB>
__device__ __forceinline__ void mask(const AttnParams& p, v16f (&s)[NB], int key0, int place, int h, bool late, bool early) {
  const int first = key0 + 4 * h;
  if (late) {
    const int end = place - first;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 32 * b + 8 * (i / 4) + i % 4 <= end ? s[b][i] : NEG_INF;
  }
  if (early) {
    const int from = place - p.window - first;
    if (key0 >= p.sinks) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] = 32 * b + 8 * (i / 4) + i % 4 > from ? s[b][i] : NEG_INF;
    } else {
      const int sinks = p.sinks - first;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = 32 * b + 8 * (i / 4) + i % 4;
          s[b][i] = c > from || c < sinks ? s[b][i] : NEG_INF;
        }
    }
  }
}

// Scores of NB blocks of 32 keys -> weights (as B operands of the second product), updating the
// running maximum, sum and, where the maximum rises, the outputs.
template <int D, int NB>
__device__ __forceinline__ void softmax(const AttnParams& p, State<D>& st, v16f (&s)[NB], v8bf (&w)[NB][2]) {
  float top = s[0][0];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
  top = both_max(top) * p.scale_log2;  // (the scale is positive)
  if (__any(top > st.m + SLACK)) {
    const float m = fmaxf(st.m, top);
    const float f = m == NEG_INF ? 1.f : exp2_hw(st.m - m);
    st.m = m;
    st.z *= f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) st.o[d][i] *= f;
  }
  const float sub = st.m == NEG_INF ? 0.f : -st.m;  // nothing seen yet: every weight is 2^-inf = 0
  float z = 0.f;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[b][i] = exp2_hw(__builtin_fmaf(s[b][i], p.scale_log2, sub));
      z += s[b][i];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      v4u x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = pack2(s[b][8 * u + 2 * i], s[b][8 * u + 2 * i + 1]);
      w[b][u] = __builtin_bit_cast(v8bf, x);
    }
  }
  st.z += z;
}

// O^T += V^T P^T over NB blocks of 32 keys of the V tile at `v` (LDS bytes), for DO values of D from d0 on.
template <int D, int DO, int NB>
__device__ __forceinline__ void product_v(State<DO>& st, const v8bf (&w)[NB][2], const uint8_t* v, int d0, int lane) {
  const int r = (lane & 15) >> 2, h = lane >> 5;
  // lane's 8 bytes within a 4-row, 32-byte group: row r, 8-byte piece lane % 4; the second 16
  // lanes of a half wave take the next 32 bytes
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = 32 * b + 16 * u + 4 * h + r;
#pragma unroll
      for (int d = 0; d < DO / 32; ++d) {
        const int chunk = v_chunk<D>(row, d0 / 8 + 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1));
        const int at = row * 2 * D + chunk * 16 + (lane & 1) * 8;
        const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LDS v4s*)(v + at));
        const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LDS v4s*)(v + at + 8 * 2 * D));
        const v8s a = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        st.o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), w[b][u], st.o[d], 0, 0, 0);
      }
    }
}

__device__ __forceinline__ float inverse(float z) { return z > 0.f ? 1.f / z : (z == z ? 0.f : z); }
__device__ __forceinline__ float log_sum(float m, float z) {
  return z > 0.f ? (m + __log2f(z)) * 0.6931471805599453f : (z == z ? NEG_INF : z);
}

// An item's result, or a part's.  Register i of 16-group d is value 32 d + 8 (i / 4) + 4 (lane / 32) + i % 4.
// z: summed over the half waves; the DO values of the row from d0 on.
template <int D, int DO>
__device__ __forceinline__ void store_row(const AttnParams& p, const Work& w, const Row& row, const v16f (&o)[DO / 32],
                                          float m, float z, int d0, int h) {
  if (!row.live) return;
  if (w.slot < 0) {
    const float f = inverse(z);
    uint16_t* dst = p.out + row.token * p.o_token_stride + row.head * p.o_head_stride + d0;
#pragma unroll
    for (int d = 0; d < DO / 32; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(v2u*)(dst + 32 * d + 8 * j + 4 * h) = (v2u){pack2(o[d][4 * j] * f, o[d][4 * j + 1] * f),
                                                      pack2(o[d][4 * j + 2] * f, o[d][4 * j + 3] * f)};
    if (p.lse && h == 0 && d0 == 0) p.lse[(int64_t)row.token * p.num_q_heads + row.head] = log_sum(m, z);
  } else {
    const int64_t at = (int64_t)w.slot * p.tile_rows + row.r - w.row0;
    float* dst = p.part_o + at * D + d0;
#pragma unroll
    for (int d = 0; d < DO / 32; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(v4f*)(dst + 32 * d + 8 * j + 4 * h) = (v4f){o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
    if (h == 0 && d0 == 0) *(v2f*)(p.part_mz + 2 * at) = (v2f){m, z};
  }
}

// ---------------------------------------------------------------- many rows: chunks of a prompt
// NW waves, each with 32 query rows, share tiles of KEYS keys.  What bounds it: a wave's tile of 64 keys takes 32
// matrix instructions of 32 cycles at D = 128 (1024 cycles; half of that at D = 64) and about as long on
// the vector unit, where 32 exponentials at a quarter of the rate are half of it.  Both units have to be
// kept busy by different waves.
//
// D = 128: eight waves, two on each SIMD, and the two halves of the workgroup take turns: while waves
// 0-3 are in the matrix phase of a tile (O^T += V^T P^T of the tile before, S^T of this one), waves 4-7
// are in the vector phase (the softmax) of theirs, half a tile behind.  One barrier a tile keeps them
// there: waves 0-3 come to it between their matrix phase of tile i and their vector phase, waves 4-7
// when their vector phase of tile i - 1 has ended.  So between two barriers, i and i + 1, waves 0-3 are
// in vector phase i and matrix phase i + 1, waves 4-7 in matrix phase i and vector phase i; a barrier
// after each phase measured 1% more.  When chosen, on 2048 queries (32 heads, 8 key heads) over 8192 keys:
// 236 us with turns, 269 without, 300 with turns but LDS reads one matrix instruction ahead instead of
// four.  D = 64 is bound by the vector unit, which a single half cannot fill: four waves without turns
// and three such workgroups a CU (61 us on 2 x 2048 queries in a window of 1024; with turns 74, eight
// waves without 70).  D = 256: a wave with the queries and outputs of 32 rows has no room beside it on its
// SIMD, and a single one is bound by how fast it issues.  So two waves, one of each half of the workgroup,
// share 32 rows: both compute their scores and weights, each half of the outputs (1536 queries, 16 heads, 4
// key heads, over 7680 keys: 314 us; with four waves, each alone with its rows, 405; now 295).
//
// Tiles lie widened in LDS.  With turns, in rings of three: stage i brings K of tile i + 2 and V of tile
// i + 1; a wave issues its loads at the end of its matrix phase of tile i, when its LDS reads are out
// (255 us when issued before them), and widens and stores them at the end of the vector phase: K to the
// slot of tile i - 1, V to that of tile i + 1.  Between the barriers around it, K of tiles i and i + 1 and
// V of tiles i - 1 and i are read: other slots of the three.  Without turns, two slots, loads a whole tile
// ahead.
// Each wave loads GR rows of K and of V of a stage (one 16-byte load a lane); where GR divides the page
// size and every one of them is seen, their address is scalar arithmetic on a page number out of 64 that
// the lanes hold, else it is found lane by lane.
template <int D>
struct Wide {
  static constexpr int NW = D == 64 ? 4 : 8, KEYS = D == 256 ? 32 : 64, NB = KEYS / 32;
  static constexpr int SHARE = D == 256 ? 2 : 1, DO = D / SHARE;  // waves that share 32 rows, a wave's values of the output
  static constexpr bool TURNS = D != 64;
  static constexpr int THREADS = NW * 64, TILE = KEYS * D * 2;  // TILE: bytes of a widened K or V tile
};

// The end of a phase, with a barrier for those whose turn ends there; no instruction is moved from one
// phase to another.
__device__ __forceinline__ void phase_end(bool wait) {
  __builtin_amdgcn_sched_barrier(0);
  if (wait) __syncthreads();
  __builtin_amdgcn_sched_barrier(0);
}

template <int D>
__global__ void __launch_bounds__(Wide<D>::THREADS, D == 64 ? 3 : 2) wide_kernel(const AttnParams p) {
  constexpr int NW = Wide<D>::NW, KEYS = Wide<D>::KEYS, NB = Wide<D>::NB, TILE = Wide<D>::TILE, DO = Wide<D>::DO;
  constexpr int CH = D / 16, GR = 64 / CH;
  static_assert(KEYS / GR == NW);
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][Wide<D>::TURNS ? 3 : 2][TILE];  // [K, V][slot]
  __shared__ int met_odd[NW];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), h = lane >> 5;
  Work w;
  if (!get_work<KEYS, true>(p, w)) return;
  make_uniform(w);
  const int rows_of = wave % (NW / Wide<D>::SHARE), d0 = wave / (NW / Wide<D>::SHARE) * DO;
  const Row row = get_row(p, w, w.row0 + rows_of * ROWS + (lane & 31));
  // the places of this wave's rows, for whole-tile decisions
  const int wr0 = w.row0 + rows_of * ROWS;
  const int place_lo = w.place0 + div(min(wr0, w.rows - 1), p.group);
  const int place_hi = w.place0 + div(min(wr0 + ROWS, w.rows) - 1, p.group);

  v8bf q[D / 16];
  const int32_t* table = p.table + w.seq * p.table_stride;
  const bool page_whole = p.c.page.d % GR == 0;
  const int c = lane % CH, r = lane / CH;
  const int64_t head_at = w.kv_head * p.c.head_stride, head_sf = w.kv_head * p.c.sf_head_stride;
  const uint32_t lane_at = (uint32_t)(r * p.c.token_stride) + 16 * c, lane_sf = (uint32_t)(r * p.c.sf_token_stride);
  // Where a lane finds its part of GR rows from key j0 on: byte offsets into codes and scales.
  struct At {
    int64_t code, sf;
  };
  // 64 entries of the block table, one a lane, from column table_from
  int table_from = INT32_MIN / 2, entries = 0;
  auto place_rows = [&](int j0) {
    At a;
    const int j1 = j0 + GR - 1;
    if (page_whole && j1 < w.key_end && (j0 >= w.key_from || j1 < p.sinks)) {
      const int col = div(j0, p.c.page);
      if ((unsigned)(col - table_from) >= 64u) {
        table_from = col;
        entries = table[min(col + lane, p.table_cols - 1)];
        entries = (unsigned)entries < (unsigned)p.c.num_pages ? entries : 0;
      }
      const uint32_t pg = __builtin_amdgcn_readlane(entries, col - table_from), off = j0 - col * p.c.page.d;
      a.code = uniform((int64_t)(pg * (uint64_t)p.c.page_stride + head_at + off * (uint32_t)p.c.token_stride)) + lane_at;
      a.sf = uniform((int64_t)(pg * (uint64_t)p.c.sf_page_stride + head_sf + off * (uint32_t)p.c.sf_token_stride)) + lane_sf;
    } else {
      const int j = key_to_load(w, p.sinks, j0 + r);
      const int col = div(j, p.c.page), off = j - col * p.c.page.d, pg = page_entry(p, table, col);
      a.code = pg * p.c.page_stride + head_at + off * p.c.token_stride + 16 * c;
      a.sf = pg * p.c.sf_page_stride + head_sf + off * p.c.sf_token_stride;
    }
    return a;
  };
  // With turns, a wave's V rows of a stage are its K rows of the stage before; without, they are of the same tile.
  constexpr bool TURNS = Wide<D>::TURNS;
  At at;
  struct Stage {
    v4u k, v;             // codes
    uint32_t k_sf, v_sf;  // and their rows' scale codes
  };
  Stage ahead;
  auto place_tile = [&](int i) { return place_rows(w.tile_key(min(max(i, w.t0), w.t1 - 1), KEYS) + wave * GR); };
  auto fetch = [&](Stage& to, int i) {
    auto get_v = [&] {
      to.v = *(const v4u*)(p.c.v + at.code);
      to.v_sf = p.c.v_sf[at.sf];
    };
    if (TURNS) get_v();
    at = place_tile(i + 2);  // (tiles past the list repeat its ends and are not read)
    if (!TURNS) get_v();
    to.k = *(const v4u*)(p.c.k + at.code);
    to.k_sf = p.c.k_sf[at.sf];
  };
  const WholeTiles whole = whole_tiles<KEYS>(p, w, w.place0 + div(w.row0, p.group), w.key_end - 1);
  // Set where a wave has cleared a value of another tile.  (All waves see it in time, as they see the tile: a barrier
  // lies between a put and the products with it.)
  if (lane == 0) met_odd[wave] = 0;
  const int rr = wave * GR + r;
  auto store = [&](uint8_t* dst, v4u x, v4u y, int c0, int c1) {
    *(v4u*)(dst + rr * 2 * D + c0 * 16) = x;
    *(v4u*)(dst + rr * 2 * D + c1 * 16) = y;
  };
  auto put = [&](const Stage& from, uint8_t* k, uint8_t* v) {
    const float ks = __uint_as_float(from.k_sf << 23), vs = __uint_as_float(from.v_sf << 23);
    store(k, widen8(from.k.x, from.k.y, ks), widen8(from.k.z, from.k.w, ks), k_chunk<D>(rr, 2 * c), k_chunk<D>(rr, 2 * c + 1));
    store(v, widen8(from.v.x, from.v.y, vs), widen8(from.v.z, from.v.w, vs), v_chunk<D>(rr, 2 * c), v_chunk<D>(rr, 2 * c + 1));
  };
  // after put, with V of tile i
  auto clear_tile = [&](const Stage& from, uint8_t* v, int i) {
    if (__builtin_expect(!whole.has(i), 0)) {
      if (__builtin_expect(__any(may_be_odd(from.v, from.v_sf)), 0)) {
        const float vs = __uint_as_float(from.v_sf << 23);
        if (lane == 0) met_odd[wave] = 1;
        store(v, clear_odd(widen8(from.v.x, from.v.y, vs)), clear_odd(widen8(from.v.z, from.v.w, vs)), v_chunk<D>(rr, 2 * c), v_chunk<D>(rr, 2 * c + 1));
      }
    }
  };

  State<DO> st;
  init(st);
  v8bf wt[NB][2];  // (zero weights go with the first matrix phase, which has no tile before it)
#pragma unroll
  for (int b = 0; b < NB; ++b) wt[b][0] = wt[b][1] = __builtin_bit_cast(v8bf, (v4u){0, 0, 0, 0});
  auto scores = [&](v16f (&s)[NB], const uint8_t* k) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int x = 0; x < 16; ++x) s[b][x] = 0.f;
      const int kr = 32 * b + (lane & 31);
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const v8bf a = *(const v8bf*)(k + kr * 2 * D + k_chunk<D>(kr, 2 * x + h) * 16);
        s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[x], s[b], 0, 0, 0);
      }
    }
  };
  auto weights = [&](int i, v16f (&s)[NB]) {
    const int key0 = w.tile_key(i, KEYS);
    const bool late = key0 + KEYS - 1 > place_lo, early = p.window && key0 <= place_hi - p.window && key0 + KEYS > p.sinks;
    if (late || early) mask<NB>(p, s, key0, row.place, h, late, early);
    softmax<DO, NB>(p, st, s, wt);
  };
  // With turns: tile i of the list, number X of three: its K is in slot X, V of the tile before in slot X - 1.
  auto step = [&](int i, auto number) {
    constexpr int X = decltype(number)::value, NEXT = (X + 1) % 3, LAST = (X + 2) % 3;
    product_v<D, DO, NB>(st, wt, lds[1][LAST], d0, lane);
    v16f s[NB];
    scores(s, lds[0][X]);
    // Four fragments are read ahead of the matrix instruction that takes them.
    constexpr int NVF = DO / 32 * NB * 2, NKF = D / 16 * NB, AHEAD = 4;  // V and K fragments (and matrix instructions)
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * AHEAD, 0);
#pragma unroll
    for (int x = 0; x < NVF - AHEAD; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
#pragma unroll
    for (int x = 0; x < NKF; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, AHEAD, 0);
    __builtin_amdgcn_sched_barrier(0);
    fetch(ahead, i);
    phase_end(wave < 4);
    weights(i, s);
    // (the weights are wanted here: left to itself, the compiler computes some in the next phase)
#pragma unroll
    for (int b = 0; b < NB; ++b) asm volatile("" : "+v"(wt[b][0]), "+v"(wt[b][1]));
    asm volatile("" : "+v"(st.z));
    __builtin_amdgcn_sched_barrier(0);
    put(ahead, lds[0][LAST], lds[1][NEXT]);
    clear_tile(ahead, lds[1][NEXT], i + 1);
    phase_end(wave >= 4 && i + 1 < w.t1);
  };
  // Without turns: tile i with K and V in slot X; leaves tile i + 1 in the other slot and tile i + 2 on its way.
  auto plain_step = [&](int i, auto slot) {
    constexpr int X = decltype(slot)::value, AHEAD = 2;
    v16f s[NB];
    scores(s, lds[0][X]);
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
    for (int x = 0; x < D / 16 * NB - AHEAD; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, AHEAD, 0);
    __builtin_amdgcn_sched_barrier(0);
    weights(i, s);
    __builtin_amdgcn_sched_barrier(0);
    product_v<D, DO, NB>(st, wt, lds[1][X], d0, lane);
    put(ahead, lds[0][1 - X], lds[1][1 - X]);
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * AHEAD, 1);
#pragma unroll
    for (int x = 0; x < D / 16 * NB - AHEAD; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 1);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, AHEAD, 1);
    __builtin_amdgcn_sched_barrier(0);
    clear_tile(ahead, lds[1][1 - X], i + 1);
    fetch(ahead, i);
    __syncthreads();
  };
  if (w.t0 < w.t1) {
    at = place_tile(w.t0);
    Stage first;
    fetch(first, w.t0 - 2);
    fetch(ahead, w.t0 - 1);
    // (after the tiles' loads, whose addresses wait for the block table: loads return in order)
    __builtin_amdgcn_sched_barrier(0);
    const uint16_t* src = p.q + row.token * p.q_token_stride + row.head * p.q_head_stride + 8 * h;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[i] = *(const v8bf*)(src + 16 * i);
    if constexpr (TURNS) {
      put(first, lds[0][0], lds[1][2]);
      clear_tile(first, lds[1][2], w.t0);
      put(ahead, lds[0][1], lds[1][0]);
      clear_tile(ahead, lds[1][0], w.t0);
      __syncthreads();
      if (wave >= 4) __syncthreads();
      int last = 0;  // slot of the last tile
      for (int i = w.t0;; i += 3) {
        step(i, Int<0>{});
        last = 0;
        if (i + 1 == w.t1) break;
        step(i + 1, Int<1>{});
        last = 1;
        if (i + 2 == w.t1) break;
        step(i + 2, Int<2>{});
        last = 2;
        if (i + 3 == w.t1) break;
      }
      product_v<D, DO, NB>(st, wt, lds[1][last], d0, lane);
    } else {
      put(first, lds[0][0], lds[1][0]);
      clear_tile(first, lds[1][0], w.t0);
      __syncthreads();
      for (int i = w.t0; i < w.t1; i += 2) {
        plain_step(i, Int<0>{});
        if (i + 1 < w.t1) plain_step(i + 1, Int<1>{});
      }
    }
    int any = 0;
#pragma unroll
    for (int x = 0; x < NW; ++x) any |= met_odd[x];
    if (__builtin_expect(uniform(any), 0)) {
      for (int i = w.t0; i < w.t1; ++i) {
        if (whole.has(i)) continue;
        const int key0 = w.tile_key(i, KEYS);
        for (int j = key0; j < min(key0 + KEYS, w.key_end); ++j) {
          if (j < w.key_from && j >= p.sinks) continue;  // (no row sees it, and its page may be gone)
          const ValueRow v = value_row(p, w, table, j);
          if (!sees(p, row.place, j)) continue;
#pragma unroll
          for (int d = 0; d < DO / 32; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const v4f add = odd_values(*(const unsigned*)(v.codes + d0 + 32 * d + 8 * x + 4 * h), v.sf);
#pragma unroll
              for (int e = 0; e < 4; ++e) st.o[d][4 * x + e] += add[e];
            }
        }
      }
    }
  }
  store_row<D, DO>(p, w, row, st.o, st.m, both_sum(st.z), d0, h);
}

// ---------------------------------------------------------------- few rows: single tokens
// Bound by reading the cache once.  The four waves share 16 RB query rows and take the item's key tiles
// (32 keys) in turn, each by itself: no barrier until their sums are joined.  A wave reads K straight
// into operand registers (the order of D within the contraction is free: lane group g takes bytes
// 16 g.. of every 64), stages V in its own LDS slice for the transposing reads, and has the next
// tile's loads on their way before the softmax.  16 x 16 matrix instructions: with 32 columns, single
// tokens of 8 heads a key head left registers for half as many waves.
//
// S^T in blocks of 16 keys: lane group g (lane / 16) holds keys 4 g + i of query lane % 16.  In the second
// product's step of 32 keys, group g's eight operand places are keys 4 g + i and 16 + 4 g + i.
// Without a common page for each 16 keys, rows are addressed lane by lane.
template <int D>
__device__ __forceinline__ int narrow_chunk(int row, int c) {
  // 32-byte pieces of a row move by its number, so that 16 lanes' 4 rows, and the next groups', differ in
  // banks; within a piece the 16-byte halves change places on odd rows, for the writes
  return c ^ (D == 64 ? ((row >> 1) & 3) << 1 : (row & 7) << 1) ^ (row & 1);
}

// Maximum and sum over the four lane groups.
__device__ __forceinline__ float groups_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return both_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float groups_sum(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return both_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Buffer descriptor from a scalar address on, 2^31 - 1 bytes long (the host keeps a head's page below that).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* base) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)uniform((int64_t)base), (short)0, 0x7FFFFFFF, 0x00020000);
}

template <int D, int RB, int NW>
__global__ void __launch_bounds__(NW * 64, D == 256 ? 1 : 2) narrow_kernel(const AttnParams p) {
  constexpr int KEYS = 32, TILE = KEYS * D * 2;
  constexpr int CH = D / 16, PASS = 64 / CH, NP = KEYS / PASS;  // V: 16-code chunks of a row, rows of a load, loads
  constexpr int ROWS_ALL = 16 * RB;
  constexpr int JD = 64;  // values of D joined at once
  constexpr int JOIN = NW * ROWS_ALL * (JD + 4) * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[NW * TILE > JOIN ? NW * TILE : JOIN];
  __shared__ float mz[NW][2][ROWS_ALL];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), g = lane >> 4, col = lane & 15;
  uint8_t* vt = lds + wave * TILE;
  const bool halves_whole = p.c.page.d % 16 == 0;
  const uint32_t k_at = (uint32_t)(col * p.c.token_stride) + 16 * g, k_sf_at = (uint32_t)(col * p.c.sf_token_stride);
  const uint32_t v_at = (uint32_t)(lane / CH * p.c.token_stride) + 16 * (lane % CH), v_sf_at = (uint32_t)(lane / CH * p.c.sf_token_stride);
  const uint32_t v_step = (uint32_t)(PASS * p.c.token_stride), v_sf_step = (uint32_t)(PASS * p.c.sf_token_stride);

  Work w;
  if (!get_work<KEYS, false>(p, w)) return;
  make_uniform(w);
  Row row[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) row[b] = get_row(p, w, w.row0 + 16 * b + col);
  const int place_lo = w.place0 + div(w.row0, p.group);
  const int place_hi = w.place0 + div(min(w.row0 + ROWS_ALL, w.rows) - 1, p.group);
  v8bf q[RB][D / 32];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const uint16_t* src = p.q + row[b].token * p.q_token_stride + row[b].head * p.q_head_stride + 16 * g;
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      q[b][2 * x] = *(const v8bf*)(src + 64 * x);
      q[b][2 * x + 1] = *(const v8bf*)(src + 64 * x + 8);
    }
  }
  const int32_t* table = p.table + w.seq * p.table_stride;
  const int64_t head_at = w.kv_head * p.c.head_stride, head_sf = w.kv_head * p.c.sf_head_stride;
  // 128 entries of the block table, two a lane, from column table_from; the second 64 are loaded when
  // the first come into use
  int table_from = INT32_MIN / 2, entries = 0, entries_next = 0;
  auto load_entries = [&](int c) {
    const int e = table[min(max(c, 0) + lane, p.table_cols - 1)];
    return (unsigned)e < (unsigned)p.c.num_pages ? e : 0;
  };
  // Byte offsets of the tile's two halves (16 keys) where that will do.
  struct Half {
    int64_t code, sf;
  };
  Half half[2];
  bool fast = false;
  int next_key = 0;
  auto place = [&](int i) {
    const int key0 = w.tile_key(i, KEYS);
    next_key = key0;
    fast = halves_whole && key0 + KEYS <= w.key_end && (key0 >= w.key_from || key0 + KEYS <= p.sinks);
    if (!fast) return;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int c = div(key0 + 16 * x, p.c.page);
      if ((unsigned)(c - table_from) >= 64u) {
        entries = (unsigned)(c - table_from) < 128u ? entries_next : load_entries(c);
        table_from = (unsigned)(c - table_from) < 128u ? table_from + 64 : c;
        entries_next = load_entries(table_from + 64);
      }
      const uint32_t pg = __builtin_amdgcn_readlane(entries, c - table_from), off = key0 + 16 * x - c * p.c.page.d;
      half[x].code = (int64_t)(pg * (uint64_t)p.c.page_stride + head_at + off * (uint32_t)p.c.token_stride);
      half[x].sf = (int64_t)(pg * (uint64_t)p.c.sf_page_stride + head_sf + off * (uint32_t)p.c.sf_token_stride);
    }
  };
  auto slow_row = [&](int j) {
    j = key_to_load(w, p.sinks, j);
    const int c = div(j, p.c.page), off = j - c * p.c.page.d, pg = page_entry(p, table, c);
    return Half{pg * p.c.page_stride + head_at + off * p.c.token_stride, pg * p.c.sf_page_stride + head_sf + off * p.c.sf_token_stride};
  };
  v4u kr[2][D / 64], vr[NP];
  uint32_t ks[2], vs[NP];
  // (Where the rows' addresses are scalar, through buffer descriptors of the halves; lane by lane, the
  // scale bytes are widened at once, so that the two ways' values meet as words: as bytes they would be
  // widened where they meet, and waited for there.)
  auto fetch_k = [&]() {
    if (fast) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const __amdgpu_buffer_rsrc_t codes = rsrc(p.c.k + half[x].code), sf = rsrc(p.c.k_sf + half[x].sf);
#pragma unroll
        for (int y = 0; y < D / 64; ++y) kr[x][y] = __builtin_amdgcn_raw_buffer_load_b128(codes, k_at + 64 * y, 0, 0);
        ks[x] = __builtin_amdgcn_raw_buffer_load_b8(sf, k_sf_at, 0, 0);
      }
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const Half a = slow_row(next_key + 16 * x + col);
#pragma unroll
        for (int y = 0; y < D / 64; ++y) kr[x][y] = *(const v4u*)(p.c.k + a.code + 16 * g + 64 * y);
        ks[x] = p.c.k_sf[a.sf];
        asm volatile("" : "+v"(ks[x]));
      }
    }
  };
  auto fetch_v = [&]() {
    if (fast) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const __amdgpu_buffer_rsrc_t codes = rsrc(p.c.v + half[x].code), sf = rsrc(p.c.v_sf + half[x].sf);
#pragma unroll
        for (int n = 0; n < NP / 2; ++n) {
          vr[x * (NP / 2) + n] = __builtin_amdgcn_raw_buffer_load_b128(codes, v_at, n * v_step, 0);
          vs[x * (NP / 2) + n] = __builtin_amdgcn_raw_buffer_load_b8(sf, v_sf_at, n * v_sf_step, 0);
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        const Half a = slow_row(next_key + n * PASS + lane / CH);
        vr[n] = *(const v4u*)(p.c.v + a.code + 16 * (lane % CH));
        vs[n] = p.c.v_sf[a.sf];
        asm volatile("" : "+v"(vs[n]));
      }
    }
  };

  v4f o[RB][D / 16];
  float m[RB], z[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    m[b] = NEG_INF;
    z[b] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[b][d] = (v4f){0.f, 0.f, 0.f, 0.f};
  }
  const WholeTiles whole = whole_tiles<KEYS>(p, w, place_lo, place_hi);
  bool odd = false;  // the wave has cleared a value of another tile
  int i = w.t0 + wave;
  if (i < w.t1) {
    place(i);
    fetch_k();
    fetch_v();
    // (keeps the compiler from carrying these through the loop as bytes, which it would widen, and so
    // wait for, where they are loaded)
#pragma unroll
    for (int x = 0; x < 2; ++x) asm volatile("" : "+v"(ks[x]));
#pragma unroll
    for (int n = 0; n < NP; ++n) asm volatile("" : "+v"(vs[n]));
  }
  for (; i < w.t1; i += NW) {
    const int key0 = w.tile_key(i, KEYS);
    const bool more = i + NW < w.t1;
    if (more) place(i + NW);
    v4f s[RB][2];
#pragma unroll
    for (int b = 0; b < RB; ++b) s[b][0] = s[b][1] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float scale = __uint_as_float(ks[x] << 23);
#pragma unroll
      for (int y = 0; y < D / 64; ++y) {
        const v8bf lo = __builtin_bit_cast(v8bf, widen8(kr[x][y].x, kr[x][y].y, scale));
        const v8bf hi = __builtin_bit_cast(v8bf, widen8(kr[x][y].z, kr[x][y].w, scale));
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          s[b][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, q[b][2 * y], s[b][x], 0, 0, 0);
          s[b][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, q[b][2 * y + 1], s[b][x], 0, 0, 0);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (more) fetch_k();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int r = lane / CH + n * PASS, c = lane % CH;
      const float scale = __uint_as_float(vs[n] << 23);
      *(v4u*)(vt + r * 2 * D + narrow_chunk<D>(r, 2 * c) * 16) = widen8(vr[n].x, vr[n].y, scale);
      *(v4u*)(vt + r * 2 * D + narrow_chunk<D>(r, 2 * c + 1) * 16) = widen8(vr[n].z, vr[n].w, scale);
    }
    if (__builtin_expect(!whole.has(i), 0)) {
      bool may = false;
#pragma unroll
      for (int n = 0; n < NP; ++n) may |= may_be_odd(vr[n], vs[n]);
      if (__builtin_expect(__any(may), 0)) {
        odd = true;
#pragma unroll 1
        for (int n = 0; n < NP; ++n) {
          const int r = lane / CH + n * PASS, c = lane % CH;
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            v4u* at = (v4u*)(vt + r * 2 * D + narrow_chunk<D>(r, 2 * c + x) * 16);
            *at = clear_odd(*at);
          }
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (more) fetch_v();
    __builtin_amdgcn_sched_barrier(0);
    const bool late = key0 + KEYS - 1 > place_lo, early = p.window && key0 <= place_hi - p.window && key0 + KEYS > p.sinks;
    v8bf wt[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (late || early) {
        const int first = key0 + 4 * g, end = row[b].place - first, from = p.window ? end - p.window : INT32_MIN, sinks = p.sinks - first;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = 16 * x + e;
            s[b][x][e] = c <= end && (c > from || c < sinks) ? s[b][x][e] : NEG_INF;
          }
      }
      float top = s[b][0][0];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, s[b][x][e]);
      top = groups_max(top) * p.scale_log2;  // (the scale is positive)
      if (__any(top > m[b] + SLACK)) {
        const float raised = fmaxf(m[b], top);
        const float f = raised == NEG_INF ? 1.f : exp2_hw(m[b] - raised);
        m[b] = raised;
        z[b] *= f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[b][d] *= f;
      }
      const float sub = m[b] == NEG_INF ? 0.f : -m[b];  // nothing seen yet: every weight is 2^-inf = 0
      v4u x4;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[b][x][e] = exp2_hw(__builtin_fmaf(s[b][x][e], p.scale_log2, sub));
          z[b] += s[b][x][e];
        }
        x4[2 * x] = pack2(s[b][x][0], s[b][x][1]);
        x4[2 * x + 1] = pack2(s[b][x][2], s[b][x][3]);
      }
      wt[b] = __builtin_bit_cast(v8bf, x4);
    }
    // the wave reads what its other lanes wrote: its LDS operations complete in order, so only the
    // compiler has to keep theirs
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int r = 4 * g + (col >> 2);
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      const int at = r * 2 * D + narrow_chunk<D>(r, 2 * d + ((lane & 3) >> 1)) * 16 + (lane & 1) * 8;
      const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LDS v4s*)(vt + at));
      const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LDS v4s*)(vt + at + 16 * 2 * D));
      const v8s a = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
      for (int b = 0; b < RB; ++b)
        o[b][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), wt[b], o[b][d], 0, 0, 0);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  if (__builtin_expect(odd, 0)) {
    for (i = w.t0 + wave; i < w.t1; i += NW) {
      const int key0 = w.tile_key(i, KEYS);
      if (whole.has(i)) continue;
      for (int j = key0; j < min(key0 + KEYS, w.key_end); ++j) {
        if (j < w.key_from && j >= p.sinks) continue;  // (no row sees it, and its page may be gone)
        const ValueRow v = value_row(p, w, table, j);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          const v4f add = odd_values(*(const unsigned*)(v.codes + 16 * d + 4 * g), v.sf);
#pragma unroll
          for (int b = 0; b < RB; ++b)
            if (sees(p, row[b].place, j)) o[b][d] += add;
        }
      }
    }
  }

  // join the waves: rescale to the common maximum and add up through LDS, JD values of D at a time
  float f[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    z[b] = groups_sum(z[b]);
    if (g == 0) {
      mz[wave][0][16 * b + col] = m[b];
      mz[wave][1][16 * b + col] = z[b];
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    float all = NEG_INF;
#pragma unroll
    for (int x = 0; x < NW; ++x) all = fmaxf(all, mz[x][0][16 * b + col]);
    f[b] = all == NEG_INF ? 1.f : exp2_hw(m[b] - all);
  }
  float* jo = (float*)lds;
  // this thread (of the first 256) adds up row jr (and jr + 16), values jd.. of JD
  const int jr = threadIdx.x >> 4, jd = 4 * (threadIdx.x & 15);
#pragma unroll
  for (int d0 = 0; d0 < D; d0 += JD) {
    if (d0) __syncthreads();
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int d = 0; d < JD / 16; ++d)
        *(v4f*)(jo + (wave * ROWS_ALL + 16 * b + col) * (JD + 4) + 16 * d + 4 * g) = o[b][d0 / 16 + d] * f[b];
    __syncthreads();
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const Row out = get_row(p, w, w.row0 + 16 * b + jr);
      if (jr >= 16 || !out.live) continue;
      float all = NEG_INF, sum = 0.f;
#pragma unroll
      for (int x = 0; x < NW; ++x) all = fmaxf(all, mz[x][0][16 * b + jr]);
#pragma unroll
      for (int x = 0; x < NW; ++x) sum += (all == NEG_INF ? 1.f : exp2_hw(mz[x][0][16 * b + jr] - all)) * mz[x][1][16 * b + jr];
      v4f a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < NW; ++x) a += *(const v4f*)(jo + (x * ROWS_ALL + 16 * b + jr) * (JD + 4) + jd);
      if (w.slot < 0) {
        a *= inverse(sum);
        *(v2u*)(p.out + out.token * p.o_token_stride + out.head * p.o_head_stride + d0 + jd) = (v2u){pack2(a.x, a.y), pack2(a.z, a.w)};
        if (p.lse && d0 == 0 && jd == 0) p.lse[(int64_t)out.token * p.num_q_heads + out.head] = log_sum(all, sum);
      } else {
        const int64_t at = (int64_t)w.slot * ROWS_ALL + 16 * b + jr;
        *(v4f*)(p.part_o + at * D + d0 + jd) = a;
        if (d0 == 0 && jd == 0) *(v2f*)(p.part_mz + 2 * at) = (v2f){all, sum};
      }
    }
  }
}

// ---------------------------------------------------------------- joining the parts
// out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) z_s over the parts s of a row's item.  A row is G groups of
// D / 4 lanes; group x takes parts x, x + G, ..., and the groups' sums are added in their order.  256
// threads for a row where rows are few and their parts many.  Otherwise G = 1 and a workgroup
// has STEPS rows for each lane group: most items may not be cut, and their workgroups' starts are what
// they cost.
template <int D, bool FEW>
struct Join {
  static constexpr int L = D / 4, G = FEW ? 256 / L : 1, PER = 256 / (L * G);  // PER: rows at a time
};

template <int D, bool FEW>
__global__ void __launch_bounds__(256) join_kernel(const AttnParams p) {
  using J = Join<D, FEW>;
  constexpr int L = J::L, G = J::G;
  const int lanes = threadIdx.x % L, group = threadIdx.x / L % G;
  const int steps = FEW ? 1 : p.join_steps, blocks = (p.join_rows + J::PER * steps - 1) / (J::PER * steps);
  const int id = blockIdx.x / blocks, kv_head = id % p.c.num_heads, item = id / p.c.num_heads;
  const int all = p.item_end[p.items - 1], end = p.item_end[item], from = item ? p.item_end[item - 1] : 0, n = end - from;
  if (n <= 1) return;  // no rows, or written as a whole
  Work w;
  item_rows<true>(p, item, w);
  w.kv_head = kv_head;
  w.place0 = 0;  // (places do not matter here)
  const int64_t step = p.tile_rows;
  for (int y = 0; y < steps; ++y) {
    const int part_row = (blockIdx.x % blocks * steps + y) * J::PER + threadIdx.x / (L * G);
    const Row row = get_row(p, w, w.row0 + part_row);
    const bool live = row.live && part_row < p.tile_rows;
    const int64_t at = (int64_t)(kv_head * all + from) * p.tile_rows + part_row;
    const v2f* mz = (const v2f*)p.part_mz + at;
    const float* part = p.part_o + at * D + 4 * lanes;
    float m = NEG_INF, z = 0.f;
    v4f o = {0.f, 0.f, 0.f, 0.f};
    if (live) {
      // (each group by its own running maximum; the loads of AT_ONCE parts go out together: 131071 keys, 96 parts
      // of 4 rows, 59.5 us, one by one 64.8)
      constexpr int AT_ONCE = 4;
      for (int x = group; x < n; x += G * AT_ONCE) {
        v2f a[AT_ONCE];
        v4f b[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
          a[u] = (v2f){NEG_INF, 0.f};
          if (x + u * G < n) {
            a[u] = mz[(x + u * G) * step];
            b[u] = *(const v4f*)(part + (x + u * G) * step * D);
          }
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
          // no part, or one in which the row sees nothing (its sum is zero; a part whose scores are all NaN has no
          // maximum either, but a NaN for its sum, which has to stay)
          if (a[u].x == NEG_INF && a[u].y == 0.f) continue;
          const float top = fmaxf(m, a[u].x), f = exp2_hw(m - top), g = exp2_hw(a[u].x - top);
          z = z * f + a[u].y * g;
          o = o * f + b[u] * g;
          m = top;
        }
      }
    }
    if constexpr (FEW) {
      __shared__ float sums[G][L][4], tops[G][2];
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
        const float f = tops[x][0] == NEG_INF ? 0.f : exp2_hw(tops[x][0] - m);
        z += f * tops[x][1];
        o += f * *(const v4f*)sums[x][lanes];
      }
    }
    if (!live) continue;
    o *= inverse(z);
    *(v2u*)(p.out + row.token * p.o_token_stride + row.head * p.o_head_stride + 4 * lanes) = (v2u){pack2(o.x, o.y), pack2(o.z, o.w)};
    if (p.lse && lanes == 0) p.lse[(int64_t)row.token * p.num_q_heads + row.head] = log_sum(m, z);
  }
}

template <int D>
hipError_t launch(const AttnParams& p, int form, hipStream_t stream) {
  const int64_t whole = (int64_t)p.items * p.c.num_heads, grid = p.head_aim ? p.most_parts : whole;
  const bool few = p.join_few;
  const int block_rows = few ? Join<D, true>::PER : Join<D, false>::PER * p.join_steps;
  const int64_t blocks = whole * ((p.join_rows + block_rows - 1) / block_rows);
  // threads of a grid stay below 2^32 (of whole items the host sees to it; cut ones are a few times the compute units)
  if (p.head_aim && (grid * Wide<128>::THREADS > int64_t(UINT32_MAX) || blocks * 256 > int64_t(UINT32_MAX))) return hipErrorInvalidValue;
  if (form == ATTN_WIDE)
    hipLaunchKernelGGL((wide_kernel<D>), dim3((unsigned)grid), dim3(Wide<D>::THREADS), 0, stream, p);
  else if (form == ATTN_NARROW_32)
    hipLaunchKernelGGL((narrow_kernel<D, 2, 4>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  else if (p.waves == 4)
    hipLaunchKernelGGL((narrow_kernel<D, 1, 4>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  else if constexpr (D != 256)
    hipLaunchKernelGGL((narrow_kernel<D, 1, 8>), dim3((unsigned)grid), dim3(512), 0, stream, p);
  else
    return hipErrorInvalidValue;
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.head_aim == 0) return e;
  if (few)
    hipLaunchKernelGGL((join_kernel<D, true>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((join_kernel<D, false>), dim3((unsigned)blocks), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace attn

hipError_t launch_attention(const AttnParams& p, int head_dim, int form, hipStream_t stream) {
  if (head_dim == 64) return attn::launch<64>(p, form, stream);
  if (head_dim == 128) return attn::launch<128>(p, form, stream);
  if (head_dim == 256) return attn::launch<256>(p, form, stream);
  return hipErrorInvalidValue;
}

}  // namespace dg
