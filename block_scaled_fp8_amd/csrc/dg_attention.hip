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

// What a workgroup works on: a tile of query rows of one (sequence, key head), and a part of the
// tiles of keys that these rows see.
struct Work {
  int seq, kv_head, split;
  int q_first;           // first packed query row (token) of the sequence
  int row0, rows;        // first row of the tile; rows of the sequence in all
  int place0;            // place of the sequence's first query (negative where queries exceed the context)
  int key_end;           // one past the last key that some row of the tile sees
  int key_from;          // first key of the window of the tile's first query
  int sink_tiles, first_tile;
  int t0, t1;            // key tiles [t0, t1) of this part, as list indices

  __device__ __forceinline__ int tile_key(int i, int keys) const { return (i < sink_tiles ? i : first_tile + i - sink_tiles) * keys; }
};

// KEYS: keys of a tile.  Returns false if there is no row.
template <int KEYS>
__device__ __forceinline__ bool get_work(const AttnParams& p, int tile_rows, Work& w) {
  // Workgroups are dealt to the eight XCDs in turn.  With the (sequence, key head) pair as the
  // fastest index, and a multiple of eight pairs, all workgroups of a pair land on one XCD and share
  // its L2, and the pairs of one sequence, as long as each other, spread over the XCDs.  Later rows
  // see more keys: they start first.
  const unsigned pairs = p.batch * p.c.num_heads;
  const unsigned pair = blockIdx.x % pairs;
  unsigned id = blockIdx.x / pairs;
  w.split = id % p.splits;
  const int qt = p.q_tiles - 1 - (int)(id / p.splits);
  w.kv_head = pair % p.c.num_heads;
  w.seq = pair / p.c.num_heads;
  int n;
  if (p.cu_q) {
    const int a = min(max(p.cu_q[w.seq], 0), p.total_q), b = min(max(p.cu_q[w.seq + 1], a), p.total_q);
    w.q_first = a;
    n = b - a;
  } else {
    w.q_first = w.seq * p.q_per_seq;
    n = p.q_per_seq;
  }
  const int g = p.group.d;
  w.rows = n * g;
  w.row0 = qt * tile_rows;
  if (w.row0 >= w.rows) return false;
  const int64_t held = (int64_t)p.table_cols * p.c.page.d;
  const int ctx = (int)min((int64_t)max(p.seq_lens[w.seq], 0), held);
  w.place0 = ctx - n;
  const int first = w.place0 + div(w.row0, p.group);
  const int last = w.place0 + div(min(w.row0 + tile_rows, w.rows) - 1, p.group);
  w.key_end = max(last + 1, 0);
  w.key_from = p.window ? max(first - p.window + 1, 0) : 0;
  w.first_tile = w.key_from / KEYS;
  w.sink_tiles = min((min(p.sinks, w.key_end) + KEYS - 1) / KEYS, w.first_tile);
  const int tiles = w.key_end > 0 ? w.sink_tiles + (w.key_end + KEYS - 1) / KEYS - w.first_tile : 0;
  w.t0 = (int)((int64_t)tiles * w.split / p.splits);
  w.t1 = (int)((int64_t)tiles * (w.split + 1) / p.splits);
  return true;
}

// The key whose row is loaded for key j: j itself where some row of the tile sees it, else one
// that is seen.  So nothing is read past a sequence's end or from pages that left the window;
// the weights of such places are zero, and a visible row times zero stays zero.
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
  bool live;
};
__device__ __forceinline__ Row get_row(const AttnParams& p, const Work& w, int r) {
  Row o;
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

// O^T += V^T P^T over NB blocks of 32 keys of the V tile at `v` (LDS bytes).
template <int D, int NB>
__device__ __forceinline__ void product_v(State<D>& st, const v8bf (&w)[NB][2], const uint8_t* v, int lane) {
  const int r = (lane & 15) >> 2, h = lane >> 5;
  // lane's 8 bytes within a 4-row, 32-byte group: row r, 8-byte piece lane % 4; the second 16
  // lanes of a half wave take the next 32 bytes
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = 32 * b + 16 * u + 4 * h + r;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) {
        const int chunk = v_chunk<D>(row, 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1));
        const int at = row * 2 * D + chunk * 16 + (lane & 1) * 8;
        const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LDS v4s*)(v + at));
        const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LDS v4s*)(v + at + 8 * 2 * D));
        const v8s a = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        st.o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), w[b][u], st.o[d], 0, 0, 0);
      }
    }
}

// A part's result, or the final one where there is a single part.  Register i of 16-group d is
// value 32 d + 8 (i / 4) + 4 (lane / 32) + i % 4.  z: summed over the half waves.
template <int D>
__device__ __forceinline__ void store_row(const AttnParams& p, const Work& w, const Row& row, const v16f (&o)[D / 32],
                                          float m, float z, int h) {
  if (!row.live) return;
  const int64_t idx = (int64_t)row.token * p.num_q_heads + row.head;
  if (p.splits == 1) {
    const float f = z > 0.f ? 1.f / z : (z == z ? 0.f : z);
    uint16_t* dst = p.out + row.token * p.o_token_stride + row.head * p.o_head_stride;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(v2u*)(dst + 32 * d + 8 * j + 4 * h) = (v2u){pack2(o[d][4 * j] * f, o[d][4 * j + 1] * f),
                                                      pack2(o[d][4 * j + 2] * f, o[d][4 * j + 3] * f)};
    if (p.lse && h == 0) p.lse[idx] = z > 0.f ? (m + __log2f(z)) * 0.6931471805599453f : (z == z ? NEG_INF : z);
  } else {
    const int64_t at = (int64_t)w.split * p.total_q * p.num_q_heads + idx;
    float* dst = p.part_o + at * D;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(v4f*)(dst + 32 * d + 8 * j + 4 * h) = (v4f){o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
    if (h == 0) {
      p.part_ml[2 * at] = m;
      p.part_ml[2 * at + 1] = z;
    }
  }
}

// ---------------------------------------------------------------- many rows: chunks of a prompt
// NW waves of 32 query rows share tiles of KEYS keys.  What bounds it: a wave's tile of 64 keys takes 32
// matrix instructions of 32 cycles at D = 128 (1024 cycles; half of that at D = 64) and about as long on
// the vector unit, where 32 exponentials at a quarter of the rate are half of it.  Both units have to be
// kept busy by different waves.
//
// D = 128: eight waves, two on each SIMD, and the two halves of the workgroup take turns: while waves
// 0-3 are in the matrix phase of a tile (O^T += V^T P^T of the tile before, S^T of this one), waves 4-7
// are in the vector phase (the softmax) of theirs, half a tile behind, with a barrier after each phase.
// Measured on 2048 queries (32 heads, 8 key heads) over 8192 keys: 236 us; 269 us without turns; 300 us
// with turns but LDS reads one matrix instruction ahead instead of four.  D = 64 is bound by the vector
// unit, which a single half cannot fill: four waves without turns and three such workgroups a CU
// (61 us on 2 x 2048 queries in a window of 1024; with turns 74, eight waves without 70).  D = 256
// fills the registers with one wave a SIMD.
//
// Tiles lie widened in LDS.  With turns, in rings of three: stage i brings K of tile i + 2 and V of tile
// i + 1; a wave issues its loads at the end of its matrix phase of tile i, when its LDS reads are out
// (255 us when issued before them), and widens and stores them at the end of the vector phase, to slots
// last read in the matrix phases of tile i - 1.  Without turns, two slots, loads a whole tile ahead.
// A load unit is GR rows of K or of V (one 16-byte load a lane), dealt to the waves; where GR divides
// the page size and every row of a unit is seen, its address is scalar arithmetic on a page number out
// of 64 that the lanes hold, else it is found lane by lane.
template <int D>
struct Wide {
  static constexpr int NW = D == 128 ? 8 : 4, KEYS = D == 256 ? 32 : 64, NB = KEYS / 32;
  static constexpr bool TURNS = D == 128;
  static constexpr int ROWS_ALL = NW * ROWS, THREADS = NW * 64, TILE = KEYS * D * 2;  // TILE: bytes of a widened K or V tile
};

// The end of a phase; no instruction is moved from one phase to another.
__device__ __forceinline__ void phase_end() {
  __builtin_amdgcn_sched_barrier(0);
  __syncthreads();
  __builtin_amdgcn_sched_barrier(0);
}

template <int D>
__global__ void __launch_bounds__(Wide<D>::THREADS, D == 256 ? 1 : D == 64 ? 3 : 2) wide_kernel(const AttnParams p) {
  constexpr int NW = Wide<D>::NW, KEYS = Wide<D>::KEYS, NB = Wide<D>::NB, TILE = Wide<D>::TILE;
  constexpr int CH = D / 16, GR = 64 / CH, GROUPS = KEYS / GR, NU = 2 * GROUPS / NW;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][Wide<D>::TURNS ? 3 : 2][TILE];  // [K, V][slot]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  Work w;
  if (!get_work<KEYS>(p, Wide<D>::ROWS_ALL, w)) return;
  const Row row = get_row(p, w, w.row0 + wave * ROWS + (lane & 31));
  // the places of this wave's rows, for whole-tile decisions
  const int wr0 = w.row0 + wave * ROWS;
  const int place_lo = w.place0 + div(min(wr0, w.rows - 1), p.group);
  const int place_hi = w.place0 + div(min(wr0 + ROWS, w.rows) - 1, p.group);

  v8bf q[D / 16];
  {
    const uint16_t* src = p.q + row.token * p.q_token_stride + row.head * p.q_head_stride + 8 * h;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[i] = *(const v8bf*)(src + 16 * i);
  }
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
      a.code = (int64_t)(pg * (uint64_t)p.c.page_stride + head_at + off * (uint32_t)p.c.token_stride) + lane_at;
      a.sf = (int64_t)(pg * (uint64_t)p.c.sf_page_stride + head_sf + off * (uint32_t)p.c.sf_token_stride) + lane_sf;
    } else {
      const int j = key_to_load(w, p.sinks, j0 + r);
      const int col = div(j, p.c.page), off = j - col * p.c.page.d, pg = page_entry(p, table, col);
      a.code = pg * p.c.page_stride + head_at + off * p.c.token_stride + 16 * c;
      a.sf = pg * p.c.sf_page_stride + head_sf + off * p.c.sf_token_stride;
    }
    return a;
  };
  // With turns, a wave's V rows of a stage are its K rows of the stage before (except where it loads
  // only one of the two); without, they are of the same tile.
  constexpr bool TURNS = Wide<D>::TURNS;
  constexpr int NK = NU > 1 ? NU / 2 : 1;
  const bool only_v = NU == 1 && wave >= GROUPS;
  At at[NK];
  v4u raw[NU];      // a stage's codes
  uint32_t sf[NU];  // and their rows' scale codes
  auto fetch = [&](int i) {
    // (tiles past the list repeat its ends and are not read)
    const int key0 = w.tile_key(min(max(TURNS && only_v ? i + 1 : i + 2, w.t0), w.t1 - 1), KEYS);
    auto get_v = [&](int n) {
      raw[NU - NK + n] = *(const v4u*)(p.c.v + at[n].code);
      sf[NU - NK + n] = p.c.v_sf[at[n].sf];
    };
#pragma unroll
    for (int n = 0; n < NK; ++n) {
      if (NU > 1 && TURNS) get_v(n);
      at[n] = place_rows(key0 + (wave + n * NW) % GROUPS * GR);
      if (NU > 1 && !TURNS) get_v(n);
      raw[n] = *(const v4u*)((only_v ? p.c.v : p.c.k) + at[n].code);
      sf[n] = (only_v ? p.c.v_sf : p.c.k_sf)[at[n].sf];
    }
  };
  auto put = [&](uint8_t* k, uint8_t* v) {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const bool is_v = NU > 1 ? n >= NK : only_v;
      const int rr = (wave + n * NW) % GROUPS * GR + r;
      uint8_t* dst = (is_v ? v : k) + rr * 2 * D;
      const int c0 = is_v ? v_chunk<D>(rr, 2 * c) : k_chunk<D>(rr, 2 * c), c1 = is_v ? v_chunk<D>(rr, 2 * c + 1) : k_chunk<D>(rr, 2 * c + 1);
      const float s = __uint_as_float(sf[n] << 23);
      *(v4u*)(dst + c0 * 16) = widen8(raw[n].x, raw[n].y, s);
      *(v4u*)(dst + c1 * 16) = widen8(raw[n].z, raw[n].w, s);
    }
  };

  State<D> st;
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
    softmax<D, NB>(p, st, s, wt);
  };
  // With turns: tile i of the list, number X of three: its K is in slot X, V of the tile before in slot X - 1.
  auto step = [&](int i, auto number) {
    constexpr int X = decltype(number)::value, NEXT = (X + 1) % 3, LAST = (X + 2) % 3;
    product_v<D, NB>(st, wt, lds[1][LAST], lane);
    v16f s[NB];
    scores(s, lds[0][X]);
    // Four fragments are read ahead of the matrix instruction that takes them.
    constexpr int NVF = D / 32 * NB * 2, NKF = D / 16 * NB, AHEAD = 4;  // V and K fragments (and matrix instructions)
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
    fetch(i);
    phase_end();
    weights(i, s);
    // (the weights are wanted here: left to itself, the compiler computes some in the next phase)
#pragma unroll
    for (int b = 0; b < NB; ++b) asm volatile("" : "+v"(wt[b][0]), "+v"(wt[b][1]));
    asm volatile("" : "+v"(st.z));
    __builtin_amdgcn_sched_barrier(0);
    put(lds[0][LAST], lds[1][NEXT]);
    phase_end();
  };
  // Without turns: tile i with K and V in slot X; leaves tile i + 1 in the other slot and tile i + 2 on its way.
  auto plain_step = [&](int i, auto slot) {
    constexpr int X = decltype(slot)::value, AHEAD = 3;
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
    product_v<D, NB>(st, wt, lds[1][X], lane);
    put(lds[0][1 - X], lds[1][1 - X]);
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * AHEAD, 1);
#pragma unroll
    for (int x = 0; x < D / 16 * NB - AHEAD; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 1);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, AHEAD, 1);
    __builtin_amdgcn_sched_barrier(0);
    fetch(i);
    __syncthreads();
  };
  if (w.t0 < w.t1) {
#pragma unroll
    for (int n = 0; n < NK; ++n) at[n] = place_rows(w.tile_key(w.t0, KEYS) + (wave + n * NW) % GROUPS * GR);
    fetch(w.t0 - 2);
    if constexpr (TURNS) {
      put(lds[0][0], lds[1][2]);
      fetch(w.t0 - 1);
      put(lds[0][1], lds[1][0]);
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
      product_v<D, NB>(st, wt, lds[1][last], lane);
      if (wave < 4) __syncthreads();
    } else {
      put(lds[0][0], lds[1][0]);
      fetch(w.t0 - 1);
      __syncthreads();
      for (int i = w.t0; i < w.t1; i += 2) {
        plain_step(i, Int<0>{});
        if (i + 1 < w.t1) plain_step(i + 1, Int<1>{});
      }
    }
  }
  store_row<D>(p, w, row, st.o, st.m, both_sum(st.z), h);
}

// ---------------------------------------------------------------- few rows: single tokens
// The four waves share up to 32 query rows and take the key tiles (32 keys) in turn.  A wave reads
// K straight into operand registers (the order of D within the contraction is free: half wave h
// takes bytes 16 h.. of every 32), stages V in its own LDS slice for the transposing reads, and
// keeps the next tile's loads in flight.  The waves' sums are joined at the end.
template <int D>
__global__ void __launch_bounds__(256) narrow_kernel(const AttnParams p) {
  constexpr int KEYS = 32, NW = 4, TILE = KEYS * D * 2;
  constexpr int CH = D / 16, PASS = 64 / CH, NP = KEYS / PASS;
  constexpr int JD = 64;  // values of D joined at once
  constexpr int JOIN = NW * ROWS * (JD + 4) * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[NW * TILE > JOIN ? NW * TILE : JOIN];
  __shared__ float ml[NW][2][ROWS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  Work w;
  if (!get_work<KEYS>(p, kAttnNarrowRows, w)) return;
  const Row row = get_row(p, w, w.row0 + (lane & 31));
  const int place_lo = w.place0 + div(w.row0, p.group);
  const int place_hi = w.place0 + div(min(w.row0 + ROWS, w.rows) - 1, p.group);
  v8bf q[D / 16];
  {
    const uint16_t* src = p.q + row.token * p.q_token_stride + row.head * p.q_head_stride + 16 * h;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      q[2 * i] = *(const v8bf*)(src + 32 * i);
      q[2 * i + 1] = *(const v8bf*)(src + 32 * i + 8);
    }
  }
  const int32_t* table = p.table + w.seq * p.table_stride;
  const int64_t head_at = w.kv_head * p.c.head_stride;
  uint8_t* vt = lds + wave * TILE;
  v4u kr[D / 32], vr[NP];
  uint32_t ks, vs[NP];
  auto fetch = [&](int i) {
    // lane and lane + 32 look the page of key lane % 32 up; V's rows take it from there
    const int j = key_to_load(w, p.sinks, w.tile_key(i, KEYS) + (lane & 31));
    const int col = div(j, p.c.page), off = j - col * p.c.page.d, pg = page_entry(p, table, col);
    const uint8_t* k = p.c.k + pg * p.c.page_stride + head_at + off * p.c.token_stride + 16 * h;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) kr[x] = *(const v4u*)(k + 32 * x);
    ks = p.c.k_sf[pg * p.c.sf_page_stride + w.kv_head * p.c.sf_head_stride + off * p.c.sf_token_stride];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int r = lane / CH + n * PASS;
      const int vpg = __shfl(pg, r), voff = __shfl(off, r);
      vr[n] = *(const v4u*)(p.c.v + vpg * p.c.page_stride + head_at + voff * p.c.token_stride + 16 * (lane % CH));
      vs[n] = p.c.v_sf[vpg * p.c.sf_page_stride + w.kv_head * p.c.sf_head_stride + voff * p.c.sf_token_stride];
    }
  };
  State<D> st;
  init(st);
  int i = w.t0 + wave;
  if (i < w.t1) fetch(i);
  for (; i < w.t1; i += NW) {
    const int key0 = w.tile_key(i, KEYS);
    v16f s[1];
#pragma unroll
    for (int x = 0; x < 16; ++x) s[0][x] = 0.f;
    const float a = __uint_as_float(ks << 23);
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      s[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, widen8(kr[x].x, kr[x].y, a)), q[2 * x], s[0], 0, 0, 0);
      s[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, widen8(kr[x].z, kr[x].w, a)), q[2 * x + 1], s[0], 0, 0, 0);
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int r = lane / CH + n * PASS, c = lane % CH;
      const float b = __uint_as_float(vs[n] << 23);
      *(v4u*)(vt + r * 2 * D + v_chunk<D>(r, 2 * c) * 16) = widen8(vr[n].x, vr[n].y, b);
      *(v4u*)(vt + r * 2 * D + v_chunk<D>(r, 2 * c + 1) * 16) = widen8(vr[n].z, vr[n].w, b);
    }
    if (i + NW < w.t1) fetch(i + NW);
    v8bf wt[1][2];
    const bool late = key0 + KEYS - 1 > place_lo, early = p.window && key0 <= place_hi - p.window && key0 + KEYS > p.sinks;
    if (late || early) mask<1>(p, s, key0, row.place, h, late, early);
    softmax<D, 1>(p, st, s, wt);
    // the wave reads what its other lanes wrote: its LDS operations complete in order, so only the
    // compiler has to keep theirs
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    product_v<D, 1>(st, wt, vt, lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  // join: rescale to the common maximum, add up through LDS
  const float z = both_sum(st.z);
  if (h == 0) {
    ml[wave][0][lane] = st.m;
    ml[wave][1][lane] = z;
  }
  __syncthreads();
  float m = NEG_INF, zz = 0.f;
#pragma unroll
  for (int x = 0; x < NW; ++x) m = fmaxf(m, ml[x][0][lane & 31]);
#pragma unroll
  for (int x = 0; x < NW; ++x) {
    const float mx = ml[x][0][lane & 31];
    zz += (m == NEG_INF ? 1.f : exp2_hw(mx - m)) * ml[x][1][lane & 31];
  }
  const float f = m == NEG_INF ? 1.f : exp2_hw(st.m - m);
  float* jo = (float*)lds;
  // JD values of D at a time: every wave puts its part, wave x adds up and keeps 32-value group x
  const int64_t idx = (int64_t)row.token * p.num_q_heads + row.head;
#pragma unroll
  for (int d0 = 0; d0 < D / 32; d0 += JD / 32) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < JD / 32; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(v4f*)(jo + (wave * ROWS + (lane & 31)) * (JD + 4) + 32 * d + 8 * j + 4 * h) =
            (v4f){st.o[d0 + d][4 * j] * f, st.o[d0 + d][4 * j + 1] * f, st.o[d0 + d][4 * j + 2] * f, st.o[d0 + d][4 * j + 3] * f};
    __syncthreads();
    // wave x, half h: values 16 x + 8 h .. + 7 of the JD
    v4f a[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int x = 0; x < NW; ++x) {
      const float* src = jo + (x * ROWS + (lane & 31)) * (JD + 4) + 16 * wave + 8 * h;
      a[0] += *(const v4f*)src;
      a[1] += *(const v4f*)(src + 4);
    }
    if (row.live) {
      const int d = 32 * d0 + 16 * wave + 8 * h;
      if (p.splits == 1) {
        const float g = zz > 0.f ? 1.f / zz : (zz == zz ? 0.f : zz);
        *(v4u*)(p.out + row.token * p.o_token_stride + row.head * p.o_head_stride + d) =
            (v4u){pack2(a[0].x * g, a[0].y * g), pack2(a[0].z * g, a[0].w * g), pack2(a[1].x * g, a[1].y * g),
                  pack2(a[1].z * g, a[1].w * g)};
      } else {
        float* dst = p.part_o + ((int64_t)w.split * p.total_q * p.num_q_heads + idx) * D + d;
        *(v4f*)dst = a[0];
        *(v4f*)(dst + 4) = a[1];
      }
    }
  }
  if (row.live && wave == 0 && h == 0) {
    if (p.splits > 1) {
      const int64_t at = (int64_t)w.split * p.total_q * p.num_q_heads + idx;
      p.part_ml[2 * at] = m;
      p.part_ml[2 * at + 1] = zz;
    } else if (p.lse) {
      p.lse[idx] = zz > 0.f ? (m + __log2f(zz)) * 0.6931471805599453f : (zz == zz ? NEG_INF : zz);
    }
  }
}

// ---------------------------------------------------------------- joining the parts
// One wave per (token, head): out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) z_s.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const AttnParams p) {
  constexpr int E = D / 64;  // values of a lane
  const int64_t rows = (int64_t)p.total_q * p.num_q_heads;
  const int64_t idx = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (idx >= rows) return;
  const int token = (int)(idx / p.num_q_heads), head = (int)(idx - (int64_t)token * p.num_q_heads);
  if (p.cu_q && (token < p.cu_q[0] || token >= p.cu_q[p.batch])) return;  // rows of no sequence
  float m = NEG_INF;
  for (int s = 0; s < p.splits; ++s) m = fmaxf(m, p.part_ml[2 * (s * rows + idx)]);
  float z = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const int64_t at = s * rows + idx;
    const float ms = p.part_ml[2 * at];
    if (ms == NEG_INF) continue;  // (a part without keys)
    const float f = exp2_hw(ms - m);
    z += f * p.part_ml[2 * at + 1];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += f * p.part_o[at * D + E * lane + e];
  }
  const float g = z > 0.f ? 1.f / z : (z == z ? 0.f : z);
  uint16_t* dst = p.out + token * p.o_token_stride + head * p.o_head_stride + E * lane;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = __builtin_bit_cast(uint16_t, (__bf16)(o[e] * g));
  if (p.lse && lane == 0) p.lse[idx] = z > 0.f ? (m + __log2f(z)) * 0.6931471805599453f : (z == z ? NEG_INF : z);
}

template <int D>
hipError_t launch(const AttnParams& p, bool wide, hipStream_t stream) {
  const int64_t grid = (int64_t)p.batch * p.c.num_heads * p.q_tiles * p.splits;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  if (wide)
    hipLaunchKernelGGL((wide_kernel<D>), dim3((unsigned)grid), dim3(Wide<D>::THREADS), 0, stream, p);
  else
    hipLaunchKernelGGL((narrow_kernel<D>), dim3((unsigned)grid), dim3(256), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)p.total_q * p.num_q_heads;
  hipLaunchKernelGGL((join_kernel<D>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace attn

hipError_t launch_attention(const AttnParams& p, int head_dim, bool wide, hipStream_t stream) {
  if (head_dim == 64) return attn::launch<64>(p, wide, stream);
  if (head_dim == 128) return attn::launch<128>(p, wide, stream);
  if (head_dim == 256) return attn::launch<256>(p, wide, stream);
  return hipErrorInvalidValue;
}

}  // namespace dg
