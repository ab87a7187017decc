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
// lanes read 4 rows x 32 bytes, and the next 16 lanes the 32 bytes beside them.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
  return c ^ (D == 64 ? (row >> 1) & 7 : row & 15);
}
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
  return c ^ (D == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2);
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
  // Workgroups are dealt to the eight XCDs in turn; renumber them so that each XCD takes a
  // contiguous run, and with it all parts of the same keys: they share its L2.
  const unsigned nb = gridDim.x, per = nb >> 3, extra = nb & 7, xcd = blockIdx.x & 7, idx = blockIdx.x >> 3;
  unsigned id = xcd < extra ? xcd * (per + 1) + idx : extra * (per + 1) + (xcd - extra) * per + idx;
  w.split = id % p.splits;
  id /= p.splits;
  const int qt = p.q_tiles - 1 - (int)(id % p.q_tiles);  // (later rows see more keys: they start first)
  id /= p.q_tiles;
  w.kv_head = id % p.c.num_heads;
  w.seq = id / p.c.num_heads;
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

// Scores of NB blocks of 32 keys -> weights (as B operands of the second product), updating the
// running maximum, sum and, where the maximum rises, the outputs.  key0: first key.
// A lane's register i of a block is key 8 (i / 4) + 4 (lane / 32) + i % 4.
template <int D, int NB, bool MASK>
__device__ __forceinline__ void softmax(const AttnParams& p, State<D>& st, v16f (&s)[NB], v8bf (&w)[NB][2], int key0, int place,
                                        int h) {
  if constexpr (MASK) {
    const int from = p.window ? place - p.window : INT32_MIN;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = key0 + 32 * b + 8 * (i / 4) + 4 * h + i % 4;
        const bool seen = j <= place && (j > from || j < p.sinks);
        s[b][i] = seen ? s[b][i] : NEG_INF;
      }
  }
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
// Four waves of 32 query rows share tiles of 64 keys.  A tile's codes are loaded into registers
// while the one before is computed, widened once, and written to the other of two LDS buffers.
template <int D>
__global__ void __launch_bounds__(256) wide_kernel(const AttnParams p) {
  constexpr int KEYS = D == 256 ? 32 : 64, NB = KEYS / 32, TILE = KEYS * D * 2;  // bytes of a widened tile
  constexpr int CH = D / 16, PASS = 256 / CH, NP = KEYS / PASS;  // 16-code chunks; rows and number of load passes
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][2][TILE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  Work w;
  if (!get_work<KEYS>(p, kAttnWideRows, w)) return;
  const Row row = get_row(p, w, w.row0 + wave * ROWS + (lane & 31));
  // the places of this wave's rows, for whole-tile decisions
  const int wr0 = w.row0 + wave * ROWS;
  const int place_lo = w.place0 + div(min(wr0, w.rows - 1), p.group);
  const int place_hi = wr0 < w.rows ? w.place0 + div(min(wr0 + ROWS, w.rows) - 1, p.group) : INT32_MIN / 2;

  v8bf q[D / 16];
  {
    const uint16_t* src = p.q + row.token * p.q_token_stride + row.head * p.q_head_stride + 8 * h;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[i] = *(const v8bf*)(src + 16 * i);
  }
  const int32_t* table = p.table + w.seq * p.table_stride;
  const int c = threadIdx.x % CH, r0 = threadIdx.x / CH;
  v4u kr[NP], vr[NP];
  uint32_t ks[NP], vs[NP];
  auto fetch = [&](int i) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int j = key_to_load(w, p.sinks, w.tile_key(i, KEYS) + r0 + n * PASS);
      const int col = div(j, p.c.page), off = j - col * p.c.page.d, pg = page_entry(p, table, col);
      const int64_t at = pg * p.c.page_stride + w.kv_head * p.c.head_stride + off * p.c.token_stride + 16 * c;
      const int64_t sf = pg * p.c.sf_page_stride + w.kv_head * p.c.sf_head_stride + off * p.c.sf_token_stride;
      kr[n] = *(const v4u*)(p.c.k + at);
      vr[n] = *(const v4u*)(p.c.v + at);
      ks[n] = p.c.k_sf[sf];
      vs[n] = p.c.v_sf[sf];
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int r = r0 + n * PASS;
      const float a = __uint_as_float(ks[n] << 23), b = __uint_as_float(vs[n] << 23);
      uint8_t* k = lds[buf][0] + r * 2 * D;
      uint8_t* v = lds[buf][1] + r * 2 * D;
      *(v4u*)(k + k_chunk<D>(r, 2 * c) * 16) = widen8(kr[n].x, kr[n].y, a);
      *(v4u*)(k + k_chunk<D>(r, 2 * c + 1) * 16) = widen8(kr[n].z, kr[n].w, a);
      *(v4u*)(v + v_chunk<D>(r, 2 * c) * 16) = widen8(vr[n].x, vr[n].y, b);
      *(v4u*)(v + v_chunk<D>(r, 2 * c + 1) * 16) = widen8(vr[n].z, vr[n].w, b);
    }
  };

  State<D> st;
  init(st);
  if (w.t0 < w.t1) {
    fetch(w.t0);
    put(0);
    if (w.t0 + 1 < w.t1) fetch(w.t0 + 1);
  }
  __syncthreads();
  for (int i = w.t0; i < w.t1; ++i) {
    const int buf = (i - w.t0) & 1, key0 = w.tile_key(i, KEYS);
    // a tile that none of the wave's rows sees is left out (tiles above the diagonal, and tiles
    // between the first keys and the window)
    const bool none = key0 > place_hi || (p.window && key0 + KEYS - 1 <= place_lo - p.window && key0 >= p.sinks);
    if (!none) {
      v16f s[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int x = 0; x < 16; ++x) s[b][x] = 0.f;
        const int r = 32 * b + (lane & 31);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const v8bf a = *(const v8bf*)(lds[buf][0] + r * 2 * D + k_chunk<D>(r, 2 * x + h) * 16);
          s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[x], s[b], 0, 0, 0);
        }
      }
      v8bf wt[NB][2];
      const bool all = key0 + KEYS - 1 <= place_lo && (!p.window || key0 > place_hi - p.window || key0 + KEYS <= p.sinks);
      if (all)
        softmax<D, NB, false>(p, st, s, wt, key0, row.place, h);
      else
        softmax<D, NB, true>(p, st, s, wt, key0, row.place, h);
      product_v<D, NB>(st, wt, lds[buf][1], lane);
    }
    if (i + 1 < w.t1) {
      put(buf ^ 1);
      if (i + 2 < w.t1) fetch(i + 2);
    }
    __syncthreads();
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
    const bool all = key0 + KEYS - 1 <= place_lo && (!p.window || key0 > place_hi - p.window || key0 + KEYS <= p.sinks);
    if (all)
      softmax<D, 1, false>(p, st, s, wt, key0, row.place, h);
    else
      softmax<D, 1, true>(p, st, s, wt, key0, row.place, h);
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
    hipLaunchKernelGGL((wide_kernel<D>), dim3((unsigned)grid), dim3(256), 0, stream, p);
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
