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
// The entries of a tile's lists go 64 to a wave at a time, one a lane: a lane looks its block up in the other tokens' lists (they
// ascend), and drops it where an earlier one has it.  The remaining ones, in segments of 64 tokens, are dealt
// in turn to the waves of the tile's workgroups, which find their own without asking each other.
#include "dg_attn_device.h"

namespace dg {
namespace sparse {

using namespace attn;

constexpr int SEGMENT = 64;

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

// A tile's entries of the blocks' lists, 64 of the tile's at a time.
struct Entries {
  int block, page;  // this lane's: its block, its page of the cache
  unsigned tokens;  // whose lists have it, by bits; 0: none, or an earlier entry stands for it
  int number;       // number among the entries that stand
};

// The first of `top` ascending numbers (negative ones, at the end, count as larger than all) that is not below v: whether it is v.
__device__ __forceinline__ bool has(const int32_t* list, int top, int v) {
  int at = 0, n = top;
  while (n > 0) {
    const int half = n >> 1, x = list[at + half];
    if (x >= 0 && x < v) {
      at += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  return at < top && list[at] == v;
}

// SHARED: several tokens, whose lists lie one after the other in LDS; else the one token's list in memory.
template <bool SHARED>
__device__ __forceinline__ void load_entries(const SparseParams& p, const Tile& t, const int32_t* lists, int from, int before, Entries& e) {
  const int lane = threadIdx.x & 63, i = from + lane;
  e.tokens = 0;
  e.block = e.page = 0;
  if (i < t.tokens * p.top) {
    const int b = lists[i];
    // (blocks past the tile's last token hold no key that counts)
    if (b >= 0 && b < p.s.table_cols && b * p.c.page.d < t.key_end) {
      unsigned tokens = 1u;
      if (SHARED) {
        const int mine = div(i, p.list);
        tokens = 1u << mine;
        for (int x = 0; x < t.tokens; ++x)
          if (x != mine && has(lists + x * p.top, p.top, b)) tokens |= 1u << x;
        if (tokens & ((1u << mine) - 1)) tokens = 0;
      }
      if (tokens) {
        const int pg = p.s.table[t.seq * p.s.table_stride + b];
        e.tokens = tokens;
        e.block = b;
        e.page = (unsigned)pg < (unsigned)p.c.num_pages ? pg : 0;  // (the host cannot see the table's contents)
      }
    }
  }
  e.number = before + (int)__popcll(__ballot(e.tokens != 0) & ((1ull << lane) - 1));
}

// 16 keys of one block.
struct Half {
  int page, offset, key0;  // place of the first key within its page, and in the sequence
  int keys;                // how many there are (0: none)
  unsigned tokens;
};

// A wave's segments, 16 keys at a time.  `share` of `shares` (a power of two).
struct Walk {
  Entries e;
  uint64_t left;           // lanes whose entries are still to come
  int from, before;        // next entries, and the number of those that stand before them
  int block, page, segment, offset, end;  // the present entry; place within its page
  unsigned tokens;
};

template <bool SHARED>
__device__ __forceinline__ bool next_segment(const SparseParams& p, const Tile& t, const int32_t* lists, int segments, int share, int shares, Walk& w) {
  w.segment += shares;
  while (w.segment >= segments) {
    while (!w.left) {
      if (w.from >= t.tokens * p.top) return false;
      load_entries<SHARED>(p, t, lists, w.from, w.before, w.e);
      w.from += 64;
      w.before += (int)__popcll(__ballot(w.e.tokens != 0));
      // segment s of entry n is number n * segments + s
      w.left = __ballot(w.e.tokens != 0 && (int)((unsigned)(share - w.e.number * segments) & (unsigned)(shares - 1)) < segments);
    }
    const int l = __builtin_ctzll(w.left);
    w.left &= w.left - 1;
    w.block = __builtin_amdgcn_readlane(w.e.block, l);
    w.page = __builtin_amdgcn_readlane(w.e.page, l);
    w.tokens = (unsigned)__builtin_amdgcn_readlane((int)w.e.tokens, l);
    w.segment = (share - __builtin_amdgcn_readlane(w.e.number, l) * segments) & (shares - 1);
  }
  return true;
}

template <int D, bool SHARED, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, D == 256 ? 1 : 2) sparse_kernel(const SparseParams p) {
  constexpr int KEYS = 32, TILE = KEYS * D * 2;
  constexpr int CH = D / 16, PASS = 64 / CH, NP = KEYS / PASS;  // V: 16-code chunks of a row, rows of a load, loads
  constexpr int JD = 64;                                        // values of D joined at once
  constexpr int JOIN = WAVES * 16 * (JD + 4) * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[WAVES * TILE > JOIN ? WAVES * TILE : JOIN];
  __shared__ float mz[WAVES][2][16];
  extern __shared__ int32_t tile_lists[];  // [tile_tokens][top] (SHARED)
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), g = lane >> 4, col = lane & 15;
  uint8_t* vt = lds + wave * TILE;
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
  const int32_t* lists = p.blocks + (int64_t)t.first_row * list_stride + t.kv_head * p.top;
  if (SHARED) {
    for (int i = threadIdx.x; i < t.tokens * p.top; i += WAVES * 64) {
      const int x = div(i, p.list);
      tile_lists[i] = lists[x * list_stride + i - x * p.top];
    }
    __syncthreads();
    lists = tile_lists;
  }
  const int segments = (p.c.page.d + SEGMENT - 1) / SEGMENT, shares = WAVES * p.parts, share = t.part * WAVES + wave;
  const int64_t head_at = t.kv_head * p.c.head_stride, head_sf = t.kv_head * p.c.sf_head_stride;
  const unsigned every = (1u << t.tokens) - 1;

  Walk w;
  // the next 16 keys of the wave's share
  auto next_half = [&](Half& h) {
    if (w.offset >= w.end) {
      if (!next_segment<SHARED>(p, t, lists, segments, share, shares, w)) {
        h.keys = 0;
        h.tokens = 0;
        return;
      }
      w.offset = w.segment * SEGMENT;
      w.end = min(min(p.c.page.d, w.offset + SEGMENT), t.key_end - w.block * p.c.page.d);
      if (w.end <= w.offset) {  // (a segment past the last token's place)
        h.keys = -1;
        return;
      }
    }
    h.page = w.page;
    h.offset = w.offset;
    h.key0 = w.block * p.c.page.d + w.offset;
    h.keys = min(16, w.end - w.offset);
    h.tokens = w.tokens;
    w.offset += 16;
  };
  auto start = [&]() {
    w.left = 0;
    w.from = w.before = 0;
    w.segment = segments;
    w.offset = w.end = 0;
  };
  // the next 32: two halves, the second one maybe empty (a copy of the first then, which no query sees)
  auto next_tile = [&](Half (&h)[2]) {
    do next_half(h[0]);
    while (h[0].keys < 0);
    if (h[0].keys == 0) return false;
    do next_half(h[1]);
    while (h[1].keys < 0);
    if (h[1].keys == 0) {
      h[1] = h[0];
      h[1].tokens = 0;
    }
    return true;
  };

  v4u kr[2][D / 64], vr[NP];
  uint32_t ks[2], vs[NP];
  // (through buffer descriptors of the pages, whose addresses are scalar)
  auto fetch_k = [&](const Half (&h)[2]) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int off = h[x].offset + min(col, h[x].keys - 1);
      const __amdgpu_buffer_rsrc_t codes = rsrc(p.c.k + h[x].page * p.c.page_stride + head_at), sf = rsrc(p.c.k_sf + h[x].page * p.c.sf_page_stride + head_sf);
#pragma unroll
      for (int y = 0; y < D / 64; ++y) kr[x][y] = __builtin_amdgcn_raw_buffer_load_b128(codes, off * (int)p.c.token_stride + 16 * g + 64 * y, 0, 0);
      ks[x] = __builtin_amdgcn_raw_buffer_load_b8(sf, off * (int)p.c.sf_token_stride, 0, 0);
    }
  };
  auto fetch_v = [&](const Half (&h)[2]) {
    __amdgpu_buffer_rsrc_t codes[2], sf[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) codes[x] = rsrc(p.c.v + h[x].page * p.c.page_stride + head_at), sf[x] = rsrc(p.c.v_sf + h[x].page * p.c.sf_page_stride + head_sf);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int r = n * PASS + lane / CH, x = n * PASS / 16;  // (a load's rows are in one half)
      const int off = h[x].offset + min(r & 15, h[x].keys - 1);
      vr[n] = __builtin_amdgcn_raw_buffer_load_b128(codes[x], off * (int)p.c.token_stride + 16 * (lane % CH), 0, 0);
      vs[n] = __builtin_amdgcn_raw_buffer_load_b8(sf[x], off * (int)p.c.sf_token_stride, 0, 0);
    }
  };

  v4f o[D / 16];
  float m, z;
  // A hidden value's weight is zero, which is not enough where it is NaN or infinite.  Nobody looks for such values at first: they
  // leave a NaN in some output.  A wave that ends with an output that is no number goes over its keys again with care: what is no number among the values
  // that some row does not see goes to LDS as zero, and is added at the end to the outputs of the rows that see it.
  bool odd = false;  // the wave has cleared a value
  Half now[2], next[2];
#pragma unroll 1
  for (int careful = 0;; ++careful) {
  m = NEG_INF, z = 0.f;
#pragma unroll
  for (int d = 0; d < D / 16; ++d) o[d] = (v4f){0.f, 0.f, 0.f, 0.f};
  start();
  bool more = next_tile(now);
  if (more) {
    fetch_k(now);
    fetch_v(now);
  }
  while (more) {
    more = next_tile(next);
    v4f s[2];
    s[0] = s[1] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float scale = __uint_as_float(ks[x] << 23);
#pragma unroll
      for (int y = 0; y < D / 64; ++y) {
        const v8bf lo = __builtin_bit_cast(v8bf, widen8(kr[x][y].x, kr[x][y].y, scale));
        const v8bf hi = __builtin_bit_cast(v8bf, widen8(kr[x][y].z, kr[x][y].w, scale));
        s[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, q[2 * y], s[x], 0, 0, 0);
        s[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, q[2 * y + 1], s[x], 0, 0, 0);
      }
    }
    if (more) fetch_k(next);
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      const int r = lane / CH + n * PASS, c = lane % CH;
      const float scale = __uint_as_float(vs[n] << 23);
      *(v4u*)(vt + r * 2 * D + narrow_chunk<D>(r, 2 * c) * 16) = widen8(vr[n].x, vr[n].y, scale);
      *(v4u*)(vt + r * 2 * D + narrow_chunk<D>(r, 2 * c + 1) * 16) = widen8(vr[n].z, vr[n].w, scale);
    }
    // whether every row sees all 32 keys
    const bool whole = now[0].tokens == every && now[1].tokens == every && now[0].keys == 16 && now[1].keys == 16 &&
                       now[0].key0 + 15 <= t.place0 && now[1].key0 + 15 <= t.place0;
    if (!whole) {
      if (__builtin_expect(careful, 0)) {
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
      // keys of each half that the lane's query sees: the first `count`
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int count = now[x].tokens >> row.token & 1 ? min(now[x].keys, place - now[x].key0 + 1) - 4 * g : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[x][e] = e < count ? s[x][e] : NEG_INF;
      }
    }
    if (more) fetch_v(next);
    float top = s[0][0];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, s[x][e]);
    top = groups_max(top) * p.scale_log2;  // (the scale is positive)
    if (__any(top > m + SLACK)) {
      const float raised = fmaxf(m, top);
      const float f = raised == NEG_INF ? 1.f : exp2_hw(m - raised);
      m = raised;
      z *= f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[d] *= f;
    }
    const float sub = m == NEG_INF ? 0.f : -m;  // nothing seen yet: every weight is 2^-inf = 0
    v4u x4;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[x][e] = exp2_hw(__builtin_fmaf(s[x][e], p.scale_log2, sub));
        z += s[x][e];
      }
      x4[2 * x] = pack2(s[x][0], s[x][1]);
      x4[2 * x + 1] = pack2(s[x][2], s[x][3]);
    }
    const v8bf wt = __builtin_bit_cast(v8bf, x4);
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
      o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), wt, o[d], 0, 0, 0);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    now[0] = next[0];
    now[1] = next[1];
  }
    if (careful) break;
    float sum = 0.f;  // (a NaN or infinity times zero is NaN)
#pragma unroll
    for (int d = 0; d < D / 16; ++d) sum += (o[d].x * 0.f + o[d].y * 0.f) + (o[d].z * 0.f + o[d].w * 0.f);
    if (__builtin_expect(!__any(sum != 0.f), 1)) break;
  }

  if (__builtin_expect(odd, 0)) {
    start();
    while (next_tile(now)) {
      if (now[0].tokens == every && now[1].tokens == every && now[0].keys == 16 && now[1].keys == 16 && now[0].key0 + 15 <= t.place0 &&
          now[1].key0 + 15 <= t.place0)
        continue;
      for (int x = 0; x < 2; ++x)
        for (int j = 0; j < now[x].keys; ++j) {
          const int off = now[x].offset + j;
          const uint8_t* codes = p.c.v + now[x].page * p.c.page_stride + head_at + off * p.c.token_stride;
          const uint32_t sf = p.c.v_sf[now[x].page * p.c.sf_page_stride + head_sf + off * p.c.sf_token_stride];
          const bool sees = (now[x].tokens >> row.token & 1) && now[x].key0 + j <= place;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const v4f add = odd_values(*(const unsigned*)(codes + 16 * d + 4 * g), sf);
            if (sees) o[d] += add;
          }
        }
    }
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
  constexpr int AT_ONCE = 4;  // (loads that go out together)
  for (int x = group; x < p.parts; x += G * AT_ONCE) {
    v2f a[AT_ONCE];
    v4f b[AT_ONCE];
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      a[u] = (v2f){NEG_INF, 0.f};
      if (x + u * G < p.parts) {
        const int64_t at = (t.slot + x + u * G) * 16 + r;
        a[u] = *(const v2f*)(p.part_mz + 2 * at);
        b[u] = *(const v4f*)(p.part_o + at * D + 4 * lanes);
      }
    }
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
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
  if (p.waves == 4 && p.tile_tokens > 1)
    hipLaunchKernelGGL((sparse_kernel<D, true, 4>), dim3(tiles * p.parts), dim3(256), lists, stream, p);
  else if (p.waves == 4)
    hipLaunchKernelGGL((sparse_kernel<D, false, 4>), dim3(tiles * p.parts), dim3(256), 0, stream, p);
  else if constexpr (D != 256) {
    if (p.tile_tokens > 1)
      hipLaunchKernelGGL((sparse_kernel<D, true, 8>), dim3(tiles * p.parts), dim3(512), lists, stream, p);
    else
      hipLaunchKernelGGL((sparse_kernel<D, false, 8>), dim3(tiles * p.parts), dim3(512), 0, stream, p);
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
