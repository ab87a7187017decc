// Block keys of the FP8 key/value cache's pages and the choice of blocks by them, for gfx950 (MI355X).
//
// A block is a page.  Its block key is, for each head, the mean of its keys as signed 8-bit codes and one power of two, the
// smallest p with |mean| <= 127 p.  A query of 8-bit codes made alike scores a block by the integer product of the codes
// times both scales: the products' sum stays below 2^22, so it is the same in any order, and so is the choice, to the
// last tie.
#include <type_traits>

#include "dg_attn_device.h"

namespace dg {
namespace blocks {

using attn::uniform;
using attn::v2f;
using attn::v2u;
using attn::v4u;
typedef int v4i __attribute__((ext_vector_type(4)));
typedef double v2d __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- block keys
// A wave has a page and head: D / 16 lanes a key of 16 codes each, 1024 / D keys at a time.  The sum is taken in 64 bits, where
// codes (multiples of 2^-9 up to 448) under scales of up to 2^25 apart add up without rounding.  Bound by reading
// the keys, for which four loads of a lane go out together (2047 pages of 64 keys and 8 heads of 128: 29 us, 4.6 TB/s; one at a time 40).
// Pages of 16 keys, 8188 of them: 67 us, bound by instructions (the vector units are busy for 90%): the sums' way through LDS, the mean and
// its codes cost the same for 2 KiB of keys as for 8 (469 vector instructions a wave, with 64 keys 718).
constexpr int KEYS_WAVES = 4;

template <int D>
__global__ void __launch_bounds__(KEYS_WAVES * 64) block_keys_kernel(const BlockKeysParams p) {
  constexpr int L = D / 16, ROWS = 64 / L, E = D / 64;  // lanes of a key, keys at a time, values of a lane at the end
  __shared__ __attribute__((aligned(16))) double sums[KEYS_WAVES][ROWS][D];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), l = lane % L, r = lane / L;
  const int heads = p.c.num_heads;
  const int64_t id = (int64_t)blockIdx.x * KEYS_WAVES + wave;
  const int entry = uniform((int)(id / heads)), head = uniform((int)(id - (int64_t)entry * heads));
  if (entry >= p.num_pages) return;
  const int page = uniform(p.pages[entry]);
  if ((unsigned)page >= (unsigned)p.c.num_pages) return;
  const uint8_t* codes = p.c.k + page * p.c.page_stride + head * p.c.head_stride + 16 * l;
  const uint8_t* sfs = p.c.k_sf + page * p.c.sf_page_stride + head * p.c.sf_head_stride;
  double s[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = 0.0;
  constexpr int TOGETHER = 4;  // loads that go out together
  for (int t0 = r; t0 < p.c.page.d; t0 += ROWS * TOGETHER) {
    v4u x[TOGETHER];
    uint32_t sf[TOGETHER];
    unsigned nan = 0;
#pragma unroll
    for (int u = 0; u < TOGETHER; ++u) {
      const int t = t0 + u * ROWS;
      x[u] = (v4u){0, 0, 0, 0};
      sf[u] = 127;
      if (t < p.c.page.d) {
        x[u] = *(const v4u*)(codes + t * p.c.token_stride);
        sf[u] = sfs[t * p.c.sf_token_stride];
      }
    }
#pragma unroll
    for (int u = 0; u < TOGETHER; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) nan |= (x[u][i] & 0x7F7F7F7Fu) + 0x01010101u;
    if (__builtin_expect(__any((nan & 0x80808080u) != 0), 0)) {  // a NaN counts as zero
#pragma unroll
      for (int u = 0; u < TOGETHER; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[u][i] &= ~(((((x[u][i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu);
    }
#pragma unroll
    for (int u = 0; u < TOGETHER; ++u) {
      const double scale = __hiloint2double((int)((sf[u] + 1023 - 127) << 20), 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[u][i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[u][i], true);
        s[4 * i] = __builtin_fma((double)lo.x, scale, s[4 * i]);
        s[4 * i + 1] = __builtin_fma((double)lo.y, scale, s[4 * i + 1]);
        s[4 * i + 2] = __builtin_fma((double)hi.x, scale, s[4 * i + 2]);
        s[4 * i + 3] = __builtin_fma((double)hi.y, scale, s[4 * i + 3]);
      }
    }
  }
#pragma unroll
  // (pairs of a lane's eight change places by the lane's number, so that lanes next to each other write to, and read from, different banks)
  for (int i = 0; i < 16; i += 2) *(v2d*)&sums[wave][r][16 * l + (i ^ 2 * (lane & 7))] = (v2d){s[i], s[i + 1]};
  // (the wave reads what its own lanes wrote: its LDS operations complete in order)
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  double mean[E];
  uint64_t top = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    mean[e] = 0.0;
#pragma unroll
    for (int x = 0; x < ROWS; ++x) mean[e] += sums[wave][x][(E * lane + e) ^ 2 * ((x * L + E * lane / 16) & 7)];
    mean[e] /= (double)p.c.page.d;
    top = max(top, (uint64_t)__double_as_longlong(__builtin_fabs(mean[e])));
  }
#pragma unroll
  for (int step = 1; step < 64; step *= 2) top = max(top, (uint64_t)__shfl_xor((unsigned long long)top, step));
  // 127 = 1.984375 * 2^6: the exponent of top's power of two, less 6, and one more where its mantissa is above that
  int e = (int)(top >> 52) - 1023 - 6 + ((top & 0xFFFFFFFFFFFFFull) > 0xFC00000000000ull ? 1 : 0);
  e = top == 0 ? 0 : min(max(e, -126), 127);
  const double inv = __hiloint2double((1023 - e) << 20, 0);
  const int64_t at = (int64_t)page * heads + head;
  int8_t* out = p.b.codes + at * D + E * lane;
#pragma unroll
  for (int i = 0; i < E; ++i) out[i] = (int8_t)min(max((int)__builtin_rint(mean[i] * inv), -127), 127);
  if (lane == 0) p.b.scales[at] = __uint_as_float((uint32_t)(e + 127) << 23);
}

// ---------------------------------------------------------------- choosing blocks
// A workgroup has a tile of tokens of one sequence and a key head.  Its waves score the blocks between the first and the last
// ones, 16 at a time: S = K Q^T on the 16 x 16 x 64 integer matrix instruction, a block key straight from memory into operand registers, the queries'
// codes as its 16 columns: a token takes 1, 2, 4, 8 or 16 of them (its group's heads, rounded up; more heads go 16 after 16).  The
// largest over a token's columns goes to LDS as a number that compares like the score.  Then a wave has a token: it
// finds the largest threshold that enough scores reach by bisection, a compare and a population count for 64 of them, and writes
// the chosen blocks in order.
//
// What bounds it: latency.  A workgroup's steps (queries to codes, keys through their pages' numbers, the choice) wait for each other; a chunk of
// 2048 tokens over 512 blocks (32 + 8 heads of 128) takes 44 us, 28 of them for the scores, with the vector units busy for half of the time.  The
// workgroup's 4 tiles of 16 columns take a block key from memory once (with 2 tiles 53 us; 8 need more registers than there are: 68), by 8 waves (with
// 4: 58).
//
// A token's scores all lie in LDS, with a place for each column of the table: a wide table leaves room for few tokens, and every tile reads all block
// keys.  The same chunk, over the same 512 blocks, takes 57 us with 1024 columns, 84 with 2048, 155 with 4096, 290 with 8192 and 550 with 16384 or
// 32768; single tokens 14 us with up to 8192 columns and 20 with more (64 sequences).
//
// Few sequences with many blocks leave most of the chip idle in that form.  There the scores go to memory, a slice of
// the blocks to a workgroup, and a second kernel with a wave for each token and key head chooses.

// The order of floats as unsigned numbers, none of which is 0.
__device__ __forceinline__ uint32_t sortable(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Largest over W = 1, 2, 4, 8 or 16 neighbouring lanes.
__device__ __forceinline__ uint32_t columns_max(uint32_t x, int w) {
  auto other = [](uint32_t v, auto ctrl) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xf, 0xf, true); };
  if (w > 1) x = max(x, other(x, std::integral_constant<int, 0xB1>()));
  if (w > 2) x = max(x, other(x, std::integral_constant<int, 0x4E>()));
  if (w > 4) x = max(x, other(x, std::integral_constant<int, 0x141>()));
  if (w > 8) x = max(x, other(x, std::integral_constant<int, 0x140>()));
  return x;
}

// A lane's 16 BF16 (two words of eight) to signed codes under the scale 1 / inv.
__device__ __forceinline__ v4u to_codes(v4u a, v4u b, float inv) {
  auto code = [&](unsigned bits) {
    const float x = __uint_as_float(bits);
    return (unsigned)(int)__builtin_rintf(__builtin_isfinite(x) ? x * inv : 0.f) & 0xFFu;
  };
  auto four = [&](unsigned x, unsigned y) {
    return code(x << 16) | code(x & 0xFFFF0000u) << 8 | code(y << 16) << 16 | code(y & 0xFFFF0000u) << 24;
  };
  return (v4u){four(a.x, a.y), four(a.z, a.w), four(b.x, b.y), four(b.z, b.w)};
}
// The largest finite magnitude of eight BF16, as bits of FP32.
__device__ __forceinline__ uint32_t largest(v4u a) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = a[i] << 16 & 0x7FFFFFFFu, hi = a[i] & 0x7FFF0000u;
    m = max(m, lo < 0x7F800000u ? lo : 0u);
    m = max(m, hi < 0x7F800000u ? hi : 0u);
  }
  return m;
}

// A tile's tokens.
struct Tokens {
  int seq, kv_head;
  int first_row, tokens;  // packed row of the first one, and how many there are
  int place0;             // place of the first one (negative where queries exceed the context)
  int64_t slot;           // number of the tile and key head
};
// Tile `id` of those of a launch; false if it has no tokens.
__device__ __forceinline__ bool get_tokens(const SelectParams& p, int id, Tokens& t) {
  // with the key head as the fastest index, and a multiple of eight heads, those of a head land on one XCD
  const int rank = id / p.num_heads;
  t.kv_head = id % p.num_heads;
  t.seq = rank % p.s.batch;
  const int tile = p.q_tiles.d - 1 - rank / p.s.batch;
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
  t.first_row += t0;
  const int ctx = min(max(uniform(p.s.seq_lens[t.seq]), 0), p.s.table_cols * p.page.d);
  t.place0 = ctx - n + t0;
  t.slot = id;
  return t.tokens > 0;
}
// Blocks up to and with a place's own.
__device__ __forceinline__ int blocks_to(const SelectParams& p, int place) { return place >= 0 ? div(place, p.page) + 1 : 0; }

// Scores of blocks [lo, hi) by the tile's tokens, of which this is the part `part` of `parts` (of 16 blocks at a time, in turn for the waves of all
// parts), to rows of p.row_words numbers from block `base` on.
template <int D, int TILES>
__device__ __forceinline__ void score(const SelectParams& p, const Tokens& t, int base, int lo, int hi, int part, int parts, uint32_t* scores,
                                      v4u (&codes)[TILES][D / 64][64], float (&query_scales)[TILES][16]) {
  // AHEAD groups of 16 blocks at a time: their pages' loads go out together, then their keys'
  constexpr int Y = D / 64, AHEAD = TILES > 1 || D == 256 ? 2 : 4;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), g = lane >> 4, col = lane & 15;
  const int width = p.group.d > 8 ? 16 : p.group.d > 4 ? 8 : p.group.d > 2 ? 4 : p.group.d;  // columns of a token
  const int per_tile = 16 / width, tiles = (t.tokens + per_tile - 1) / per_tile;
  const int32_t* table = p.s.table + t.seq * p.s.table_stride;
  const int first = lo + 16 * (part * SELECT_WAVES + wave), step = 16 * SELECT_WAVES * parts;
  int pages[AHEAD];
  auto load_pages = [&](int b0) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) pages[a] = table[min(b0 + step * a + col, hi - 1)];
  };
  for (int head0 = 0; head0 < p.group.d; head0 += 16) {
    if (head0) __syncthreads();
    load_pages(first);
    for (int c = wave; c < tiles; c += SELECT_WAVES) {
      const int token = c * per_tile + col / width, h = head0 + col % width;
      const uint16_t* src = p.s.q + (t.first_row + min(token, t.tokens - 1)) * p.s.q_token_stride +
                            (t.kv_head * p.group.d + min(h, p.group.d - 1)) * p.s.q_head_stride + 16 * g;
      v4u x[Y][2];
      uint32_t m = 0;
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        x[y][0] = *(const v4u*)(src + 64 * y);
        x[y][1] = *(const v4u*)(src + 64 * y + 8);
        m = max(m, max(largest(x[y][0]), largest(x[y][1])));
      }
      m = __float_as_uint(attn::groups_max(__uint_as_float(m)));
      const uint32_t e = m ? max((int)(m >> 23) - 6 + ((m & 0x7FFFFFu) > 0x7E0000u ? 1 : 0), 1) : 127u;
      const float inv = __uint_as_float((254u - e) << 23);
      if (g == 0) query_scales[c][col] = __uint_as_float(e << 23);
#pragma unroll
      for (int y = 0; y < Y; ++y) codes[c][y][lane] = to_codes(x[y][0], x[y][1], inv);
    }
    __syncthreads();
    v4u q[TILES][Y];
    float sq[TILES];
#pragma unroll
    for (int c = 0; c < TILES; ++c) {
      if (c >= tiles) continue;
      sq[c] = query_scales[c][col];
#pragma unroll
      for (int y = 0; y < Y; ++y) q[c][y] = codes[c][y][lane];
    }
    // (columns of a token without a head)
    const bool part_empty = head0 + width > p.group.d, dead = head0 + col % width >= p.group.d;
    for (int b0 = first; b0 < hi; b0 += step * AHEAD) {
      v4u k[AHEAD][Y];
      float scale[AHEAD];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int64_t at = (int64_t)((unsigned)pages[a] < (unsigned)p.num_pages ? pages[a] : 0) * p.num_heads + t.kv_head;
        const int8_t* key = p.b.codes + at * D + 16 * g;
        if (b0 + step * a >= hi) continue;
#pragma unroll
        for (int y = 0; y < Y; ++y) k[a][y] = *(const v4u*)(key + 64 * y);
        scale[a] = p.b.scales[at];
      }
      load_pages(b0 + step * AHEAD);
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int from = b0 + step * a;
        if (from >= hi) continue;
        float sk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sk[i] = __shfl(scale[a], 4 * g + i);
#pragma unroll
        for (int c = 0; c < TILES; ++c) {
          if (c >= tiles) continue;
          v4i s = {0, 0, 0, 0};
#pragma unroll
          for (int y = 0; y < Y; ++y)
            s = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, k[a][y]), __builtin_bit_cast(v4i, q[c][y]), s, 0, 0, 0);
          v4u w;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = sortable((float)s[i] * sk[i] * sq[c]);
            if (part_empty) w[i] = dead ? 0u : w[i];
            w[i] = columns_max(w[i], width);
          }
          const int token = c * per_tile + col / width;
          if (col % width == 0 && token < t.tokens) {
            v4u* dst = (v4u*)(scores + token * p.row_words + from - base + 4 * g);
            if (head0) {  // (the same lane's, of the heads before)
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = max(w[i], (*dst)[i]);
            }
            *dst = w;
          }
        }
      }
    }
  }
}

// Largest of the lanes' numbers.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  auto from = [&](auto ctrl, auto rows) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, decltype(rows)::value, 0xf, false); };
  using std::integral_constant;
  x = max(x, from(integral_constant<int, 0x111>(), integral_constant<int, 0xf>()));  // 1, 2, 4, 8 lanes before, in rows of 16
  x = max(x, from(integral_constant<int, 0x112>(), integral_constant<int, 0xf>()));
  x = max(x, from(integral_constant<int, 0x114>(), integral_constant<int, 0xf>()));
  x = max(x, from(integral_constant<int, 0x118>(), integral_constant<int, 0xf>()));
  x = max(x, from(integral_constant<int, 0x142>(), integral_constant<int, 0xa>()));  // the last lane of row 0 (2) into row 1 (3)
  x = max(x, from(integral_constant<int, 0x143>(), integral_constant<int, 0xc>()));  // lane 31 into rows 2 and 3
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// The largest number that at least `need` of what `count` counts reach, from `low`, which `reach` of them do, to `high`; or any smaller one that no
// more than `enough` reach.  Leaves in `reach` how many reach it, and in `high` a number that is no smaller than the largest.
template <class Count>
__device__ __forceinline__ uint32_t threshold(uint32_t low, uint32_t& high, int need, int enough, int& reach, Count count) {
  while (low < high && reach > enough) {
    const uint32_t mid = low + (high - low) / 2 + 1;
    const int n = count(mid);
    if (n >= need)
      low = mid, reach = n;
    else
      high = mid - 1;
  }
  return low;
}

constexpr int CANDIDATES = SELECT_CANDIDATES;

// The blocks of the token at `place`, by a wave, into `out`.  row: its scores, from block `first` on.
__device__ __forceinline__ void choose(const SelectParams& p, int place, const uint32_t* row, uint32_t* candidates, int32_t* out) {
  const int lane = threadIdx.x & 63, all = blocks_to(p, place);
  if (all <= p.top) {
    for (int i = lane; i < p.top; i += 64) out[i] = i < all ? i : -1;
    return;
  }
  // (first + last <= top < all, so they do not meet)
  const int need = p.top - p.first - p.last, count = all - p.last - p.first;
  for (int i = lane; i < p.first; i += 64) out[i] = i;
  for (int i = lane; i < p.last; i += 64) out[p.first + need + i] = all - p.last + i;
  if (need == 0) return;
  const uint64_t below = (1ull << lane) - 1;
  constexpr int HELD = CANDIDATES / 64;
  uint32_t x[HELD] = {};  // up to CANDIDATES scores that hold the chosen ones, number i in lane i % 64's register i / 64
  uint32_t low, high;
  int held = count;
  if (count > CANDIDATES) {
    // A lane's KEPT largest of every 64th score: `need` of all lanes' reach some number, so of all scores at least as many do, and
    // the threshold is no smaller.  Few others reach it, unless lanes have many more than they kept.
    constexpr int KEPT = 4;
    uint32_t kept[KEPT] = {};
#pragma unroll 8
    for (int i = lane; i < count; i += 64) {
      uint32_t y = row[i];
#pragma unroll
      for (int k = 0; k < KEPT; ++k) {
        const uint32_t larger = max(kept[k], y);
        y = min(kept[k], y);
        kept[k] = larger;
      }
    }
    auto keeping = [&](uint32_t t) {
      int n = 0;
#pragma unroll
      for (int k = 0; k < KEPT; ++k) n += (int)__popcll(__ballot(kept[k] >= t));
      return n;
    };
    high = wave_max(kept[0]);
    // (the smallest of the lanes' largest is reached by every lane; no score is 0)
    low = need <= 64 ? max(~wave_max(~kept[0]), 1u) : 1u;
    int reach = keeping(low);
    if (reach >= need) {
      uint32_t end = high;
      low = threshold(low, end, need, need, reach, keeping);
    }
    held = 0;
#pragma unroll 4
    for (int i0 = 0; i0 < count; i0 += 64) {
      const uint32_t y = row[min(i0 + lane, count - 1)];
      const bool may = i0 + lane < count && y >= low;
      const uint64_t some = __ballot(may);
      const int at = held + (int)__popcll(some & below);
      if (may && at < CANDIDATES) candidates[at] = y;
      held += (int)__popcll(some);
    }
    if (held <= CANDIDATES) {
      // (the wave reads what its other lanes wrote: its LDS operations complete in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int r = 0; r < HELD; ++r)
        if (64 * r + lane < held) x[r] = candidates[64 * r + lane];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    uint32_t most = 0;
#pragma unroll
    for (int r = 0; r < HELD; ++r)
      if (64 * r < count) {
        if (64 * r + lane < count) x[r] = row[64 * r + lane];
        most = max(most, x[r]);
      }
    high = wave_max(most);
    low = need <= 64 ? max(~wave_max(~most), 1u) : 1u;
  }
  auto search = [&](auto reaching, int reach) {
    const uint32_t t = threshold(low, high, need, need, reach, reaching);
    if (reach == need) {
      int at = p.first;
#pragma unroll 4
      for (int i0 = 0; i0 < count; i0 += 64) {
        const bool take = i0 + lane < count && row[min(i0 + lane, count - 1)] >= t;
        const uint64_t taken = __ballot(take);
        if (take) out[at + (int)__popcll(taken & below)] = p.first + i0 + lane;
        at += (int)__popcll(taken);
      }
      return;
    }
    // those above it, and of those equal to it the first ones
    int at = p.first, equals = need - (t == UINT32_MAX ? 0 : reaching(t + 1));
    for (int i0 = 0; i0 < count; i0 += 64) {
      const uint32_t y = i0 + lane < count ? row[i0 + lane] : 0u;
      const uint64_t same = __ballot(y == t);
      const bool take = y > t || (y == t && (int)__popcll(same & below) < equals);
      const uint64_t taken = __ballot(take);
      if (take) out[at + (int)__popcll(taken & below)] = p.first + i0 + lane;
      at += (int)__popcll(taken);
      equals -= min((int)__popcll(same), equals);
    }
  };
  auto search_held = [&](auto registers) {
    constexpr int R = decltype(registers)::value;
    auto reaching = [&](uint32_t t) {
      int n = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) n += (int)__popcll(__ballot(x[r] >= t));
      return n;
    };
    int reach = reaching(low);
    if (need <= 64) {
      // down to 64 of them, which then go to a lane each
      low = threshold(low, high, need, 64, reach, reaching);
      if (reach <= 64) {
        int n = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint64_t some = __ballot(x[r] >= low);
          if (x[r] >= low) candidates[n + (int)__popcll(some & below)] = x[r];
          n += (int)__popcll(some);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const uint32_t y = lane < reach ? candidates[lane] : 0u;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        return search([&](uint32_t t) { return (int)__popcll(__ballot(y >= t)); }, reach);
      }
    }
    search(reaching, reach);
  };
  if (held <= 128)
    search_held(std::integral_constant<int, 2>());
  else if (held <= CANDIDATES)
    search_held(std::integral_constant<int, HELD>());
  else {  // (more candidates than there is room for: more than 256 blocks to choose, or many equal scores)
    const auto reaching = [&](uint32_t t) {
      int n = 0;
#pragma unroll 8
      for (int i0 = 0; i0 < count; i0 += 64) n += (int)__popcll(__ballot(i0 + lane < count && row[min(i0 + lane, count - 1)] >= t));
      return n;
    };
    search(reaching, reaching(low));
  }
}

template <int D, int TILES>
__global__ void __launch_bounds__(SELECT_WAVES * 64, D == 256 ? 2 : 4) select_kernel(const SelectParams p) {
  extern __shared__ __attribute__((aligned(16))) uint32_t scores[];  // [tile_tokens][row_words], then [waves][CANDIDATES]
  __shared__ __attribute__((aligned(16))) v4u codes[TILES][D / 64][64];  // the queries as operands
  __shared__ float query_scales[TILES][16];
  Tokens t;
  if (!get_tokens(p, blockIdx.x, t)) return;
  const int wave = uniform((int)threadIdx.x >> 6), blocks = blocks_to(p, t.place0 + t.tokens - 1);
  if (blocks > p.top) {
    score<D, TILES>(p, t, p.first, p.first, blocks - p.last, 0, 1, scores, codes, query_scales);
    __syncthreads();
  }
  for (int token = wave; token < t.tokens; token += SELECT_WAVES)
    choose(p, t.place0 + token, scores + token * p.row_words, scores + p.tile_tokens * p.row_words + wave * CANDIDATES,
           p.out + ((int64_t)(t.first_row + token) * p.num_heads + t.kv_head) * p.top);
}

// The two steps as kernels of their own, with the scores in memory.
template <int D>
__global__ void __launch_bounds__(SELECT_WAVES * 64, D == 256 ? 2 : 4) score_kernel(const SelectParams p) {
  __shared__ __attribute__((aligned(16))) v4u codes[1][D / 64][64];
  __shared__ float query_scales[1][16];
  Tokens t;
  const int tiles = p.items * p.num_heads;
  if (!get_tokens(p, blockIdx.x % tiles, t)) return;
  const int blocks = blocks_to(p, t.place0 + t.tokens - 1);
  if (blocks > p.top)
    score<D, 1>(p, t, p.first, p.first, blocks - p.last, blockIdx.x / tiles, p.parts, p.scores + t.slot * p.tile_tokens * p.row_words, codes, query_scales);
}

// (a workgroup for a token and key head: all of it brings the scores to LDS, where one wave goes over them several times)
constexpr int CHOOSE_THREADS = 256;
__global__ void __launch_bounds__(CHOOSE_THREADS) choose_kernel(const SelectParams p) {
  extern __shared__ __attribute__((aligned(16))) uint32_t scores[];  // [row_words], then [CANDIDATES]
  Tokens t;
  const int tiles = p.items * p.num_heads, token = blockIdx.x / tiles;
  if (!get_tokens(p, blockIdx.x % tiles, t) || token >= t.tokens) return;
  const int count = blocks_to(p, t.place0 + token) - p.last - p.first;
  const uint32_t* row = p.scores + (t.slot * p.tile_tokens + token) * p.row_words;
  if (count + p.first + p.last > p.top) {
#pragma unroll 4
    for (int i = 4 * threadIdx.x; i < count; i += 4 * CHOOSE_THREADS) *(v4u*)(scores + i) = *(const v4u*)(row + i);  // (whole groups of 16 are written)
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  choose(p, t.place0 + token, scores, scores + p.row_words, p.out + ((int64_t)(t.first_row + token) * p.num_heads + t.kv_head) * p.top);
}

template <int D>
hipError_t select(const SelectParams& p, bool one_tile, hipStream_t stream) {
  const unsigned tiles = (unsigned)((int64_t)p.items * p.num_heads);
  const dim3 threads(SELECT_WAVES * 64);
  if (p.parts > 1) {
    hipLaunchKernelGGL((score_kernel<D>), dim3(tiles * p.parts), threads, 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((choose_kernel), dim3(tiles * p.tile_tokens), dim3(CHOOSE_THREADS), (size_t)(p.row_words + CANDIDATES) * 4, stream, p);
    return hipGetLastError();
  }
  const size_t lds = ((size_t)p.tile_tokens * p.row_words + (size_t)SELECT_WAVES * CANDIDATES) * 4;
  if (one_tile)
    hipLaunchKernelGGL((select_kernel<D, 1>), dim3(tiles), threads, lds, stream, p);
  else
    hipLaunchKernelGGL((select_kernel<D, select_tiles(D)>), dim3(tiles), threads, lds, stream, p);
  return hipGetLastError();
}

}  // namespace blocks

hipError_t launch_block_keys(const BlockKeysParams& p, int head_dim, hipStream_t stream) {
  const int64_t waves = (int64_t)p.num_pages * p.c.num_heads;
  const dim3 grid((unsigned)((waves + blocks::KEYS_WAVES - 1) / blocks::KEYS_WAVES)), threads(blocks::KEYS_WAVES * 64);
  if (head_dim == 64)
    hipLaunchKernelGGL((blocks::block_keys_kernel<64>), grid, threads, 0, stream, p);
  else if (head_dim == 128)
    hipLaunchKernelGGL((blocks::block_keys_kernel<128>), grid, threads, 0, stream, p);
  else if (head_dim == 256)
    hipLaunchKernelGGL((blocks::block_keys_kernel<256>), grid, threads, 0, stream, p);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_select_blocks(const SelectParams& p, int head_dim, bool one_tile, hipStream_t stream) {
  if (head_dim == 64) return blocks::select<64>(p, one_tile, stream);
  if (head_dim == 128) return blocks::select<128>(p, one_tile, stream);
  if (head_dim == 256) return blocks::select<256>(p, one_tile, stream);
  return hipErrorInvalidValue;
}

}  // namespace dg
