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
// the keys.
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
  for (int t = r; t < p.c.page.d; t += ROWS) {
    v4u x = *(const v4u*)(codes + t * p.c.token_stride);
    const uint32_t sf = sfs[t * p.c.sf_token_stride];
    const double scale = __hiloint2double((int)((sf + 1023 - 127) << 20), 0);
    if (__builtin_expect(__any(attn::may_be_odd(x, 0)), 0)) {  // a NaN counts as zero
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned nan = (((x[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;  // one for each NaN
        x[i] &= ~(nan * 0xFFu);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[i], true);
      s[4 * i] = __builtin_fma((double)lo.x, scale, s[4 * i]);
      s[4 * i + 1] = __builtin_fma((double)lo.y, scale, s[4 * i + 1]);
      s[4 * i + 2] = __builtin_fma((double)hi.x, scale, s[4 * i + 2]);
      s[4 * i + 3] = __builtin_fma((double)hi.y, scale, s[4 * i + 3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; i += 2) *(v2d*)&sums[wave][r][16 * l + i] = (v2d){s[i], s[i + 1]};
  // (the wave reads what its own lanes wrote: its LDS operations complete in order)
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  double mean[E];
  uint64_t top = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    mean[e] = 0.0;
#pragma unroll
    for (int x = 0; x < ROWS; ++x) mean[e] += sums[wave][x][E * lane + e];
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
// largest over a token's columns goes to LDS as a number that compares like the score.  Then a wave has a token:
// it finds the largest threshold that enough scores reach, bit by bit, and writes the chosen blocks in order.

// The order of floats as unsigned numbers, none of which is 0.
__device__ __forceinline__ uint32_t sortable(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Largest over W = 1, 2, 4, 8 or 16 neighbouring lanes.
__device__ __forceinline__ float columns_max(float x, int w) {
  auto other = [](float v, auto ctrl) { return __uint_as_float((unsigned)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, true)); };
  if (w > 1) x = fmaxf(x, other(x, std::integral_constant<int, 0xB1>()));
  if (w > 2) x = fmaxf(x, other(x, std::integral_constant<int, 0x4E>()));
  if (w > 4) x = fmaxf(x, other(x, std::integral_constant<int, 0x141>()));
  if (w > 8) x = fmaxf(x, other(x, std::integral_constant<int, 0x140>()));
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

template <int D>
__global__ void __launch_bounds__(512) select_kernel(const SelectParams p) {
  constexpr int Y = D / 64, TILES = select_tiles(D);
  extern __shared__ __attribute__((aligned(16))) uint32_t scores[];  // [tile_tokens][row_words]
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), g = lane >> 4, col = lane & 15;
  const int kv_head = blockIdx.x % p.num_heads, rank = blockIdx.x / p.num_heads;
  const int seq = rank % p.s.batch, tile = p.q_tiles.d - 1 - rank / p.s.batch;
  // the tile's tokens and their places
  int first_row, n;
  if (p.s.cu_q) {
    const int a = uniform(p.s.cu_q[seq]), b = uniform(p.s.cu_q[seq + 1]);
    first_row = min(max(a, 0), p.s.total_q);
    n = min(max(b, first_row), p.s.total_q) - first_row;
  } else {
    first_row = seq * p.s.q_per_seq;
    n = p.s.q_per_seq;
  }
  const int t0 = tile * p.tile_tokens, tokens = min(p.tile_tokens, n - t0);
  if (tokens <= 0) return;
  const int ctx = min(max(uniform(p.s.seq_lens[seq]), 0), p.s.table_cols * p.page.d);
  const int place0 = ctx - n + t0;  // of the tile's first token
  // blocks that are scored: of the tile's last token
  const int last_place = place0 + tokens - 1, own = last_place >= 0 ? div(last_place, p.page) : -1;
  const int lo = p.first, hi = own + 1 - p.last;
  const int32_t* table = p.s.table + seq * p.s.table_stride;
  if (own + 1 > p.top) {
    const int width = p.group.d > 8 ? 16 : p.group.d > 4 ? 8 : p.group.d > 2 ? 4 : p.group.d;  // columns of a token
    const int per_tile = 16 / width, tiles = (tokens + per_tile - 1) / per_tile;
    for (int head0 = 0; head0 < p.group.d; head0 += 16) {
      v4u q[TILES][Y];
      float sq[TILES];
#pragma unroll
      for (int c = 0; c < TILES; ++c) {
        const int token = c * per_tile + col / width, h = head0 + col % width;
        const bool live = token < tokens && h < p.group.d;
        const uint16_t* src = p.s.q + (first_row + t0 + min(token, tokens - 1)) * p.s.q_token_stride +
                              (kv_head * p.group.d + min(h, p.group.d - 1)) * p.s.q_head_stride + 16 * g;
        v4u x[Y][2];
        uint32_t m = 0;
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          x[y][0] = x[y][1] = (v4u){0, 0, 0, 0};
          if (c < tiles) {
            x[y][0] = *(const v4u*)(src + 64 * y);
            x[y][1] = *(const v4u*)(src + 64 * y + 8);
          }
          m = max(m, max(largest(x[y][0]), largest(x[y][1])));
        }
        m = __float_as_uint(attn::groups_max(__uint_as_float(m)));
        const uint32_t e = m ? max((int)(m >> 23) - 6 + ((m & 0x7FFFFFu) > 0x7E0000u ? 1 : 0), 1) : 127u;
        const float inv = __uint_as_float((254u - e) << 23);
        sq[c] = live ? __uint_as_float(e << 23) : attn::NEG_INF;
#pragma unroll
        for (int y = 0; y < Y; ++y) q[c][y] = to_codes(x[y][0], x[y][1], inv);
      }
      for (int b0 = lo + 16 * wave; b0 < hi; b0 += 16 * p.waves) {
        int page = table[min(b0 + col, hi - 1)];
        if ((unsigned)page >= (unsigned)p.num_pages) page = 0;
        const int64_t at = (int64_t)page * p.num_heads + kv_head;
        const int8_t* key = p.b.codes + at * D + 16 * g;
        v4u k[Y];
#pragma unroll
        for (int y = 0; y < Y; ++y) k[y] = *(const v4u*)(key + 64 * y);
        const float scale = p.b.scales[at];
        float sk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sk[i] = __shfl(scale, 4 * g + i);
#pragma unroll
        for (int c = 0; c < TILES; ++c) {
          if (c >= tiles) continue;
          v4i s = {0, 0, 0, 0};
#pragma unroll
          for (int y = 0; y < Y; ++y)
            s = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, k[y]), __builtin_bit_cast(v4i, q[c][y]), s, 0, 0, 0);
          v4u w;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = sq[c] == attn::NEG_INF ? sq[c] : (float)s[i] * sk[i] * sq[c];
            w[i] = sortable(columns_max(x, width));
          }
          const int token = c * per_tile + col / width;
          if (col % width == 0 && token < tokens) {
            v4u* dst = (v4u*)(scores + token * p.row_words + b0 - lo + 4 * g);
            if (head0) {  // (the same lane's, of the heads before)
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = max(w[i], (*dst)[i]);
            }
            *dst = w;
          }
        }
      }
    }
    __syncthreads();
  }
  for (int token = wave; token < tokens; token += p.waves) {
    const int place = place0 + token, mine = place >= 0 ? div(place, p.page) : -1;
    int32_t* out = p.out + ((int64_t)(first_row + t0 + token) * p.num_heads + kv_head) * p.top;
    const int all = mine + 1;
    if (all <= p.top) {
      for (int i = lane; i < p.top; i += 64) out[i] = i < all ? i : -1;
      continue;
    }
    // (first + last <= top < all, so they do not meet)
    const int need = p.top - p.first - p.last, count = all - p.last - p.first;
    for (int i = lane; i < p.first; i += 64) out[i] = i;
    for (int i = lane; i < p.last; i += 64) out[p.first + need + i] = all - p.last + i;
    if (need == 0) continue;
    const uint32_t* row = scores + token * p.row_words;
    // the largest threshold that at least `need` scores reach, and how many do
    uint32_t t = 0;
    int reach = count;
    for (uint32_t bit = 1u << 31; bit && reach > need; bit >>= 1) {
      int x = 0;
      for (int i = lane; i < count; i += 64) x += row[i] >= (t | bit) ? 1 : 0;
#pragma unroll
      for (int step = 1; step < 64; step *= 2) x += __shfl_xor(x, step);
      if (x >= need) t |= bit, reach = x;
    }
    // those above it, and of those equal to it the first ones
    int above = 0;
    if (reach > need) {
      for (int i = lane; i < count; i += 64) above += row[i] > t ? 1 : 0;
#pragma unroll
      for (int step = 1; step < 64; step *= 2) above += __shfl_xor(above, step);
    }
    int equals = reach > need ? need - above : INT32_MAX, at = p.first;
    for (int i0 = 0; i0 < count; i0 += 64) {
      const int i = i0 + lane;
      const uint32_t x = i < count ? row[i] : 0u;
      const uint64_t same = __ballot(i < count && x == t);
      const uint64_t below = (1ull << lane) - 1;
      const bool take = i < count && (x > t || (x == t && (int)__popcll(same & below) < equals));
      const uint64_t taken = __ballot(take);
      if (take) out[at + (int)__popcll(taken & below)] = p.first + i;
      at += (int)__popcll(taken);
      equals -= min((int)__popcll(same), equals);
    }
  }
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

hipError_t launch_select_blocks(const SelectParams& p, int head_dim, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.items * p.num_heads)), threads(p.waves * 64);
  const size_t lds = (size_t)p.tile_tokens * p.row_words * 4;
  if (head_dim == 64)
    hipLaunchKernelGGL((blocks::select_kernel<64>), grid, threads, lds, stream, p);
  else if (head_dim == 128)
    hipLaunchKernelGGL((blocks::select_kernel<128>), grid, threads, lds, stream, p);
  else if (head_dim == 256)
    hipLaunchKernelGGL((blocks::select_kernel<256>), grid, threads, lds, stream, p);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace dg
