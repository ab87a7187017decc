// Norm and rotation of queries and keys for each head, for gfx950 (MI355X): forward, forward into the FP8
// key/value cache, and backward.
//
// For a row x (one token and head, D values), weights w and the token's angles a_i, i < R / 2:
//   y = w x r,  r = 1 / sqrt(mean(x^2) + eps),  and each pair (y_i, y_j) of the first R values turns:
//   (y_i cos a_i - y_j sin a_i, y_i sin a_i + y_j cos a_i),  j = i + R / 2, or (2 i, 2 i + 1) interleaved.
// Backward, with t the gradient of the result turned back, u = x r and g = w t:
//   dx = r (g - u mean(g u)),  dw = sum of t u over tokens and heads.
// All of it in FP32, rounded once at the end.
//
// Bound by memory.  A row is D / 16 lanes of 16 values, two chunks of eight that hold whole pairs: lane l < R / 16
// has chunks l and l + R / 16 (interleaved: 2 l and 2 l + 1), so a pair never leaves its lane, and both
// forms take the same cosines and sines, 8 l to 8 l + 7.  The rest of the row goes in pairs of chunks to the
// lanes after those.  A wave takes 1024 / D heads of one token, all of them queries, keys or values, and its loads go out together, before anything
// waits.  8192 tokens of 32 + 8 heads of 128, BF16: forward 26 us (168 MB: 6.5 TB/s with what the caches hold), backward 44 (252 MB, 5.7 TB/s)
// and 4 for the weights, forward into the cache 30 (189 MB, 6.3 TB/s).  FP32: 4096 tokens forward 29 us (168 MB, 5.8 TB/s), backward with the weights
// 48 (252 MB, 5.2 TB/s); 8192 tokens 67 and 103 (5.0 and 4.9 TB/s).
#include <type_traits>

#include "dg_kv_device.h"

namespace dg {
namespace rope {

constexpr int THREADS = 256, WAVES = THREADS / 64;

// A lane's place in its row.
struct Lane {
  int c0, c1;  // its chunks, as offsets of values
  bool turns;
};
template <int D, bool INTER>
__device__ __forceinline__ Lane lane_of(int l, int rot) {
  const int r = rot / 16;
  const bool turns = l < r;
  if (INTER) return {16 * l, 16 * l + 8, turns};
  // (past the turning lanes, 2 r + 2 (l - r) = 2 l)
  return turns ? Lane{8 * l, 8 * l + 8 * r, true} : Lane{16 * l, 16 * l + 8, false};
}

template <bool BF16>
__device__ __forceinline__ void load16(const void* base, int64_t at, const Lane& l, float (&x)[16]) {
  load8<BF16>(base, at + l.c0, *(float(*)[8])x);
  load8<BF16>(base, at + l.c1, *(float(*)[8])(x + 8));
}

__device__ __forceinline__ unsigned pack2(float x, float y) {
  return __builtin_bit_cast(unsigned, (v2bf){(__bf16)x, (__bf16)y});
}
// The second-level cache writes results through as they come instead of all at once when the kernel ends, where a store of a wave covers whole
// lines' halves: BF16 rows of which all values turn, in halves, on such addresses (8192 tokens of 32 + 8 heads of 128, forward and backward 78.0 us, by ordinary stores 79.6; into
// the FP8 cache 36.0 and 37.2).  Elsewhere a lane's 16 bytes have others' behind them, which that cache has to gather (FP32, 3307 tokens of 48 + 3 heads of
// 256, interleaved: forward 80 us, written through 159; BF16 heads of 128 interleaved 29 and 49).  (Stores past all caches are faster alone, but
// whoever reads the results has to fetch them from HBM: forward and its reader with cold caches 64.9 us, else 55.)
template <int D, bool BF16, bool INTER>
__device__ __forceinline__ bool whole_lines(int rot, const Rows& to) {
  return BF16 && !INTER && rot == D && (((uintptr_t)to.p | (uintptr_t)(2 * to.token_stride) | (uintptr_t)(2 * to.head_stride)) & 63) == 0;
}
__device__ __forceinline__ void store_through(v4u* to, v4u x) {
  // (a wave may not write the registers of such a store in the next cycle)
  asm volatile("global_store_dwordx4 %0, %1, off sc1\n\ts_nop 1" ::"v"(to), "v"(x) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void store16(void* base, int64_t at, const Lane& l, bool through, const float (&x)[16]) {
  constexpr int N = BF16 ? 1 : 2;  // 16-byte pieces of a chunk
  v4u out[2][N];
  v4u* dst[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int64_t to = at + (c ? l.c1 : l.c0);
    dst[c] = BF16 ? (v4u*)((uint16_t*)base + to) : (v4u*)((float*)base + to);
    const float* y = x + 8 * c;
    if constexpr (BF16) {
      out[c][0] = (v4u){pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7])};
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        out[c][i] = (v4u){__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), __float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3])};
    }
  }
  if (through) {
    store_through(dst[0], out[0][0]);
    store_through(dst[1], out[1][0]);
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < N; ++i) dst[c][i] = out[c][i];
  }
}

// Sum over the L lanes of a row, 4, 8 or 16 consecutive ones, in all of them.
template <int L>
__device__ __forceinline__ float row_sum(float x) {
  auto from = [](float v, auto ctrl) { return __uint_as_float((unsigned)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, true)); };
  x += from(x, std::integral_constant<int, 0xB1>());
  x += from(x, std::integral_constant<int, 0x4E>());
  if constexpr (L >= 8) x += from(x, std::integral_constant<int, 0x141>());
  if constexpr (L >= 16) x += from(x, std::integral_constant<int, 0x140>());
  return x;
}

template <int D>
__device__ __forceinline__ float inverse_rms(const float (&x)[16], float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s = __builtin_fmaf(x[i], x[i], s);
  return 1.f / __builtin_sqrtf(__builtin_fmaf(row_sum<D / 16>(s), 1.f / D, eps));
}

struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const RopeParams& p, int64_t position, int l, Angles& a) {
  const float* row = p.cos_sin + position * p.cos_sin_stride + 8 * l;
  load8<false>(row, 0, a.c);
  load8<false>(row, p.rot / 2, a.s);
}
// The pairs turned by the angles (SIGN 1) or back (-1).
template <bool INTER, int SIGN>
__device__ __forceinline__ void turn(float (&y)[16], const Angles& a) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float &u = y[INTER ? 2 * i : i], &v = y[INTER ? 2 * i + 1 : 8 + i];
    const float s = SIGN * a.s[i], x = __builtin_fmaf(u, a.c[i], -(v * s));
    v = __builtin_fmaf(u, s, v * a.c[i]);
    u = x;
  }
}

__device__ __forceinline__ void load_weights(const void* w, bool bf16, const Lane& l, float (&x)[16]) {
  if (bf16)
    load16<true>(w, 0, l, x);
  else
    load16<false>(w, 0, l, x);
}

// ---------------------------------------------------------------- forward
template <int D, bool BF16, bool INTER, bool WRITE>
__global__ void __launch_bounds__(THREADS) forward_kernel(const RopeParams p) {
  constexpr int L = D / 16, HEADS = 64 / L;
  const int lane = threadIdx.x & 63, l = lane % L;
  const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * WAVES + (threadIdx.x >> 6));
  const int token = div(wave, p.pieces);
  if (token >= p.num_tokens) return;
  // a wave's rows are all queries, all keys or all values (where these are written), so what depends on that is scalar
  const int piece = wave - token * p.pieces.d, after_q = piece - p.q_pieces, after_k = after_q - p.kv_pieces;
  const bool is_q = after_q < 0, is_v = WRITE && after_k >= 0;
  const int head = (is_q ? piece : is_v ? after_k : after_q) * HEADS + lane / L;
  if (head >= (is_q ? p.q_heads : p.kv_heads)) return;
  const int64_t position = p.positions[token];
  const bool live = (uint64_t)position < (uint64_t)p.num_positions;
  int64_t slot = 0;
  if (WRITE) slot = p.slots[token];
  const Lane my = is_v ? Lane{16 * l, 16 * l + 8, false} : lane_of<D, INTER>(l, p.rot);
  const Rows from = is_q ? p.q : is_v ? p.v : p.k, to = is_q ? p.q_out : p.k_out;
  const int64_t to_row = token * to.token_stride + head * to.head_stride;
  const bool through = whole_lines<D, BF16, INTER>(p.rot, to);
  float x[16];  // (on its way before its position is known)
  load16<BF16>(from.p, token * from.token_stride + head * from.head_stride, my, x);
  if (!live) {
    const float zeros[16] = {};
    if (!WRITE || is_q) store16<BF16>(to.p, to_row, my, through, zeros);
    return;
  }
  if (!is_v) {
    float w[16];
    Angles a;
    load_angles(p, position, my.turns ? l : 0, a);
    // (last: what has come by the branch on their type is waited for in it)
    load_weights(is_q ? p.q_weight : p.k_weight, p.weights_bf16, my, w);
    const float r = inverse_rms<D>(x, p.eps);
    // Squares past FP32's range: finite values become zeros before their products pass it too, whose infinities times r would be NaN.
    if (__builtin_expect(r == 0.f, 0)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= 0.f;
    }
    // (the weight first: two BF16's product is exact; r last: it rounds once what the turn has rounded)
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= w[i];
    if (my.turns) turn<INTER, 1>(x, a);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= r;
  }
  if (WRITE && !is_q) {
    Place at;
    if (!place_of(p.c, slot, head, at)) return;
    uint32_t sf;
    v2u codes[2];
    encode<L>(x, codes, sf);
    uint8_t* dst = (is_v ? p.c.v : p.c.k) + at.code;
    *(v2u*)(dst + my.c0) = codes[0];
    *(v2u*)(dst + my.c1) = codes[1];
    if (l == 0) (is_v ? p.c.v_sf : p.c.k_sf)[at.sf] = (uint8_t)sf;
    return;
  }
  store16<BF16>(to.p, to_row, my, through, x);
}

// ---------------------------------------------------------------- backward
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(THREADS) backward_kernel(const RopeParams p) {
  constexpr int L = D / 16, HEADS = 64 / L;
  __shared__ float sums[2][WAVES][D];
  const int lane = threadIdx.x & 63, l = lane % L, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Lane my = lane_of<D, INTER>(l, p.rot);
#pragma unroll 1
  for (int section = 0; section < 2; ++section) {
    const Rows from = section ? p.k : p.q, grad = section ? p.dk : p.dq, to = section ? p.k_out : p.q_out;
    const int heads = section ? p.kv_heads : p.q_heads, pieces = section ? p.kv_pieces : p.q_pieces;
    const bool through = whole_lines<D, BF16, INTER>(p.rot, to);
    float w[16], dw[16] = {};
    load_weights(section ? p.k_weight : p.q_weight, p.weights_bf16, my, w);
    // every (workgroups * WAVES)th piece
    const int step = p.workgroups * WAVES, step_token = step / pieces, step_piece = step - step_token * pieces;
    const int id = blockIdx.x * WAVES + wave;
    int token = id / pieces, piece = id - token * pieces;
    for (; token < p.num_tokens; token += step_token) {
      const int head = piece * HEADS + lane / L, at = token;
      piece += step_piece;
      if (piece >= pieces) piece -= pieces, ++token;
      if (head >= heads) continue;
      // (no result overlaps the positions, so the load may be scalar)
      const int64_t position = ((const __attribute__((address_space(4))) int64_t*)p.positions)[at];
      const int64_t to_row = at * to.token_stride + head * to.head_stride;
      float x[16], t[16];  // (on their way before the position is known)
      load16<BF16>(from.p, at * from.token_stride + head * from.head_stride, my, x);
      load16<BF16>(grad.p, at * grad.token_stride + head * grad.head_stride, my, t);
      if ((uint64_t)position >= (uint64_t)p.num_positions) {
        const float zeros[16] = {};
        store16<BF16>(to.p, to_row, my, through, zeros);
        continue;
      }
      Angles a;
      load_angles(p, position, my.turns ? l : 0, a);
      const float r = inverse_rms<D>(x, p.eps);
      // (loaded with the rows, not where only the turning lanes are)
#pragma unroll
      for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(a.c[i]), "+v"(a.s[i]));
      if (my.turns) turn<INTER, -1>(t, a);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[i] *= r;
        dw[i] = __builtin_fmaf(t[i], x[i], dw[i]);
        t[i] *= w[i];
        s = __builtin_fmaf(t[i], x[i], s);
      }
      const float mean = row_sum<L>(s) * (1.f / D);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = r * (t[i] - x[i] * mean);
      store16<BF16>(to.p, to_row, my, through, x);
    }
    // over the wave's rows: lanes l, l + L, ...
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
      for (int step = L; step < 64; step *= 2) dw[i] += __shfl_xor(dw[i], step);
    }
    if (lane < L) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sums[section][wave][(i < 8 ? my.c0 + i : my.c1 + i - 8)] = dw[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
    const int section = i / D, d = i % D;
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < WAVES; ++x) s += sums[section][x][d];
    if (p.workgroups == 1)
      (section ? p.dk_weight : p.dq_weight)[d] = s;
    else
      p.parts[(int64_t)blockIdx.x * 2 * D + i] = s;
  }
}

// The workgroups' sums of the weights' gradients, added up: a workgroup for 32 values.
template <int D>
__global__ void __launch_bounds__(1024) weights_kernel(const RopeParams p) {
  __shared__ float sums[32][33];
  const int i = blockIdx.x * 32 + (threadIdx.x & 31), group = threadIdx.x >> 5;
  float s = 0.f;
#pragma unroll 8
  for (int b = group; b < p.workgroups; b += 32) s += p.parts[(int64_t)b * 2 * D + i];
  sums[group][threadIdx.x & 31] = s;
  __syncthreads();
  if (group) return;
  s = 0.f;
#pragma unroll
  for (int x = 0; x < 32; ++x) s += sums[x][threadIdx.x];
  (i < D ? p.dq_weight : p.dk_weight)[i % D] = s;
}

template <int D, bool BF16, bool INTER>
hipError_t forward(const RopeParams& p, bool write, hipStream_t stream) {
  const unsigned grid = (unsigned)(((int64_t)p.num_tokens * p.pieces.d + WAVES - 1) / WAVES);
  if (write)
    hipLaunchKernelGGL((forward_kernel<D, BF16, INTER, true>), dim3(grid), dim3(THREADS), 0, stream, p);
  else
    hipLaunchKernelGGL((forward_kernel<D, BF16, INTER, false>), dim3(grid), dim3(THREADS), 0, stream, p);
  return hipGetLastError();
}

template <int D, bool BF16, bool INTER>
hipError_t backward(const RopeParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((backward_kernel<D, BF16, INTER>), dim3(p.workgroups), dim3(THREADS), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.workgroups == 1) return e;
  hipLaunchKernelGGL((weights_kernel<D>), dim3(2 * D / 32), dim3(1024), 0, stream, p);
  return hipGetLastError();
}

}  // namespace rope

#define DG_ROPE_CASES(CALL, ...)                                                                       \
  switch (head_dim) {                                                                                  \
    case 64: return bf16 ? (interleaved ? rope::CALL<64, true, true>(__VA_ARGS__) : rope::CALL<64, true, false>(__VA_ARGS__))    \
                         : (interleaved ? rope::CALL<64, false, true>(__VA_ARGS__) : rope::CALL<64, false, false>(__VA_ARGS__)); \
    case 128: return bf16 ? (interleaved ? rope::CALL<128, true, true>(__VA_ARGS__) : rope::CALL<128, true, false>(__VA_ARGS__))    \
                          : (interleaved ? rope::CALL<128, false, true>(__VA_ARGS__) : rope::CALL<128, false, false>(__VA_ARGS__)); \
    case 256: return bf16 ? (interleaved ? rope::CALL<256, true, true>(__VA_ARGS__) : rope::CALL<256, true, false>(__VA_ARGS__))    \
                          : (interleaved ? rope::CALL<256, false, true>(__VA_ARGS__) : rope::CALL<256, false, false>(__VA_ARGS__)); \
  }                                                                                                    \
  return hipErrorInvalidValue

hipError_t launch_norm_rope(const RopeParams& p, int head_dim, bool bf16, bool interleaved, bool write, hipStream_t stream) {
  DG_ROPE_CASES(forward, p, write, stream);
}
hipError_t launch_norm_rope_backward(const RopeParams& p, int head_dim, bool bf16, bool interleaved, hipStream_t stream) {
  DG_ROPE_CASES(backward, p, stream);
}
#undef DG_ROPE_CASES

}  // namespace dg
