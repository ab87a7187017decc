// FP8 key/value cache for gfx950 (MI355X): quantising tokens' keys and values into their slots,
// and reading them back.
//
// A row is one token and head: D values (64, 128 or 256), stored as E4M3 codes with one
// power-of-two scale, s = amax / 448 raised to the next power of two (1 for a row of zeros), kept
// as its exponent code sf (UE8M0): value = code * 2^(sf - 127).  A power of two costs E4M3 no
// relative precision (both the quotient and the product with it are exact) and lets a reader
// widen codes to BF16 exactly in one conversion.
//
// Both directions are bound by memory: D * (input size + 1) + 1 bytes a row.  A row is D / 8
// lanes of 8 values (16 bytes of BF16), a lane handles the key and the value row of its token
// and head, and a workgroup takes consecutive tokens of one head, whose cache rows and scale
// bytes are neighbours when their slots are.  Measured, BF16, 8 heads of 128: writing 8192 tokens
// 10.4 us (4.9 TB/s; 12.1 with a check of each value for infinities and NaN and the row's maximum through
// LDS: the vector unit was busy 92% of the time.  In that form, 11.9 with one token a lane, 14.4 with two,
// 15.7 with four, 12.8 with the rows loaded before the slot is known: more, smaller waves hide the latency
// better); reading 16384 tokens back 16.2 us (6.2 TB/s, part of it out of the last-level cache; 16.8 with
// one token a lane); 2.4 us for a decode step's 24 tokens.
#include "dg_kv.h"

namespace dg {
namespace {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int THREADS = 256;
constexpr int READ_ITEMS = 4;  // tokens of a lane of the read kernel

template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&x)[8]) {
  if constexpr (BF16) {
    const v4u r = *(const v4u*)((const uint16_t*)base + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  } else {
    const v4u r0 = *(const v4u*)((const float*)base + at), r1 = *(const v4u*)((const float*)base + at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __uint_as_float(r0[i]);
      x[4 + i] = __uint_as_float(r1[i]);
    }
  }
}

// The largest x of a row's lanes, L = 8, 16 or 32 consecutive ones: neighbours, pairs, quads (mirrored halves of
// eight), eights (mirrored rows), and the two rows of 16.
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, true));
  if constexpr (L >= 16) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xf, 0xf, true));
  if constexpr (L == 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max(r[0], r[1]);
  }
  return x;
}

// Codes of a lane's 8 values and the row's scale code.  The row's lanes are L consecutive ones.
// An infinite value does not count for the scale and saturates; a NaN becomes the NaN code.  Waves
// without either, whose values stay within 448 s by the choice of s, need no check for each value.
template <int L>
__device__ __forceinline__ v2u encode8(const float (&x)[8], uint32_t& sf) {
  constexpr uint32_t INF = 0x7F800000u;
  uint32_t b = 0;  // the largest magnitude, as bits
#pragma unroll
  for (int i = 0; i < 8; ++i) b = max(b, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  const bool special = __any(b >= INF);
  if (special) {
    b = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
      b = a < INF ? max(b, a) : b;
    }
  }
  b = row_max<L>(b);
  // 448 = 1.75 * 2^8: the smallest power of two >= amax / 448 has amax's exponent minus 8, plus
  // one when amax's mantissa is above 1.75
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  // (up to 224 of FP32's smallest steps, amax / 448 is zero in FP32, as for a row of zeros)
  sf = b <= 224u ? 127u : (uint32_t)max(e, 1);
  const float inv = __uint_as_float((254u - sf) << 23);  // 1 / s, exact (s <= 2^120)
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = x[i] * inv;
  if (special) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = x[i] == x[i] ? fminf(fmaxf(c[i], -448.f), 448.f) : x[i];
  }
  v2u r;
  r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
  r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], (int)r.x, true);
  r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
  r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], (int)r.y, true);
  return r;
}

struct Place {
  int64_t code, sf;  // byte offsets of the row
};
__device__ __forceinline__ bool place_of(const KvCache& c, int64_t slot, int head, Place& at) {
  const int64_t slots = (int64_t)c.num_pages * c.page.d;
  if (slot < 0 || slot >= slots) return false;
  // (the host keeps num_pages * page size below 2^31)
  const int32_t page = div((int32_t)slot, c.page), off = (int32_t)slot - page * c.page.d;
  at.code = page * c.page_stride + head * c.head_stride + off * c.token_stride;
  at.sf = page * c.sf_page_stride + head * c.sf_head_stride + off * c.sf_token_stride;
  return true;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS) kv_write_kernel(const KvMoveParams p) {
  constexpr int L = D / 8;
  const int token = blockIdx.x * (THREADS / L) + threadIdx.x / L, head = blockIdx.y, l = threadIdx.x % L;
  // (a whole row's lanes leave together, so the shuffles below stay within live lanes)
  if (token >= p.num_tokens) return;
  Place at;
  if (!place_of(p.c, p.slots[token], head, at)) return;
  float k[8], v[8];
  load8<BF16>(p.k, token * p.k_token_stride + head * p.k_head_stride + 8 * l, k);
  load8<BF16>(p.v, token * p.v_token_stride + head * p.v_head_stride + 8 * l, v);
  uint32_t ksf, vsf;
  const v2u kc = encode8<L>(k, ksf), vc = encode8<L>(v, vsf);
  *(v2u*)(p.c.k + at.code + 8 * l) = kc;
  *(v2u*)(p.c.v + at.code + 8 * l) = vc;
  if (l == 0) {
    p.c.k_sf[at.sf] = (uint8_t)ksf;
    p.c.v_sf[at.sf] = (uint8_t)vsf;
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t at, v2u codes, uint32_t sf) {
  const float s = __uint_as_float(sf << 23);
  if constexpr (BF16) {
    v4u r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[2 * i] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], s, false));
      r[2 * i + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], s, true));
    }
    *(v4u*)((uint16_t*)base + at) = r;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[i], s, false);
      const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[i], s, true);
      *(v4u*)((float*)base + at + 4 * i) =
          (v4u){__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)};
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS) kv_read_kernel(const KvMoveParams p) {
  constexpr int L = D / 8, PASS = THREADS / L, ITEMS = READ_ITEMS;
  const int token0 = blockIdx.x * (PASS * ITEMS) + threadIdx.x / L, head = blockIdx.y, l = threadIdx.x % L;
  v2u kc[ITEMS], vc[ITEMS];
  uint32_t ksf[ITEMS], vsf[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int token = token0 + i * PASS;
    kc[i] = vc[i] = (v2u){0, 0};
    ksf[i] = vsf[i] = 127;  // a skipped slot reads as zeros
    Place at;
    if (token < p.num_tokens && place_of(p.c, p.slots[token], head, at)) {
      kc[i] = *(const v2u*)(p.c.k + at.code + 8 * l);
      vc[i] = *(const v2u*)(p.c.v + at.code + 8 * l);
      ksf[i] = p.c.k_sf[at.sf];
      vsf[i] = p.c.v_sf[at.sf];
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int token = token0 + i * PASS;
    if (token >= p.num_tokens) continue;
    store8<BF16>(p.k, token * p.k_token_stride + head * p.k_head_stride + 8 * l, kc[i], ksf[i]);
    store8<BF16>(p.v, token * p.v_token_stride + head * p.v_head_stride + 8 * l, vc[i], vsf[i]);
  }
}

}  // namespace

#define DG_KV_CASE(K, D, B, ITEMS)                                                                                     \
  if (head_dim == D && bf16 == B) {                                                                                    \
    const int per = THREADS / (D / 8) * ITEMS;                                                                         \
    hipLaunchKernelGGL((K<D, B>), dim3((p.num_tokens + per - 1) / per, p.c.num_heads), dim3(THREADS), 0, stream, p);   \
    return hipGetLastError();                                                                                          \
  }
#define DG_KV_CASES(K, ITEMS)                                                                    \
  DG_KV_CASE(K, 64, true, ITEMS) DG_KV_CASE(K, 64, false, ITEMS) DG_KV_CASE(K, 128, true, ITEMS) \
  DG_KV_CASE(K, 128, false, ITEMS) DG_KV_CASE(K, 256, true, ITEMS) DG_KV_CASE(K, 256, false, ITEMS)

hipError_t launch_kv_write(const KvMoveParams& p, int head_dim, bool bf16, hipStream_t stream) {
  DG_KV_CASES(kv_write_kernel, 1)
  return hipErrorInvalidValue;
}

hipError_t launch_kv_read(const KvMoveParams& p, int head_dim, bool bf16, hipStream_t stream) {
  DG_KV_CASES(kv_read_kernel, READ_ITEMS)
  return hipErrorInvalidValue;
}
#undef DG_KV_CASES
#undef DG_KV_CASE

}  // namespace dg
