// What the kernels that fill the FP8 key/value cache share: reading rows, quantising them, finding their place.
#pragma once

#include "dg_kv.h"

namespace dg {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

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

// The largest x of a row's lanes, L = 4, 8, 16 or 32 consecutive ones: neighbours, pairs, quads (mirrored halves of
// eight), eights (mirrored rows), and the two rows of 16.
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xf, 0xf, true));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xf, 0xf, true));
  if constexpr (L >= 8) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, true));
  if constexpr (L >= 16) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xf, 0xf, true));
  if constexpr (L == 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max(r[0], r[1]);
  }
  return x;
}

// Codes of a lane's N values (8 to a pair of words) and the row's scale code.  The row's lanes are L consecutive ones.
// An infinite value does not count for the scale and saturates; a NaN becomes the NaN code.  Waves
// without either, whose values stay within 448 s by the choice of s, need no check for each value.
template <int L, int N>
__device__ __forceinline__ void encode(const float (&x)[N], v2u (&codes)[N / 8], uint32_t& sf) {
  constexpr uint32_t INF = 0x7F800000u;
  uint32_t b = 0;  // the largest magnitude, as bits
#pragma unroll
  for (int i = 0; i < N; ++i) b = max(b, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  const bool special = __any(b >= INF);
  if (special) {
    b = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
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
  float c[N];
#pragma unroll
  for (int i = 0; i < N; ++i) c[i] = x[i] * inv;
  if (special) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = x[i] == x[i] ? fminf(fmaxf(c[i], -448.f), 448.f) : x[i];
  }
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    v2u r;
    r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[8 * i], c[8 * i + 1], 0, false);
    r.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[8 * i + 2], c[8 * i + 3], (int)r.x, true);
    r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[8 * i + 4], c[8 * i + 5], 0, false);
    r.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[8 * i + 6], c[8 * i + 7], (int)r.y, true);
    codes[i] = r;
  }
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

}  // namespace dg
