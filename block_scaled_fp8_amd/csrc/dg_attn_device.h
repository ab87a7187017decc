// What the attention kernels over the FP8 cache share.
#pragma once

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

constexpr float NEG_INF = -__builtin_inff();
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

// A value that is the same for all lanes, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32 | (uint32_t)uniform((int)x));
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
// What clear_odd has taken out of four places of a row: NaN, infinities, or nothing.
__device__ __forceinline__ v4f odd_values(unsigned codes, uint32_t sf) {
  const float s = __uint_as_float(sf << 23);
  const unsigned lo = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, false));
  const unsigned hi = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, true));
  auto odd = [](unsigned bits) { return (bits & 0x7F800000u) == 0x7F800000u ? __uint_as_float(bits) : 0.f; };
  return (v4f){odd(lo << 16), odd(lo & 0xFFFF0000u), odd(hi << 16), odd(hi & 0xFFFF0000u)};
}
__device__ __forceinline__ float inverse(float z) { return z > 0.f ? 1.f / z : (z == z ? 0.f : z); }
__device__ __forceinline__ float log_sum(float m, float z) {
  return z > 0.f ? (m + __log2f(z)) * 0.6931471805599453f : (z == z ? NEG_INF : z);
}

// Few rows' V tiles in LDS: BF16 rows of D values in 16-byte chunks.
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

// Buffer descriptor from a scalar address on, 2^31 - 1 bytes long (the host keeps a head's page below that).  With 0 bytes, loads
// give zeros and read nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* base, int bytes = 0x7FFFFFFF) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)uniform((int64_t)base), (short)0, bytes, 0x00020000);
}

}  // namespace attn
}  // namespace dg
