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
#include "dg_kv_device.h"

namespace dg {
namespace {

constexpr int THREADS = 256;
constexpr int READ_ITEMS = 4;  // tokens of a lane of the read kernel

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
  v2u kc[1], vc[1];
  encode<L>(k, kc, ksf);
  encode<L>(v, vc, vsf);
  *(v2u*)(p.c.k + at.code + 8 * l) = kc[0];
  *(v2u*)(p.c.v + at.code + 8 * l) = vc[0];
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
