// layer_device.h -- device helpers of the layer operators' kernels.
//
// Rows are [count, hidden] with no padding, so a row of an odd `hidden`
// starts at any element.  Vectors of eight elements are therefore loaded and
// stored through types that promise only the element's own alignment: gfx950
// takes 16- and 8-byte global accesses at any byte address in one
// instruction, and where the address is aligned they cost what the aligned
// ones do.  Only a row's last vector, where hidden % 8 != 0, goes element by
// element.
#pragma once

#include "fp8q_device.h"

namespace fp8q {

typedef u32x4 u32x4_el2 __attribute__((aligned(2)));   // eight bf16
typedef u32x2 u32x2_el1 __attribute__((aligned(1)));   // eight codes
typedef f32x4 f32x4_el4 __attribute__((aligned(4)));   // four fp32

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Sum over the wave, the same bits on every lane (each step adds the same two
// numbers on both sides of an exchange).
__device__ __forceinline__ float sum_wave(float v) {
  v = dpp_add<kDppQuadXor1>(v);
  v = dpp_add<kDppQuadXor2>(v);
  v = dpp_add<kDppRowHalfMirror>(v);
  v = dpp_add<kDppRowMirror>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Eight bf16 from p, of which the first n exist (n >= 8: all); the rest read
// as zero.  NT: a non-temporal load, for data that is read once.
template <bool NT>
__device__ __forceinline__ u32x4 load8_bf16(const uint16_t *p, int n) {
  if (n >= 8) {
    if constexpr (NT)
      return __builtin_nontemporal_load(reinterpret_cast<const u32x4_el2 *>(p));
    else
      return *reinterpret_cast<const u32x4_el2 *>(p);
  }
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
  return u32x4{w[0], w[1], w[2], w[3]};
}

template <bool NT>
__device__ __forceinline__ void store8_bf16(uint16_t *p, u32x4 v, int n) {
  if (n >= 8) {
    if constexpr (NT)
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_el2 *>(p));
    else
      *reinterpret_cast<u32x4_el2 *>(p) = v;
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) p[j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
}

template <bool NT>
__device__ __forceinline__ u32x2 load8_codes(const uint8_t *p, int n) {
  if (n >= 8) {
    if constexpr (NT)
      return __builtin_nontemporal_load(reinterpret_cast<const u32x2_el1 *>(p));
    else
      return *reinterpret_cast<const u32x2_el1 *>(p);
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return u32x2{w[0], w[1]};
}

template <bool NT>
__device__ __forceinline__ void store8_codes(uint8_t *p, u32x2 v, int n) {
  if (n >= 8) {
    if constexpr (NT)
      __builtin_nontemporal_store(v, reinterpret_cast<u32x2_el1 *>(p));
    else
      *reinterpret_cast<u32x2_el1 *>(p) = v;
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) p[j] = (uint8_t)(v[j >> 2] >> (8 * (j & 3)));
}

__device__ __forceinline__ void widen8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(v[j]);
    f[2 * j + 1] = bf16_hi(v[j]);
  }
}

__device__ __forceinline__ u32x4 round8_bf16(const float (&f)[8]) {
  return u32x4{bf16_pack2(f[0], f[1]), bf16_pack2(f[2], f[3]), bf16_pack2(f[4], f[5]),
               bf16_pack2(f[6], f[7])};
}

// Eight weights of a norm, fp32 or bf16 in memory (the same for every row, so
// the load may stay in the caches).  Elements at and past n read as zero.
__device__ __forceinline__ void load8_weight(const void *w, bool is_bf16, uint32_t e, int n,
                                             float (&f)[8]) {
  if (is_bf16) {
    widen8(load8_bf16<false>(static_cast<const uint16_t *>(w) + e, n), f);
    return;
  }
  const float *p = static_cast<const float *>(w) + e;
  if (n >= 8) {
    const f32x4 a = *reinterpret_cast<const f32x4_el4 *>(p);
    const f32x4 b = *reinterpret_cast<const f32x4_el4 *>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = a[j];
      f[4 + j] = b[j];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = j < n ? p[j] : 0.0f;
}

}  // namespace fp8q
