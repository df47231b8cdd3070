// layer_device.h -- device helpers of the layer operators' kernels.
//
// Rows are [count, hidden] with no padding, so a row of an odd `hidden`
// starts at any element.  Vectors of eight elements are therefore loaded and
// stored through types that promise no alignment: gfx950 takes 16- and 8-byte
// global accesses at any byte address in one instruction, and where the
// address is aligned they cost what the aligned ones do.
//
// Column e of a vector may lie at or past the row's end: the loads below then
// read inside the row all the same, and zeros are selected afterwards, so that
// they need no branch.
// EDGE says how a row ends:
//   kEven  hidden % 8 == 0: a vector is inside the row or outside;
//   kOdd   any hidden from 8 on: the row's last vector is loaded eight
//          elements before its end and shifted into place;
//   kTiny  hidden < 8: element by element.
#pragma once

#include "fp8q_device.h"

namespace fp8q {

typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// 16 and 8 bytes at any address; NT: non-temporal, for data touched once.
template <bool NT>
__device__ __forceinline__ u32x4 load16(const void *p) {
  const u32x4_any *q = static_cast<const u32x4_any *>(p);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  return *q;
}

template <bool NT>
__device__ __forceinline__ u32x2 load8(const void *p) {
  const u32x2_any *q = static_cast<const u32x2_any *>(p);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  return *q;
}

template <bool NT>
__device__ __forceinline__ void store16(void *p, u32x4 v) {
  u32x4_any *q = static_cast<u32x4_any *>(p);
  if constexpr (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

template <bool NT>
__device__ __forceinline__ void store8(void *p, u32x2 v) {
  u32x2_any *q = static_cast<u32x2_any *>(p);
  if constexpr (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

enum Edge : int { kEven = 0, kOdd = 1, kTiny = 2 };

constexpr Edge edge_of(uint64_t hidden) { return hidden % 8 == 0 ? kEven : hidden >= 8 ? kOdd : kTiny; }

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Sum over the wave, the same bits on every lane: DPP steps inside the rows of
// 16 (each adds the same two numbers on both sides of an exchange), then the
// four rows' sums through scalar registers, with no LDS access to wait for.
__device__ __forceinline__ float sum_wave(float v) {
  v = dpp_add<kDppQuadXor1>(v);
  v = dpp_add<kDppQuadXor2>(v);
  v = dpp_add<kDppRowHalfMirror>(v);
  v = dpp_add<kDppRowMirror>(v);
  const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
  const float b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
  const float c = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
  const float d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
  return (a + b) + (c + d);
}

// v's elements moved down by n of `bits` bits each, zeros behind them.
__device__ __forceinline__ u32x4 shift_down(u32x4 v, uint32_t n, uint32_t bits) {
  const uint64_t lo = v.x | ((uint64_t)v.y << 32), hi = v.z | ((uint64_t)v.w << 32);
  const uint32_t s = n * bits, t = s & 63u;
  const uint64_t cross = t ? hi << (64u - t) : 0ull;
  const uint64_t l = s < 64u ? (lo >> t) | cross : s < 128u ? hi >> t : 0ull;
  const uint64_t h = s < 64u ? hi >> t : 0ull;
  return u32x4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
}

// Column from which the vector of columns [e, e + 8) is loaded.
template <Edge EDGE>
__device__ __forceinline__ uint32_t inside(uint32_t e, uint32_t hidden) {
  if constexpr (EDGE == kOdd) return e + 8u <= hidden ? e : hidden - 8u;
  return e < hidden ? e : 0u;
}

// The 16 bytes that hold bf16 columns [e, e + 8) of a row, where they are in
// the row (take8 puts zeros past its end).
template <Edge EDGE, bool NT>
__device__ __forceinline__ u32x4 load8_bf16(const uint16_t *row, uint32_t e, uint32_t hidden) {
  if constexpr (EDGE == kTiny) {
    u32x4 w = {0u, 0u, 0u, 0u};
    for (uint32_t j = 0; j < hidden; ++j) w[j >> 1] |= (uint32_t)row[j] << (16 * (j & 1));
    return w;
  }
  return load16<NT>(row + inside<EDGE>(e, hidden));
}

// Columns [e, e + 8) from what load8_bf16 returned, zeros past the row's end.
template <Edge EDGE>
__device__ __forceinline__ u32x4 take8_bf16(u32x4 v, uint32_t e, uint32_t hidden) {
  const u32x4 zero = {0u, 0u, 0u, 0u};
  if constexpr (EDGE == kTiny) return e ? zero : v;
  if constexpr (EDGE == kOdd) return e + 8u <= hidden ? v : shift_down(v, e + 8u - hidden, 16u);
  return e < hidden ? v : zero;
}

// The same for codes.
template <Edge EDGE, bool NT>
__device__ __forceinline__ u32x2 load8_codes(const uint8_t *row, uint32_t e, uint32_t hidden) {
  if constexpr (EDGE == kTiny) {
    u32x2 w = {0u, 0u};
    for (uint32_t j = 0; j < hidden; ++j) w[j >> 2] |= (uint32_t)row[j] << (8 * (j & 3));
    return w;
  }
  return load8<NT>(row + inside<EDGE>(e, hidden));
}

template <Edge EDGE>
__device__ __forceinline__ u32x2 take8_codes(u32x2 v, uint32_t e, uint32_t hidden) {
  const u32x2 zero = {0u, 0u};
  if constexpr (EDGE == kTiny) return e ? zero : v;
  if constexpr (EDGE == kOdd) {
    const u32x4 w = shift_down(u32x4{v.x, v.y, 0u, 0u}, e + 8u - hidden, 8u);
    return e + 8u <= hidden ? v : u32x2{w.x, w.y};
  }
  return e < hidden ? v : zero;
}

// Ends a group of loads: nothing is moved across, so that the loads before it
// are all in flight before the first wait.  (Left to itself the compiler
// saves registers by waiting for each load before it issues the next.)
__device__ __forceinline__ void loads_issued() { __builtin_amdgcn_sched_barrier(0); }

// The elements of [e, e + 8) that are inside the row.  Callers have e < hidden.
template <Edge EDGE, bool NT>
__device__ __forceinline__ void store8_bf16(uint16_t *row, uint32_t e, uint32_t hidden, u32x4 v) {
  if (EDGE == kEven || e + 8u <= hidden) {
    store16<NT>(row + e, v);
    return;
  }
  for (uint32_t j = 0; e + j < hidden; ++j) row[e + j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
}

template <Edge EDGE, bool NT>
__device__ __forceinline__ void store8_codes(uint8_t *row, uint32_t e, uint32_t hidden, u32x2 v) {
  if (EDGE == kEven || e + 8u <= hidden) {
    store8<NT>(row + e, v);
    return;
  }
  for (uint32_t j = 0; e + j < hidden; ++j) row[e + j] = (uint8_t)(v[j >> 2] >> (8 * (j & 3)));
}

template <Edge EDGE, bool NT>
__device__ __forceinline__ void store8_f32(float *row, uint32_t e, uint32_t hidden, const float (&f)[8]) {
  if (EDGE == kEven || e + 8u <= hidden) {
    store16<NT>(row + e, __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]}));
    store16<NT>(row + e + 4, __builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]}));
    return;
  }
#pragma unroll
  for (uint32_t j = 0; j < 7; ++j)
    if (e + j < hidden) row[e + j] = f[j];
}

__device__ __forceinline__ void widen8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(v[j]);
    f[2 * j + 1] = bf16_hi(v[j]);
  }
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two fp32 values as bf16, round to nearest even (one conversion on gfx950).
__device__ __forceinline__ uint32_t round2_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

__device__ __forceinline__ u32x4 round8_bf16(const float (&f)[8]) {
  return u32x4{round2_bf16(f[0], f[1]), round2_bf16(f[2], f[3]), round2_bf16(f[4], f[5]),
               round2_bf16(f[6], f[7])};
}

// Bits of the largest magnitude of eight values; above every finite value's
// where one is an inf or a NaN (the three-operand maximum hands NaN on).
__device__ __forceinline__ uint32_t amax8_bits(const float (&f)[8]) {
  float m = __builtin_elementwise_maximum(
      __builtin_elementwise_maximum(__builtin_fabsf(f[0]), __builtin_fabsf(f[1])), __builtin_fabsf(f[2]));
#pragma unroll
  for (int j = 3; j < 7; j += 2)
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(f[j])),
                                      __builtin_fabsf(f[j + 1]));
  m = __builtin_elementwise_maximum(m, __builtin_fabsf(f[7]));
  return __float_as_uint(m) & 0x7FFFFFFFu;
}

// Eight weights of a norm, fp32 or bf16 (WB) in memory (the same for every
// row, so the loads may stay in the caches): loaded, and then taken, as rows
// are.
template <Edge EDGE, bool WB>
struct Weights8 {
  u32x4 raw[WB ? 1 : 2];
  __device__ __forceinline__ void load(const void *w, uint32_t e, uint32_t hidden) {
    if constexpr (WB) {
      raw[0] = load8_bf16<EDGE, false>(static_cast<const uint16_t *>(w), e, hidden);
    } else {
      const float *p = static_cast<const float *>(w);
      if constexpr (EDGE != kEven) {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j)
          raw[j / 4][j % 4] = __float_as_uint(p[e + j < hidden ? e + j : 0u]);
      } else {
        raw[0] = load16<false>(p + inside<EDGE>(e, hidden));
        raw[1] = load16<false>(p + inside<EDGE>(e, hidden) + 4);
      }
    }
  }
  __device__ __forceinline__ void take(uint32_t e, uint32_t hidden, float (&f)[8]) const {
    if constexpr (WB) {
      widen8(take8_bf16<EDGE>(raw[0], e, hidden), f);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j)
        f[j] = (EDGE == kEven ? e : e + j) < hidden ? __uint_as_float(raw[j / 4][j % 4]) : 0.0f;
    }
  }
};

}  // namespace fp8q
