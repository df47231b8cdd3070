// f32_encode.h -- FP8 codes of fp32 values with one fp32 scale per block: the
// encode of the kernels that quantize sums or normed rows held in registers
// (the divide-free quotient and its bounds are described in
// dequant_reduce.hip, at the requantize, and in fp8q_device.h).
#pragma once

#include "fp8q_device.h"

namespace fp8q {

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct F32Scale {
  float s;        // the stored scale (NaN for a non-finite block)
  float sp;       // s * f
  float rp;       // RN(1 / sp)
  float f;        // 2^64 for blocks with amax below 2^-60, else 1
  bool finite;
};

template <int FMT>
__device__ __forceinline__ F32Scale f32_block_scale(uint32_t amax_bits) {
  F32Scale r;
  r.finite = amax_bits < 0x7F800000u;
  const float s = scale_from_amax<FMT>(__uint_as_float(amax_bits));  // = IEEE amax / M
  r.f = amax_bits < 0x21800000u ? 0x1p64f : 1.0f;          // amax < 2^-60
  r.sp = s * r.f;
  r.rp = recip_rn(r.sp);                                    // = IEEE 1 / sp
  r.s = r.finite ? s : __uint_as_float(0x7FC00000u);
  return r;
}

// SCALED = false may only be used where b.f == 1 (it skips x' = v * f).
// The quotient goes to cvt4 with no clamp: |RN(v / s)| <= quotient_bound
// for every v of a finite block (fp8q_device.h).
template <int FMT, bool SCALED = true>
__device__ __forceinline__ float f32_quot(float v, const F32Scale &b) {
  const float xp = SCALED ? v * b.f : v;
  return markstein_quotient(xp, b.sp, b.rp);
}

template <int FOUT, bool SCALED>
__device__ __forceinline__ u32x2 quot8(const float (&a)[8], const F32Scale &sc) {
  return u32x2{cvt4<FOUT>(f32_quot<FOUT, SCALED>(a[0], sc), f32_quot<FOUT, SCALED>(a[1], sc),
                          f32_quot<FOUT, SCALED>(a[2], sc), f32_quot<FOUT, SCALED>(a[3], sc)),
               cvt4<FOUT>(f32_quot<FOUT, SCALED>(a[4], sc), f32_quot<FOUT, SCALED>(a[5], sc),
                          f32_quot<FOUT, SCALED>(a[6], sc), f32_quot<FOUT, SCALED>(a[7], sc))};
}

}  // namespace fp8q
