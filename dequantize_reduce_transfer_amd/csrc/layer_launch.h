// layer_launch.h -- internal launchers behind include/fp8q_layer.h (not
// exported).
//
// Each launcher assumes arguments that the C-ABI layer has validated: present,
// aligned, disjoint where they must be, sizes above zero and within the
// header's limits.  It only sizes the grid and enqueues on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

// Workgroups of `waves` waves in one grid, at most: FP8Q_LAYER_MAX_WAVES waves
// (2^30 work-items, well inside the dispatch packet's 32 bits).  Launchers
// split what is more into several launches.
#ifndef FP8Q_LAYER_MAX_WAVES
#define FP8Q_LAYER_MAX_WAVES (1ull << 24)
#endif
constexpr uint64_t max_workgroups(uint32_t waves) {
  return FP8Q_LAYER_MAX_WAVES < waves ? 1 : FP8Q_LAYER_MAX_WAVES / waves;
}

struct NormForward {
  const void *x;
  const void *residual;       // or null
  const void *weight;
  bool weight_bf16;
  float eps;
  uint32_t hidden;
  float inv_hidden;           // 1 / hidden
  uint64_t rows;
  void *h_out;                // or null
  void *y_out;                // or null
  void *q_out;
  void *scales_out;           // fp32 or E8M0
  float *rstd_out;            // or null
};

// out: 0 = E4M3 and 1 = E5M2 with fp32 scales per 128, 2 = MXFP8.
hipError_t launch_rms_norm(int out, const NormForward &a, hipStream_t stream);

struct NormBackward {
  const void *dy;
  const void *h;
  const void *weight;
  bool weight_bf16;
  const float *rstd;
  const void *dh;             // or null
  uint32_t hidden;
  float inv_hidden;           // 1 / hidden
  uint64_t rows;              // 0 is allowed: dweight is cleared
  void *dx;
  float *dweight;
  float *workspace;           // norm_backward_workspace bytes
};
uint64_t norm_backward_workspace(uint64_t rows, uint32_t hidden);
hipError_t launch_rms_norm_backward(const NormBackward &a, hipStream_t stream);

struct MoeSort {
  const void *ids;
  bool ids64;
  uint32_t pairs;             // tokens * topk; 0 is allowed: offsets are cleared
  uint32_t experts;
  int *slots;
  int *pairs_out;
  int *offsets;
  uint32_t *workspace;        // moe_sort_workspace bytes
};
uint64_t moe_sort_workspace(uint32_t pairs, uint32_t experts);
hipError_t launch_moe_sort(const MoeSort &a, hipStream_t stream);

struct MoePermute {
  const void *src;
  const void *src_scales;
  uint64_t row_bytes;
  uint64_t scale_row_bytes;
  const int *slots;
  uint32_t tokens;
  uint32_t topk;
  uint64_t dst_rows;
  void *dst;
  void *dst_scales;
  void advance(uint64_t n) {  // past the first n tokens
    src = static_cast<const uint8_t *>(src) + n * row_bytes;
    if (src_scales) src_scales = static_cast<const uint8_t *>(src_scales) + n * scale_row_bytes;
  }
};
hipError_t launch_moe_permute(const MoePermute &a, hipStream_t stream);

struct MoeCombine {
  const void *rows;
  const void *scales;         // or null
  const int *slots;
  const float *weights;       // or null
  uint32_t tokens;
  uint32_t topk;
  uint64_t row_count;
  uint64_t hidden;
  void *out;
  bool out_bf16;
  void advance(uint64_t n) {
    if (weights) weights += n * topk;
    out = static_cast<uint8_t *>(out) + n * hidden * (out_bf16 ? 2 : 4);
  }
};
// format: the fp8q_row_format values.
hipError_t launch_moe_combine(int format, const MoeCombine &a, hipStream_t stream);

struct MoeCombineBackward {
  const void *dy;
  const void *rows;
  const int *slots;
  const float *weights;
  uint32_t tokens;
  uint32_t topk;
  uint64_t row_count;
  uint64_t hidden;
  void *drows;
  float *dweights;
  void advance(uint64_t n) {
    dy = static_cast<const uint16_t *>(dy) + n * hidden;
    weights += n * topk;
    dweights += n * topk;
  }
};
hipError_t launch_moe_combine_backward(const MoeCombineBackward &a, hipStream_t stream);

}  // namespace fp8q
