// model_launch.h -- internal launchers behind include/fp8q_model.h (not
// exported).
//
// Each launcher assumes arguments that the C-ABI layer has validated: present,
// aligned, disjoint where they must be, sizes above zero (unless a comment
// allows it) and within the header's limits.  It only sizes the grid and
// enqueues on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

// Workgroups of `waves` waves in one grid, at most: FP8Q_MODEL_MAX_WAVES waves
// (2^30 work-items, well inside the dispatch packet's 32 bits).  Launchers
// split what is more into several launches, or let a workgroup take several
// pieces.
#ifndef FP8Q_MODEL_MAX_WAVES
#define FP8Q_MODEL_MAX_WAVES (1ull << 24)
#endif

struct MoeRoute {
  const void *logits;
  bool bf16;
  uint64_t tokens;
  uint32_t experts;
  uint32_t topk;
  bool normalize;
  float *weights;
  int *ids;
};
hipError_t launch_moe_route(const MoeRoute &a, hipStream_t stream);

struct MoeRouteBackward {
  const float *dweights;
  const void *logits;         // not read with `normalize`
  bool bf16;
  const float *weights;
  const int *ids;
  uint64_t tokens;
  uint32_t experts;
  uint32_t topk;
  bool normalize;
  void *dlogits;
};
hipError_t launch_moe_route_backward(const MoeRouteBackward &a, hipStream_t stream);

// One matrix of every expert; scales null for bf16.
struct ExpertMatrix {
  const uint8_t *rows;
  const uint8_t *scales;
  uint64_t expert_rows;
};

struct MoeExperts {
  const uint16_t *x;
  const void *ids;
  bool ids64;
  const float *weights;
  ExpertMatrix gate, up, down;
  uint32_t tokens;
  uint32_t topk;
  uint32_t experts;
  uint32_t hidden;
  uint32_t inter;             // 0 is allowed: out is cleared
  void *out;
  bool out_bf16;
  uint16_t *workspace;        // moe_experts_workspace bytes
};
uint64_t moe_experts_workspace(uint32_t pairs, uint32_t experts, uint32_t hidden, uint32_t inter, bool out_bf16);
// format: the fp8q_row_format values.
hipError_t launch_moe_experts(int format, const MoeExperts &a, hipStream_t stream);

// A gradient of a list: kind 0 fp32, 1 bf16, 2 E4M3 and 3 E5M2 codes (with one
// scale per 128, or `one_scale`).
struct Grad {
  void *data;
  const float *scales;
  uint64_t count;             // 0 is allowed
  int kind;
  bool one_scale;
};
uint64_t grad_sumsq_workspace(const Grad *grads, uint64_t n);
hipError_t launch_grad_sumsq(const Grad *grads, uint64_t n, double *sumsq, double *workspace,
                             hipStream_t stream);
// kinds 0 and 1 only: of codes, the caller passes the scales as fp32 values.
hipError_t launch_grad_clip(const Grad *grads, uint64_t n, const double *sumsq, double max_norm,
                            double eps, float *norm, hipStream_t stream);

}  // namespace fp8q
