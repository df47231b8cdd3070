// moe_route.hip -- a router's logits into each token's experts and their
// weights, and the gradient of the logits, on gfx950.
//
// A token is a group of G lanes (16, 32 or 64, so several tokens may share a
// wave), which hold its logits in registers, V neighbouring ones a lane.  The
// choices are made one after the other: the largest of a lane's values, of the
// group's by DPP and shuffles, and of the lanes that hold it the lowest, which
// takes its lowest one out.  So equal logits go to the lower index, and no
// logit is read twice.
//
// A logit is ordered as an integer (its bits, with the magnitude of negative
// ones turned round): NaN, made the largest, needs no care then, and -inf, which
// is no candidate, is known by its value.
//
// The bytes are few (9.4 MB at 16384 tokens of 128 experts, 1.5 us at what a
// large copy reaches); the chain of choices and the launch bound it.
#include "fp8q_device.h"
#include "layer_device.h"
#include "model_launch.h"

namespace fp8q {
namespace {

constexpr int kNoLogit = INT32_MIN;                     // behind the last expert, or taken
constexpr int kMinusInf = (int)0x807FFFFFu;             // order_of(-inf)

// An integer that orders as the logit does; -0 as +0, every NaN as the largest.
__device__ __forceinline__ int order_of(float l) {
  const int b = __float_as_int(l + 0.0f);
  return l != l ? INT32_MAX : b ^ ((b >> 31) & 0x7FFFFFFF);
}

// The logit again (a NaN where it was one).
__device__ __forceinline__ float logit_of(int order) {
  return __int_as_float(order ^ ((order >> 31) & 0x7FFFFFFF));
}

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}

// Largest value of the group, on each of its lanes.
template <int G>
__device__ __forceinline__ int max_group(int v) {
  const auto larger = [](int a, int b) { return a > b ? a : b; };
  v = larger(v, dpp<kDppQuadXor1>(v));
  v = larger(v, dpp<kDppQuadXor2>(v));
  v = larger(v, dpp<kDppRowHalfMirror>(v));
  v = larger(v, dpp<kDppRowMirror>(v));
  if constexpr (G >= 32) v = larger(v, __shfl_xor(v, 16));
  if constexpr (G >= 64) v = larger(v, __shfl_xor(v, 32));
  return v;
}

// Sum over the group, the same bits on each of its lanes.
template <int G>
__device__ __forceinline__ float sum_group(float v) {
  v = dpp_add<kDppQuadXor1>(v);
  v = dpp_add<kDppQuadXor2>(v);
  v = dpp_add<kDppRowHalfMirror>(v);
  v = dpp_add<kDppRowMirror>(v);
  if constexpr (G >= 32) v += __shfl_xor(v, 16);
  if constexpr (G >= 64) v += __shfl_xor(v, 32);
  return v;
}

// A lane's V logits of a row, -inf behind its end.  A row starts at any
// element, so a lane whose V are all inside loads them as vectors of any
// alignment, and the others one by one.
template <int V, bool BF16>
__device__ __forceinline__ void load_logits(const void *logits, uint64_t t, uint32_t experts, uint32_t e0,
                                            float (&l)[V]) {
  if constexpr (BF16) {
    const uint16_t *row = static_cast<const uint16_t *>(logits) + t * experts;
    if constexpr (V % 8 == 0) {
      if (experts % V == 0) {
        if (e0 < experts) {
#pragma unroll
          for (int i = 0; i < V; i += 8) {
            const u32x4 v = load16<false>(row + e0 + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              l[i + 2 * j] = bf16_lo(v[j]);
              l[i + 2 * j + 1] = bf16_hi(v[j]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) l[i] = -INFINITY;
        }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < experts ? __uint_as_float((uint32_t)row[e0 + i] << 16) : -INFINITY;
  } else {
    const float *row = static_cast<const float *>(logits) + t * experts;
    if constexpr (V % 4 == 0) {
      if (experts % V == 0) {
        if (e0 < experts) {
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            const u32x4 v = load16<false>(row + e0 + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) l[i + j] = __uint_as_float(v[j]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) l[i] = -INFINITY;
        }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < experts ? row[e0 + i] : -INFINITY;
  }
}

constexpr int kRouteWaves = 4;

template <int G, int V, bool BF16>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(const void *logits, uint64_t tokens, uint32_t experts,
                                                                 uint32_t topk, uint32_t normalize, float *weights,
                                                                 int *ids) {
  const uint32_t lane = lane_id(), g = lane % G;
  const uint64_t token = ((uint64_t)blockIdx.x * kRouteWaves + threadIdx.x / kWave) * (kWave / G) + lane / G;
  const uint64_t t = token < tokens ? token : tokens - 1;   // what is past the end is done twice, not written
  const uint32_t e0 = g * V;
  float l[V];
  load_logits<V, BF16>(logits, t, experts, e0, l);
  int order[V];
#pragma unroll
  for (int i = 0; i < V; ++i) order[i] = e0 + i < experts ? order_of(l[i]) : kNoLogit;
  float most = 0.0f, sum = 0.0f, mine = 0.0f;
  for (uint32_t j = 0; j < topk; ++j) {
    int best = order[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = order[i] > best ? order[i] : best;
    const int top = max_group<G>(best);
    if (j == 0) {
      most = top <= kMinusInf ? 0.0f : logit_of(top);
      if (!normalize) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) s += order[i] <= kMinusInf ? 0.0f : expf(l[i] - most);
        sum = sum_group<G>(s);
      }
    }
    const bool none = top <= kMinusInf;
    // the lowest lane of the group that holds it
    const uint64_t all = __builtin_amdgcn_ballot_w64(best == top);
    const uint64_t below = all & ((1ull << lane) - 1ull) & (~0ull << (lane - g));
    const bool winner = best == top && below == 0;
    uint32_t at = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) at = order[i] == top ? (uint32_t)i : at;
    if (winner) {
#pragma unroll
      for (int i = 0; i < V; ++i) order[i] = at == (uint32_t)i ? kNoLogit : order[i];
      if (token < tokens) ids[t * topk + j] = none ? -1 : (int)(e0 + at);
    }
    const float e = none ? 0.0f : expf(logit_of(top) - most);
    if (normalize) sum += e;
    mine = g != j ? mine : none ? -1.0f : e;
  }
  if (token < tokens && g < topk) weights[t * topk + g] = mine == -1.0f ? 0.0f : mine / sum;
}

// A lane's V values of a row, inside it.
template <int V, bool BF16>
__device__ __forceinline__ void store_logits(void *out, uint64_t t, uint32_t experts, uint32_t e0, const float (&d)[V]) {
  if constexpr (BF16) {
    uint16_t *row = static_cast<uint16_t *>(out) + t * experts;
    if constexpr (V % 8 == 0) {
      if (experts % V == 0) {
        if (e0 < experts)
#pragma unroll
          for (int i = 0; i < V; i += 8)
            store16<false>(row + e0 + i, u32x4{round2_bf16(d[i], d[i + 1]), round2_bf16(d[i + 2], d[i + 3]),
                                               round2_bf16(d[i + 4], d[i + 5]), round2_bf16(d[i + 6], d[i + 7])});
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < experts) row[e0 + i] = (uint16_t)round2_bf16(d[i], 0.0f);
  } else {
    float *row = static_cast<float *>(out) + t * experts;
    if constexpr (V % 4 == 0) {
      if (experts % V == 0) {
        if (e0 < experts)
#pragma unroll
          for (int i = 0; i < V; i += 4)
            store16<false>(row + e0 + i, __builtin_bit_cast(u32x4, f32x4{d[i], d[i + 1], d[i + 2], d[i + 3]}));
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < experts) row[e0 + i] = d[i];
  }
}

// The choices' gradients go to every lane of the group one after the other,
// and a lane adds those of its experts, in the order of the choices.
template <int G, int V, bool BF16>
__global__ __launch_bounds__(64 * kRouteWaves) void route_backward_kernel(const float *dweights, const void *logits,
                                                                          const float *weights, const int *ids,
                                                                          uint64_t tokens, uint32_t experts,
                                                                          uint32_t topk, uint32_t normalize,
                                                                          void *dlogits) {
  const uint32_t lane = lane_id(), g = lane % G;
  const uint64_t token = ((uint64_t)blockIdx.x * kRouteWaves + threadIdx.x / kWave) * (kWave / G) + lane / G;
  const uint64_t t = token < tokens ? token : tokens - 1;
  const uint32_t e0 = g * V;
  float d[V];
  int id = -1;
  float w = 0.0f, dw = 0.0f;
  if (g < topk) {
    id = ids[t * topk + g];
    w = weights[t * topk + g];
    dw = dweights[t * topk + g];
  }
  if (id < 0 || id >= (int)experts) {
    id = -1;
    w = dw = 0.0f;
  }
  const float s = sum_group<G>(w * dw);
  if (normalize) {
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.0f;
  } else {
    float l[V];
    load_logits<V, BF16>(logits, t, experts, e0, l);
    int best = kNoLogit;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int o = order_of(l[i]);
      best = o > best ? o : best;
    }
    best = max_group<G>(best);
    const float most = best <= kMinusInf ? 0.0f : logit_of(best);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      d[i] = l[i] == -INFINITY ? 0.0f : expf(l[i] - most);
      sum += d[i];
    }
    sum = sum_group<G>(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = l[i] == -INFINITY ? 0.0f : -(d[i] / sum) * s;
  }
  const float mine = id < 0 ? 0.0f : normalize ? w * (dw - s) : w * dw;
  for (uint32_t j = 0; j < topk; ++j) {
    const int from = (int)(lane - g + j);
    const uint32_t at = (uint32_t)__shfl(id, from) - e0;
    const float v = __shfl(mine, from);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = at == (uint32_t)i ? d[i] + v : d[i];
  }
  if (token < tokens) store_logits<V, BF16>(dlogits, t, experts, e0, d);
}

// Lanes a token, and values a lane.  A group has a lane for each choice, and at
// most eight values a lane up to 512 experts.
uint32_t group_lanes(uint32_t experts, uint32_t topk) {
  if (experts <= 128 && topk <= 16) return 16;
  return experts <= 256 && topk <= 32 ? 32 : 64;
}

template <typename Launch>
hipError_t each_grid(uint64_t tokens, uint32_t lanes, Launch &&launch) {
  const uint64_t per = kRouteWaves * (kWave / lanes);    // tokens a workgroup
  const uint64_t most = FP8Q_MODEL_MAX_WAVES / kRouteWaves < 1 ? 1 : FP8Q_MODEL_MAX_WAVES / kRouteWaves;
  for (uint64_t t = 0; t < tokens; t += most * per) {
    const uint64_t n = tokens - t < most * per ? tokens - t : most * per;
    launch(t, n, (uint32_t)((n + per - 1) / per));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int G, int V, bool BF16>
hipError_t route_launch(const MoeRoute &a, hipStream_t stream) {
  return each_grid(a.tokens, G, [&](uint64_t t, uint64_t n, uint32_t grid) {
    hipLaunchKernelGGL((route_kernel<G, V, BF16>), dim3(grid), dim3(64 * kRouteWaves), 0, stream,
                       static_cast<const uint8_t *>(a.logits) + t * a.experts * (BF16 ? 2 : 4), n, a.experts, a.topk,
                       a.normalize ? 1u : 0u, a.weights + t * a.topk, a.ids + t * a.topk);
  });
}

template <int G, int V, bool BF16>
hipError_t route_launch(const MoeRouteBackward &a, hipStream_t stream) {
  return each_grid(a.tokens, G, [&](uint64_t t, uint64_t n, uint32_t grid) {
    const uint64_t at = t * a.experts * (BF16 ? 2 : 4);
    hipLaunchKernelGGL((route_backward_kernel<G, V, BF16>), dim3(grid), dim3(64 * kRouteWaves), 0, stream,
                       a.dweights + t * a.topk, static_cast<const uint8_t *>(a.logits) + at, a.weights + t * a.topk,
                       a.ids + t * a.topk, n, a.experts, a.topk, a.normalize ? 1u : 0u,
                       static_cast<uint8_t *>(a.dlogits) + at);
  });
}

// The kernel whose group and values a lane hold `experts` logits.
template <bool BF16, typename Args>
hipError_t by_shape(const Args &a, hipStream_t stream) {
  const uint32_t lanes = group_lanes(a.experts, a.topk), per = (a.experts + lanes - 1) / lanes;
  if (lanes == 16) return per <= 1 ? route_launch<16, 1, BF16>(a, stream)
                        : per <= 4 ? route_launch<16, 4, BF16>(a, stream)
                                   : route_launch<16, 8, BF16>(a, stream);
  if (lanes == 32) return per <= 4 ? route_launch<32, 4, BF16>(a, stream) : route_launch<32, 8, BF16>(a, stream);
  return per <= 4   ? route_launch<64, 4, BF16>(a, stream)
         : per <= 8 ? route_launch<64, 8, BF16>(a, stream)
                    : route_launch<64, 16, BF16>(a, stream);
}

}  // namespace

hipError_t launch_moe_route(const MoeRoute &a, hipStream_t stream) {
  return a.bf16 ? by_shape<true>(a, stream) : by_shape<false>(a, stream);
}

hipError_t launch_moe_route_backward(const MoeRouteBackward &a, hipStream_t stream) {
  return a.bf16 ? by_shape<true>(a, stream) : by_shape<false>(a, stream);
}

}  // namespace fp8q
