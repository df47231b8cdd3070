// rms_norm.hip -- root-mean-square norm with the residual's addition into
// 8-bit rows, and its backward pass, on gfx950.
//
// Forward, per row, in fp32:
//   h = x + residual,  rstd = 1 / sqrt(sum(h^2) / hidden + eps),
//   y = (h * rstd) * weight,
// and y's blocks become codes and scales by the codec's rules (fp32 scale per
// 128 elements, or E8M0 per 32).  The row stays in registers between the sum
// and the encode, so each input byte is read once and nothing but the outputs
// is written.  It is bound by HBM bandwidth: 2 B (x) + 2 (residual) in, 2 (h)
// + 1 (codes) + 4/128 or 1/32 (scales), + 2 (y) out per element.
//
// A lane holds eight consecutive elements of a vector (16-byte loads), so a
// block of 128 is a 16-lane row and a block of 32 a quad: the block maxima
// are DPP steps, and no LDS is used but for the sum over the row's waves.
//
// Backward: dx needs one sum over the row, dweight one over the rows.  A
// workgroup walks rows, keeps its dweight sums in registers, and writes them
// once into the workspace; a second kernel adds the workgroups' parts in a
// fixed order.
#include "f32_encode.h"
#include "fp8q_device.h"
#include "layer_device.h"
#include "layer_launch.h"

namespace fp8q {
namespace {

constexpr int kMx8 = 2;          // OUT: 0 = E4M3, 1 = E5M2 (fp32 scales), 2 = MXFP8

// Sum over the W waves that share a row; every thread gets it.  `part` is W
// floats of LDS that no other sum in flight uses.
template <int W>
__device__ __forceinline__ float sum_row(float v, float *part) {
  v = sum_wave(v);
  if constexpr (W > 1) {
    const uint32_t wid = uniform(threadIdx.x / kWave);
    if (lane_id() == 0) part[wid] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w];
  }
  return v;
}

// E8M0 code of an fp32 block maximum and the multiplier 2^-X, as
// mx8_quantize.hip has them for bf16: code = max(exponent field, 8) - 8.
struct MxF32 {
  uint32_t code;
  float mul;
  bool finite;
};

__device__ __forceinline__ MxF32 mx_f32_scale(uint32_t amax_bits) {
  MxF32 m;
  const uint32_t e = amax_bits >> 23;
  m.finite = amax_bits < 0x7F800000u;
  const uint32_t code = e > 8u ? e - 8u : 0u;
  m.code = m.finite ? code : 0xFFu;
  m.mul = __uint_as_float((254u - code) << 23);
  return m;
}

// Codes of the lane's eight values of a block, and the block's scale: an fp32
// scale's bits, or an E8M0 code.
template <int OUT>
__device__ __forceinline__ u32x2 encode8(const float (&y)[8], uint32_t *scale) {
  uint32_t m = abs_bits(y[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) m = m > abs_bits(y[j]) ? m : abs_bits(y[j]);
  u32x2 q;
  bool finite;
  if constexpr (OUT == kMx8) {
    const MxF32 s = mx_f32_scale(max_quad(m));
    *scale = s.code;
    finite = s.finite;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      q[j] = cvt4<0>(sat_clamp<0>(y[4 * j] * s.mul), sat_clamp<0>(y[4 * j + 1] * s.mul),
                     sat_clamp<0>(y[4 * j + 2] * s.mul), sat_clamp<0>(y[4 * j + 3] * s.mul));
  } else {
    const F32Scale s = f32_block_scale<OUT>(max_row16(m));
    *scale = __float_as_uint(s.s);
    finite = s.finite;
    q = quot8<OUT, true>(y, s);
  }
  if (!finite) q = u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
  return q;
}

// One row per W waves, V vectors of eight elements a lane (W * V * 512 >=
// hidden); workgroups of max(W, 4) waves.  The grid covers the rows, and
// beyond the grid limit the workgroups stride; the row sum's LDS slot
// alternates between rounds, so the one barrier inside it is enough.
template <int OUT, bool RES, int W, int V>
__global__ __launch_bounds__(64 * (W > 4 ? W : 4)) void norm_kernel(NormForward a) {
  constexpr int kRows = W >= 4 ? 1 : 4 / W;              // rows a workgroup
  constexpr uint32_t kThreads = 64 * W;                  // threads a row
  __shared__ float part[2][kRows * W];
  const uint32_t sub = W >= 4 ? 0 : uniform(threadIdx.x / kThreads);
  const uint32_t tid = threadIdx.x % kThreads;
  const int hidden = (int)a.hidden;
  uint32_t turn = 0;
  for (uint64_t row0 = (uint64_t)blockIdx.x * kRows; row0 < a.rows;
       row0 += (uint64_t)gridDim.x * kRows, turn ^= 1) {
    const uint64_t row = row0 + sub;
    const bool live = row < a.rows;                      // uniform over the row's waves
    const uint64_t base = (live ? row : 0) * (uint64_t)a.hidden;
    const uint16_t *x = static_cast<const uint16_t *>(a.x) + base;
    const uint16_t *r = RES ? static_cast<const uint16_t *>(a.residual) + base : nullptr;

    u32x4 xv[V], rv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 8 * (int)(v * kThreads + tid), n = hidden - e;
      xv[v] = rv[v] = u32x4{0u, 0u, 0u, 0u};
      if (live && n > 0) {
        xv[v] = load8_bf16<false>(x + e, n);
        if constexpr (RES) rv[v] = load8_bf16<false>(r + e, n);
      }
    }
    float h[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      widen8(xv[v], h[v]);
      if constexpr (RES) {
        float t[8];
        widen8(rv[v], t);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[v][j] += t[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(h[v][j], h[v][j], ss);
    }
    ss = sum_row<W>(ss, part[turn] + sub * W);
    const float rstd = 1.0f / sqrtf(ss / (float)hidden + a.eps);
    if (!live) continue;
    if (a.rstd_out && tid == 0) a.rstd_out[row] = rstd;

    uint16_t *ho = a.h_out ? static_cast<uint16_t *>(a.h_out) + base : nullptr;
    uint16_t *yo = a.y_out ? static_cast<uint16_t *>(a.y_out) + base : nullptr;
    uint8_t *q = static_cast<uint8_t *>(a.q_out) + base;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t i = v * kThreads + tid;             // the lane's vector of the row
      const int e = 8 * (int)i, n = hidden - e;
      float y[8];
      if (n > 0) {
        float w[8];
        load8_weight(a.weight, a.weight_bf16, e, n, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = j < n ? (h[v][j] * rstd) * w[j] : 0.0f;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
      }
      uint32_t scale;
      const u32x2 codes = encode8<OUT>(y, &scale);
      if (n > 0) {
        if (RES && ho) store8_bf16<false>(ho + e, round8_bf16(h[v]), n);
        if (yo) store8_bf16<false>(yo + e, round8_bf16(y), n);
        store8_codes<false>(q + e, codes, n);
        if constexpr (OUT == kMx8) {
          if ((i & 3) == 0)
            static_cast<uint8_t *>(a.scales_out)[row * (a.hidden / kMxBlock) + i / 4] = (uint8_t)scale;
        } else {
          const uint32_t blocks = (a.hidden + kBlock - 1) / kBlock;
          if ((i & 15) == 0)
            static_cast<uint32_t *>(a.scales_out)[row * (uint64_t)blocks + i / 16] = scale;
        }
      }
    }
  }
}

template <int OUT, bool RES, int W, int V>
hipError_t norm_launch(const NormForward &a, hipStream_t stream) {
  constexpr int kRows = W >= 4 ? 1 : 4 / W, kWgWaves = W > 4 ? W : 4;
  hipLaunchKernelGGL((norm_kernel<OUT, RES, W, V>), dim3(grid_for(a.rows, kRows, kWgWaves)),
                     dim3(64 * kWgWaves), 0, stream, a);
  return hipGetLastError();
}

template <int OUT, bool RES>
hipError_t norm_dispatch(const NormForward &a, hipStream_t stream) {
  if (a.hidden <= 2048) return norm_launch<OUT, RES, 4, 1>(a, stream);
  if (a.hidden <= 4096) return norm_launch<OUT, RES, 4, 2>(a, stream);
  if (a.hidden <= 8192) return norm_launch<OUT, RES, 4, 4>(a, stream);
  if (a.hidden <= 16384) return norm_launch<OUT, RES, 8, 4>(a, stream);
  return norm_launch<OUT, RES, 16, 4>(a, stream);
}

// A workgroup of W waves walks rows blockIdx.x, blockIdx.x + gridDim.x, ...;
// its dweight sums go to parts[blockIdx.x] (or, alone, to dweight itself).
// The row sum's LDS slot alternates, so one barrier a row is enough: a wave
// that is a row ahead writes the other slot, and it can only be two ahead
// once every wave has passed the barrier between.
template <int W, int V>
__global__ __launch_bounds__(64 * W) void norm_backward_kernel(NormBackward a, float *parts) {
  constexpr uint32_t kThreads = 64 * W;
  __shared__ float part[2][W];
  const uint32_t tid = threadIdx.x;
  const int hidden = (int)a.hidden;
  float w[V][8], dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 8 * (int)(v * kThreads + tid), n = hidden - e;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[v][j] = dw[v][j] = 0.0f;
    if (n > 0) load8_weight(a.weight, a.weight_bf16, e, n, w[v]);
  }
  uint32_t turn = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const uint64_t base = row * (uint64_t)a.hidden;
    const uint16_t *dy = static_cast<const uint16_t *>(a.dy) + base;
    const uint16_t *hp = static_cast<const uint16_t *>(a.h) + base;
    const uint16_t *dh = a.dh ? static_cast<const uint16_t *>(a.dh) + base : nullptr;
    uint16_t *dx = static_cast<uint16_t *>(a.dx) + base;
    const float rstd = a.rstd[row];
    u32x4 yv[V], hv[V], sv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 8 * (int)(v * kThreads + tid), n = hidden - e;
      yv[v] = hv[v] = sv[v] = u32x4{0u, 0u, 0u, 0u};
      if (n > 0) {
        yv[v] = load8_bf16<false>(dy + e, n);
        hv[v] = load8_bf16<false>(hp + e, n);
        if (dh) sv[v] = load8_bf16<false>(dh + e, n);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float y[8], h[8];
      widen8(yv[v], y);
      widen8(hv[v], h);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = __builtin_fmaf(y[j] * w[v][j], h[j], sum);
        dw[v][j] = __builtin_fmaf(y[j], h[j] * rstd, dw[v][j]);
      }
    }
    sum = sum_row<W>(sum, part[turn]);
    const float c = sum / (float)hidden * rstd * rstd * rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 8 * (int)(v * kThreads + tid), n = hidden - e;
      if (n <= 0) continue;
      float y[8], h[8], s[8], d[8];
      widen8(yv[v], y);
      widen8(hv[v], h);
      widen8(sv[v], s);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        d[j] = __builtin_fmaf(-h[j], c, __builtin_fmaf(y[j] * w[v][j], rstd, s[j]));
      store8_bf16<false>(dx + e, round8_bf16(d), n);
    }
  }
  float *out = parts ? parts + (uint64_t)blockIdx.x * a.hidden : a.dweight;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 8 * (int)(v * kThreads + tid), n = hidden - e;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) out[e + j] = dw[v][j];
  }
}

// dweight[e] = parts[0][e] + parts[1][e] + ...: 64 columns a workgroup, each
// wave a run of parts, the waves' sums added in order.
constexpr int kPartWaves = 16;
__global__ __launch_bounds__(64 * kPartWaves) void norm_parts_kernel(const float *parts,
                                                                     uint32_t count, uint32_t hidden,
                                                                     float *dweight) {
  __shared__ float sums[kPartWaves][64];
  const uint32_t lane = lane_id(), wid = uniform(threadIdx.x / kWave);
  const uint32_t e = blockIdx.x * 64 + lane;
  const uint32_t run = (count + kPartWaves - 1) / kPartWaves;
  const uint32_t first = wid * run, last = first + run < count ? first + run : count;
  float s = 0.0f;
  if (e < hidden)
    for (uint32_t p = first; p < last; ++p) s += parts[(uint64_t)p * hidden + e];
  sums[wid][lane] = s;
  __syncthreads();
  if (wid == 0 && e < hidden) {
    s = sums[0][lane];
#pragma unroll
    for (int w = 1; w < kPartWaves; ++w) s += sums[w][lane];
    dweight[e] = s;
  }
}

// Workgroups of the backward kernel: at most kBackwardWgs.
constexpr uint64_t kBackwardWgs = 1024;
uint32_t backward_wgs(uint64_t rows) { return (uint32_t)(rows < kBackwardWgs ? rows : kBackwardWgs); }

template <int W, int V>
hipError_t backward_launch(const NormBackward &a, hipStream_t stream) {
  const uint32_t wgs = backward_wgs(a.rows);
  float *parts = wgs > 1 ? a.workspace : nullptr;
  if (wgs) {
    hipLaunchKernelGGL((norm_backward_kernel<W, V>), dim3(wgs), dim3(64 * W), 0, stream, a, parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (wgs != 1)
    hipLaunchKernelGGL(norm_parts_kernel, dim3((a.hidden + 63) / 64), dim3(64 * kPartWaves), 0,
                       stream, parts, wgs, a.hidden, a.dweight);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(int out, const NormForward &a, hipStream_t stream) {
  const bool res = a.residual != nullptr;
  if (out == 0) return res ? norm_dispatch<0, true>(a, stream) : norm_dispatch<0, false>(a, stream);
  if (out == 1) return res ? norm_dispatch<1, true>(a, stream) : norm_dispatch<1, false>(a, stream);
  return res ? norm_dispatch<kMx8, true>(a, stream) : norm_dispatch<kMx8, false>(a, stream);
}

uint64_t norm_backward_workspace(uint64_t rows, uint32_t hidden) {
  const uint32_t wgs = backward_wgs(rows);
  return wgs > 1 ? 4ull * wgs * hidden : 0;
}

hipError_t launch_rms_norm_backward(const NormBackward &a, hipStream_t stream) {
  if (a.hidden <= 2048) return backward_launch<4, 1>(a, stream);
  if (a.hidden <= 4096) return backward_launch<4, 2>(a, stream);
  if (a.hidden <= 8192) return backward_launch<8, 2>(a, stream);
  if (a.hidden <= 16384) return backward_launch<16, 2>(a, stream);
  return backward_launch<16, 4>(a, stream);
}

}  // namespace fp8q
