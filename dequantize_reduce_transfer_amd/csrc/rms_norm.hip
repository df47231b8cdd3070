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
// Waves are added before vectors: a row of up to 4096 is spread so that each
// lane has one vector, which measured best on MI355X (65536 rows of 2048,
// e4m3, residual: 146 us with 4 waves x 1 vector, 152 with 2 x 2, 154 with
// 1 x 4).  What is left above HBM's own time is instructions, so the kernel has
// no row loop (the host splits launches beyond the grid limit): bases stay in
// scalar registers and lane offsets in 32 bits.  Non-temporal loads and
// stores, and runs of 64 workgroups an XCD, are worth 2-5% at large sizes.
// Measured (median, rotating inputs): 16384 x 8192 e4m3 with residual 151 us,
// 6.24 TB/s, where a plain stream with the same 4 bytes in and 3 out reaches
// 6.36; 65536 x 2048 146 us, 6.45 TB/s; one row of 2048 2.0 us in a graph.
//
// Backward: dx needs one sum over the row, dweight one over the rows.  A
// workgroup walks rows, each row's loads issued a row ahead, keeps its
// dweight sums in registers, and writes them once into the workspace; a
// second kernel adds the workgroups' parts in a fixed order.  Fewer
// workgroups mean fewer parts to write and read back, more of them more loads
// in flight: 2048 waves measured best (16384 x 4096 with the residual's
// gradient, 8 bytes an element: 87 us, 6.2 TB/s, with 256 workgroups of 8
// waves; 89 with 512, 92 with 1024; 32768 x 2048 in 4-wave workgroups: 88 us
// with 512, 112 with 256, 92 with 1024).  The gradients of a few rows, which
// launches bound, and of very wide ones come from one kernel that reads dy and
// h twice.
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
    const uint32_t wid = uniform(threadIdx.x / kWave) % W;
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
  const uint32_t m = amax8_bits(y);
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
    if (wave_any(s.f != 1.0f))
      q = quot8<OUT, true>(y, s);
    else
      q = quot8<OUT, false>(y, s);
  }
  if (!finite) q = u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
  return q;
}

// One row per W waves, V vectors of eight elements a lane (W * V * 512 >=
// hidden); workgroups of max(W, 4) waves.
template <int OUT, bool RES, bool WB, Edge EDGE, int W, int V>
__global__ __launch_bounds__(64 * (W > 4 ? W : 4)) void norm_kernel(NormForward a) {
  constexpr int kRows = W >= 4 ? 1 : 4 / W;              // rows a workgroup
  constexpr uint32_t kThreads = 64 * W;                  // threads a row
  __shared__ float part[kRows * W];
  const uint32_t sub = W >= 4 ? 0 : uniform(threadIdx.x / kThreads);
  const uint32_t tid = threadIdx.x % kThreads;
  const uint32_t hidden = a.hidden;
  const uint64_t row0 = (uint64_t)block_position() * kRows;
  const bool live = row0 + sub < a.rows;                 // the same for the row's waves
  const uint64_t row = live ? row0 + sub : row0;
  const uint64_t base = row * (uint64_t)hidden;
  const uint16_t *x = static_cast<const uint16_t *>(a.x) + base;
  const uint16_t *r = static_cast<const uint16_t *>(a.residual) + base;

  u32x4 xv[V], rv[V];
  Weights8<EDGE, WB> wv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t e = 8 * (v * kThreads + tid);
    xv[v] = load8_bf16<EDGE, true>(x, e, hidden);
    if constexpr (RES) rv[v] = load8_bf16<EDGE, true>(r, e, hidden);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) wv[v].load(a.weight, 8 * (v * kThreads + tid), hidden);
  loads_issued();
  float h[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t e = 8 * (v * kThreads + tid);
    widen8(take8_bf16<EDGE>(xv[v], e, hidden), h[v]);
    if constexpr (RES) {
      float t[8];
      widen8(take8_bf16<EDGE>(rv[v], e, hidden), t);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] += t[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(h[v][j], h[v][j], ss);
  }
  ss = sum_row<W>(ss, part + sub * W);
  if (!live) return;
  const float rstd = rsqrtf(__builtin_fmaf(ss, a.inv_hidden, a.eps));
  if (a.rstd_out && tid == 0) a.rstd_out[row] = rstd;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t i = v * kThreads + tid, e = 8 * i;    // the lane's vector of the row
    float y[8], w[8];
    wv[v].take(e, hidden, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = (h[v][j] * rstd) * w[j];
    if (EDGE == kEven ? e >= hidden : e + 8u > hidden) { // past the row: not 0 * inf where rstd is inf
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) y[j] = e + j < hidden ? y[j] : 0.0f;
    }
    uint32_t scale;
    const u32x2 codes = encode8<OUT>(y, &scale);
    if (e < hidden) {
      if (RES && a.h_out)
        store8_bf16<EDGE, true>(static_cast<uint16_t *>(a.h_out) + base, e, hidden, round8_bf16(h[v]));
      if (a.y_out)
        store8_bf16<EDGE, true>(static_cast<uint16_t *>(a.y_out) + base, e, hidden, round8_bf16(y));
      store8_codes<EDGE, true>(static_cast<uint8_t *>(a.q_out) + base, e, hidden, codes);
      if constexpr (OUT == kMx8) {
        uint8_t *scales = static_cast<uint8_t *>(a.scales_out) + row * (hidden / kMxBlock);
        if ((i & 3) == 0) scales[i / 4] = (uint8_t)scale;
      } else {
        uint32_t *scales = static_cast<uint32_t *>(a.scales_out) + row * ((hidden + kBlock - 1) / kBlock);
        if ((i & 15) == 0) scales[i / 16] = scale;
      }
    }
  }
}

// Launches over all rows, in grids of at most max_workgroups.
template <int OUT, bool RES, bool WB, Edge EDGE, int W, int V>
hipError_t norm_launch(NormForward a, hipStream_t stream) {
  constexpr int kRows = W >= 4 ? 1 : 4 / W, kWgWaves = W > 4 ? W : 4;
  constexpr uint64_t kMost = max_workgroups(kWgWaves) * kRows;
  const uint64_t blocks = OUT == kMx8 ? a.hidden / kMxBlock : (a.hidden + kBlock - 1) / kBlock;
  for (uint64_t left = a.rows; left;) {
    const uint64_t rows = left < kMost ? left : kMost, n = rows * a.hidden;
    a.rows = rows;
    hipLaunchKernelGGL((norm_kernel<OUT, RES, WB, EDGE, W, V>), dim3((uint32_t)((rows + kRows - 1) / kRows)),
                       dim3(64 * kWgWaves), 0, stream, a);
    left -= rows;
    if (!left) break;
    a.x = static_cast<const uint16_t *>(a.x) + n;
    if (RES) a.residual = static_cast<const uint16_t *>(a.residual) + n;
    if (a.h_out) a.h_out = static_cast<uint16_t *>(a.h_out) + n;
    if (a.y_out) a.y_out = static_cast<uint16_t *>(a.y_out) + n;
    a.q_out = static_cast<uint8_t *>(a.q_out) + n;
    a.scales_out = static_cast<uint8_t *>(a.scales_out) + rows * blocks * (OUT == kMx8 ? 1 : 4);
    if (a.rstd_out) a.rstd_out += rows;
  }
  return hipGetLastError();
}

template <int OUT, bool RES, bool WB, Edge EDGE>
hipError_t norm_dispatch(const NormForward &a, hipStream_t stream) {
  if constexpr (EDGE == kTiny) {                         // hidden < 8: no other shape is built
    return norm_launch<OUT, RES, WB, kTiny, 1, 1>(a, stream);
  } else {
    if (a.hidden <= 512) return norm_launch<OUT, RES, WB, EDGE, 1, 1>(a, stream);
    if (a.hidden <= 1024) return norm_launch<OUT, RES, WB, EDGE, 2, 1>(a, stream);
    if (a.hidden <= 2048) return norm_launch<OUT, RES, WB, EDGE, 4, 1>(a, stream);
    if (a.hidden <= 4096) return norm_launch<OUT, RES, WB, EDGE, 8, 1>(a, stream);
    if (a.hidden <= 8192) return norm_launch<OUT, RES, WB, EDGE, 8, 2>(a, stream);
    if (a.hidden <= 16384) return norm_launch<OUT, RES, WB, EDGE, 16, 2>(a, stream);
    return norm_launch<OUT, RES, WB, EDGE, 16, 4>(a, stream);
  }
}

template <int OUT, Edge EDGE>
hipError_t norm_rows(const NormForward &a, hipStream_t stream) {
  if (a.residual)
    return a.weight_bf16 ? norm_dispatch<OUT, true, true, EDGE>(a, stream)
                         : norm_dispatch<OUT, true, false, EDGE>(a, stream);
  return a.weight_bf16 ? norm_dispatch<OUT, false, true, EDGE>(a, stream)
                       : norm_dispatch<OUT, false, false, EDGE>(a, stream);
}

// Floats from one workgroup's dweight sums to the next one's in the workspace.
__host__ __device__ constexpr uint32_t part_stride(uint32_t hidden) { return (hidden + 7) / 8 * 8; }

// What a lane holds of a row.
template <Edge EDGE, int W, int V>
struct BackwardRow {
  u32x4 dy[V], h[V], dh[V];
  float rstd;
  __device__ __forceinline__ void load(const NormBackward &a, uint64_t row, uint32_t tid) {
    uint64_t base = row * (uint64_t)a.hidden;
    asm volatile("" : "+s"(base));       // keeps a scalar base and 32-bit offsets in the row loop
    const uint16_t *yp = static_cast<const uint16_t *>(a.dy) + base;
    const uint16_t *hp = static_cast<const uint16_t *>(a.h) + base;
    const uint16_t *sp = static_cast<const uint16_t *>(a.dh) + base;
    rstd = a.rstd[row];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t e = 8 * (v * 64 * W + tid);
      dy[v] = load8_bf16<EDGE, true>(yp, e, a.hidden);
      h[v] = load8_bf16<EDGE, true>(hp, e, a.hidden);
      if (a.dh) dh[v] = load8_bf16<EDGE, true>(sp, e, a.hidden);
    }
    loads_issued();
  }
};

// The lane's part of sum(weight * dy * h) over the row; settles dy and h past
// the row's end.
template <Edge EDGE, int W, int V>
__device__ __forceinline__ float backward_dot(BackwardRow<EDGE, W, V> &r, const float (&w)[V][8],
                                              uint32_t tid, uint32_t hidden) {
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t e = 8 * (v * 64 * W + tid);
    float y[8], h[8];
    r.dy[v] = take8_bf16<EDGE>(r.dy[v], e, hidden);
    r.h[v] = take8_bf16<EDGE>(r.h[v], e, hidden);
    widen8(r.dy[v], y);
    widen8(r.h[v], h);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(y[j] * w[v][j], h[j], sum);
  }
  return sum;
}

// The lane's dx, with the row's sum: (g - h * c) * rstd + dh, whose c is of the
// order of g * rstd.  rstd^3 leaves fp32's range for rows whose dx is well
// inside it.
template <Edge EDGE, int W, int V>
__device__ __forceinline__ void backward_dx(const NormBackward &a, const BackwardRow<EDGE, W, V> &r,
                                            const float (&w)[V][8], float sum, uint64_t row,
                                            uint32_t tid, bool live) {
  const float c = sum * a.inv_hidden * r.rstd * r.rstd;
  uint64_t base = row * (uint64_t)a.hidden;
  asm volatile("" : "+s"(base));
  uint16_t *dx = static_cast<uint16_t *>(a.dx) + base;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t e = 8 * (v * 64 * W + tid);
    float y[8], h[8], d[8];
    widen8(r.dy[v], y);
    widen8(r.h[v], h);
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = 0.0f;
    if (a.dh) widen8(take8_bf16<EDGE>(r.dh[v], e, a.hidden), d);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      d[j] = __builtin_fmaf(__builtin_fmaf(-h[j], c, y[j] * w[v][j]), r.rstd, d[j]);
    if (live && e < a.hidden) store8_bf16<EDGE, false>(dx, e, a.hidden, round8_bf16(d));
  }
}

template <bool WB, Edge EDGE, int W, int V>
__device__ __forceinline__ void backward_weights(const NormBackward &a, uint32_t tid, float (&w)[V][8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t e = 8 * (v * 64 * W + tid);
    Weights8<EDGE, WB> raw;
    raw.load(a.weight, e, a.hidden);
    raw.take(e, a.hidden, w[v]);
  }
}

// W waves walk rows, each row's loads issued before the sum of the one
// before; workgroups of max(W, 4) waves.  A workgroup's dweight sums go to
// parts[blockIdx.x].  The row sum's LDS slot alternates, so one barrier a row
// is enough: a wave that is a row ahead writes the other slot, and it can only
// be two ahead once every wave has passed the barrier between.
template <bool WB, Edge EDGE, int W, int V>
__global__ __launch_bounds__(64 * (W > 4 ? W : 4)) void norm_backward_kernel(NormBackward a, float *parts) {
  constexpr int kRows = W >= 4 ? 1 : 4 / W;              // rows a workgroup has in hand
  constexpr uint32_t kThreads = 64 * W;                  // threads a row
  __shared__ float part[2][kRows * W];
  __shared__ float joined[kRows > 1 ? (kRows - 1) * kThreads * V * 8 : 1];
  const uint32_t sub = W >= 4 ? 0 : uniform(threadIdx.x / kThreads);
  const uint32_t tid = threadIdx.x % kThreads, hidden = a.hidden;
  const uint64_t stride = (uint64_t)gridDim.x * kRows;
  uint64_t row0 = (uint64_t)blockIdx.x * kRows;
  BackwardRow<EDGE, W, V> next;
  next.load(a, row0 + sub < a.rows ? row0 + sub : row0, tid);
  float w[V][8], dw[V][8];
  backward_weights<WB, EDGE, W>(a, tid, w);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = 0.0f;
  for (uint32_t turn = 0; row0 < a.rows; row0 += stride, turn ^= 1) {
    const bool live = row0 + sub < a.rows;               // the same for the row's waves
    BackwardRow<EDGE, W, V> cur = next;
    if (row0 + stride < a.rows)
      next.load(a, row0 + stride + sub < a.rows ? row0 + stride + sub : row0 + stride, tid);
    float sum = backward_dot(cur, w, tid, hidden);
    if (live) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float y[8], h[8];
        widen8(cur.dy[v], y);
        widen8(cur.h[v], h);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[v][j] = __builtin_fmaf(y[j], h[j] * cur.rstd, dw[v][j]);
      }
    }
    sum = sum_row<W>(sum, part[turn] + sub * W);
    backward_dx(a, cur, w, sum, row0 + sub, tid, live);
  }
  if constexpr (kRows > 1) {
    if (sub) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) joined[(((sub - 1) * V + v) * 8 + j) * kThreads + tid] = dw[v][j];
    }
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int q = 0; q < kRows - 1; ++q) dw[v][j] += joined[((q * V + v) * 8 + j) * kThreads + tid];
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {                          // whole vectors, zeros past the row's end
    const uint32_t e = 8 * (v * kThreads + tid);
    if (e < hidden)
      store8_f32<kEven, false>(parts + (uint64_t)blockIdx.x * part_stride(hidden), e, hidden, dw[v]);
  }
}

// dweight over the lane's columns [e, e + 8) of the rows first, first + STEP, ...,
// DEPTH of them loaded at once.
template <Edge EDGE, uint32_t STEP, uint32_t DEPTH>
__device__ __forceinline__ void backward_columns(const NormBackward &a, uint32_t first, uint32_t e, float (&dw)[8]) {
  const uint32_t hidden = a.hidden;
  for (uint64_t row = first; row < a.rows; row += STEP * DEPTH) {
    u32x4 dy[DEPTH], h[DEPTH];
    float rstd[DEPTH];
#pragma unroll
    for (uint32_t k = 0; k < DEPTH; ++k) {
      const uint64_t r = row + k * STEP < a.rows ? row + k * STEP : row;
      dy[k] = load8_bf16<EDGE, false>(static_cast<const uint16_t *>(a.dy) + r * hidden, e, hidden);
      h[k] = load8_bf16<EDGE, false>(static_cast<const uint16_t *>(a.h) + r * hidden, e, hidden);
      rstd[k] = a.rstd[r];
    }
    loads_issued();
#pragma unroll
    for (uint32_t k = 0; k < DEPTH; ++k) {
      if (row + k * STEP >= a.rows) break;
      float y8[8], h8[8];
      widen8(take8_bf16<EDGE>(dy[k], e, hidden), y8);
      widen8(take8_bf16<EDGE>(h[k], e, hidden), h8);
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[j] = __builtin_fmaf(y8[j], h8[j] * rstd[k], dw[j]);
    }
  }
}

// Columns of a workgroup that sums them.  32 fill more of the chip, 64 are
// whole cache lines and half as many workgroups in the rows' way: 509 rows of
// 1000 3.0 us in a graph with 32, 4.0 with 64; 509 of 8192 11.5 and 8.2.
constexpr uint32_t group_columns(int waves) { return waves <= 4 ? 32 : 64; }

// Both gradients in one launch: dweight does not need the rows'
// sums, so the first `column_wgs` workgroups take group_columns of all rows each,
// and the rest the rows, one per W waves.  dy and h are read twice (the second
// time from the caches), in no order: dx must not be dy.  Latency bounds it, so
// a lane's rows are loaded 4 at a time, or 8 where there are more (509 rows of
// 2888, read from HBM: 7.8 us with 8, 8.5 with 4; 200 rows 5.1 and 4.6), and
// all threads add up the lanes' sums, 8 each and then the slices'.
template <bool WB, Edge EDGE, int W, int V>
__global__ __launch_bounds__(64 * (W > 4 ? W : 4)) void norm_backward_columns_kernel(NormBackward a,
                                                                                 uint32_t column_wgs) {
  constexpr int kRows = W >= 4 ? 1 : 4 / W;
  constexpr uint32_t kThreads = 64 * W;                  // threads a row
  constexpr uint32_t kColumns = group_columns(W), kLanes = kColumns / 8;
  constexpr uint32_t kGroups = 64 * (W > 4 ? W : 4) / kLanes, kSlices = kGroups / 8;
  __shared__ float part[kRows * W];
  __shared__ float sums[kGroups][kColumns], slices[kSlices][kColumns];
  const uint32_t hidden = a.hidden;
  if (blockIdx.x < column_wgs) {
    const uint32_t group = threadIdx.x / kLanes, c = 8 * (threadIdx.x % kLanes);
    const uint32_t first = blockIdx.x * kColumns;
    float dw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = 0.0f;
    if (a.rows > 4 * kGroups)
      backward_columns<EDGE, kGroups, 8>(a, group, first + c, dw);
    else
      backward_columns<EDGE, kGroups, 4>(a, group, first + c, dw);
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[group][c + j] = dw[j];
    __syncthreads();
    const uint32_t column = threadIdx.x % kColumns, slice = threadIdx.x / kColumns;
    float t = sums[8 * slice][column];
#pragma unroll
    for (uint32_t g = 1; g < 8; ++g) t += sums[8 * slice + g][column];
    slices[slice][column] = t;
    __syncthreads();
    if (slice == 0 && first + column < hidden) {
#pragma unroll
      for (uint32_t g = 1; g < kSlices; ++g) t += slices[g][column];
      a.dweight[first + column] = t;
    }
    return;
  }
  const uint32_t sub = W >= 4 ? 0 : uniform(threadIdx.x / kThreads);
  const uint32_t tid = threadIdx.x % kThreads;
  const uint64_t row0 = (uint64_t)(blockIdx.x - column_wgs) * kRows;
  const bool live = row0 + sub < a.rows;                 // the same for the row's waves
  BackwardRow<EDGE, W, V> row;
  row.load(a, live ? row0 + sub : row0, tid);
  float w[V][8];
  backward_weights<WB, EDGE, W>(a, tid, w);
  const float sum = sum_row<W>(backward_dot(row, w, tid, hidden), part + sub * W);
  backward_dx(a, row, w, sum, row0 + sub, tid, live);
}

// dweight[e] = parts[0][e] + parts[1][e] + ...  A workgroup takes 64 columns,
// a lane four of them of every 64th part (16 waves x 4 lane groups), and the
// groups' sums are added in order.
constexpr int kPartWaves = 16;
constexpr int kPartGroups = 4 * kPartWaves;
__global__ __launch_bounds__(64 * kPartWaves) void norm_parts_kernel(const float *parts, uint32_t count,
                                                                     uint32_t hidden, float *dweight) {
  __shared__ float sums[kPartGroups][64];
  const uint32_t tid = threadIdx.x, group = tid / 16, c = 4 * (tid % 16);
  const uint32_t e = blockIdx.x * 64 + c;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (e < hidden) {
#pragma unroll 8
    for (uint32_t p = group; p < count; p += kPartGroups) {
      const f32x4 v = __builtin_bit_cast(f32x4, load16<false>(parts + (uint64_t)p * part_stride(hidden) + e));
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) sums[group][c + j] = s[j];
  __syncthreads();
  const uint32_t column = blockIdx.x * 64 + tid;
  if (tid < 64 && column < hidden) {
    float t = sums[0][tid];
#pragma unroll
    for (int g = 1; g < kPartGroups; ++g) t += sums[g][tid];
    dweight[column] = t;
  }
}

// The backward kernel's rows in hand (4 / W where W < 4 waves share a row) and
// its workgroups, at most: 2048 waves in all, and one workgroup a CU at least.
struct BackwardShape {
  uint32_t rows;               // rows a workgroup has in hand
  uint32_t most;               // workgroups
};
constexpr BackwardShape backward_shape(uint32_t hidden) {
  if (hidden <= 512) return {4, 512};
  if (hidden <= 1024) return {2, 512};
  return {1, hidden <= 2048 ? 512u : 256u};
}

// Up to 512 rows both gradients come from one launch.  On MI355X in a graph,
// operands from HBM, one launch against two: 1 row of 2048 1.9 against 4.0 us,
// 256 rows 4.4 against 7.0, 509 rows 7.0 against 10.9, 768 rows 10.1 against
// 9.4; of 512 columns 3.8 against 5.0 (256 rows), 5.6 against 5.6 (509) and
// 8.1 against 6.0 (768); of 16384 columns 18.8 against 26.6 (512).
// Where dx is dy itself it takes two: a row written would be missing from the
// columns' sums.
// Rows of more than 16384 always go this way, their dweight sums being far too
// many for the row kernel's registers: the second reading costs less than what
// it spilled (4096 x 20000 188 us against 741, 4096 x 32768 310 against 831).
// Rows of 8193 to 16384 stay with the row kernel, which spills less there (16
// registers a lane, 30 where hidden % 8 != 0): 4096 x 12288 99 us, 4096 x 16384
// 119, 4096 x 16383 218, from HBM.
constexpr uint64_t kFewRows = 512;
constexpr uint32_t kWideRow = 16384;
bool by_columns(const NormBackward &a) {
  return a.rows == 0 || a.hidden > kWideRow || (a.rows <= kFewRows && a.dx != a.dy);
}

uint32_t backward_wgs(uint64_t rows, uint32_t hidden) {
  if (hidden > kWideRow) return 0;
  const BackwardShape shape = backward_shape(hidden);
  const uint64_t wgs = (rows + shape.rows - 1) / shape.rows;
  return (uint32_t)(wgs < shape.most ? wgs : shape.most);
}

// The columns and, unless dx is dy, rows in one grid; then what rows are left,
// in grids of at most max_workgroups.
template <bool WB, Edge EDGE, int W, int V>
hipError_t columns_launch(NormBackward a, hipStream_t stream) {
  constexpr uint32_t kRows = W >= 4 ? 1 : 4 / W, kWgWaves = W > 4 ? W : 4;
  constexpr uint64_t kMost = max_workgroups(kWgWaves) * kRows;
  uint32_t columns = (a.hidden + group_columns(W) - 1) / group_columns(W);
  uint64_t rows = a.dx == a.dy ? 0 : a.rows < kMost ? a.rows : kMost;
  for (;;) {
    hipLaunchKernelGGL((norm_backward_columns_kernel<WB, EDGE, W, V>),
                       dim3(columns + (uint32_t)((rows + kRows - 1) / kRows)), dim3(64 * kWgWaves), 0, stream, a,
                       columns);
    const uint64_t n = rows * a.hidden;
    a.rows -= rows;
    if (!a.rows) return hipGetLastError();
    a.dy = static_cast<const uint16_t *>(a.dy) + n;
    a.h = static_cast<const uint16_t *>(a.h) + n;
    if (a.dh) a.dh = static_cast<const uint16_t *>(a.dh) + n;
    a.rstd += rows;
    a.dx = static_cast<uint16_t *>(a.dx) + n;
    columns = 0;
    rows = a.rows < kMost ? a.rows : kMost;
  }
}

template <bool WB, Edge EDGE, int W, int V>
hipError_t backward_launch(const NormBackward &a, hipStream_t stream) {
  if (by_columns(a)) return columns_launch<WB, EDGE, W, V>(a, stream);
  const dim3 block(64 * (W > 4 ? W : 4));
  const uint32_t wgs = backward_wgs(a.rows, a.hidden);
  hipLaunchKernelGGL((norm_backward_kernel<WB, EDGE, W, V>), dim3(wgs), block, 0, stream, a, a.workspace);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_parts_kernel, dim3((a.hidden + 63) / 64), dim3(64 * kPartWaves), 0, stream,
                     a.workspace, wgs, a.hidden, a.dweight);
  return hipGetLastError();
}

template <int OUT>
hipError_t norm_edges(const NormForward &a, hipStream_t stream) {
  switch (edge_of(a.hidden)) {
    case kEven: return norm_rows<OUT, kEven>(a, stream);
    case kOdd: return norm_rows<OUT, kOdd>(a, stream);
    default: return norm_rows<OUT, kTiny>(a, stream);
  }
}

template <bool WB, Edge EDGE>
hipError_t backward_dispatch(const NormBackward &a, hipStream_t stream) {
  if constexpr (EDGE == kTiny) {
    return backward_launch<WB, kTiny, 1, 1>(a, stream);
  } else {
    if (a.hidden <= 512) return backward_launch<WB, EDGE, 1, 1>(a, stream);
    if (a.hidden <= 1024) return backward_launch<WB, EDGE, 2, 1>(a, stream);
    if (a.hidden <= 2048) return backward_launch<WB, EDGE, 4, 1>(a, stream);
    if (a.hidden <= 4096) return backward_launch<WB, EDGE, 8, 1>(a, stream);
    if (a.hidden <= 8192) return backward_launch<WB, EDGE, 8, 2>(a, stream);
    if (a.hidden <= kWideRow) return backward_launch<WB, EDGE, 16, 2>(a, stream);
    return columns_launch<WB, EDGE, 16, 4>(a, stream);
  }
}

template <bool WB>
hipError_t backward_edges(const NormBackward &a, hipStream_t stream) {
  switch (edge_of(a.hidden)) {
    case kEven: return backward_dispatch<WB, kEven>(a, stream);
    case kOdd: return backward_dispatch<WB, kOdd>(a, stream);
    default: return backward_dispatch<WB, kTiny>(a, stream);
  }
}

}  // namespace

hipError_t launch_rms_norm(int out, const NormForward &a, hipStream_t stream) {
  if (out == kMx8) return norm_rows<kMx8, kEven>(a, stream);   // hidden % 32 == 0
  return out == 0 ? norm_edges<0>(a, stream) : norm_edges<1>(a, stream);
}

uint64_t norm_backward_workspace(uint64_t rows, uint32_t hidden) {
  return 4ull * backward_wgs(rows, hidden) * part_stride(hidden);
}

hipError_t launch_rms_norm_backward(const NormBackward &a, hipStream_t stream) {
  return a.weight_bf16 ? backward_edges<true>(a, stream) : backward_edges<false>(a, stream);
}

}  // namespace fp8q
