// moe_rows.hip -- rows to their experts and back on gfx950: permute, combine,
// and combine's backward pass.
//
// All three walk tokens, not places: a token's row (or its gradient) is read
// once and written to, or summed from, its topk places, whose rows are whole
// and contiguous, so every access but the slots' is a run of 16-byte loads or
// stores.  They are bound by HBM bandwidth: the expert rows, topk times as
// many as the tokens', are what moves.  No atomics: each output has one
// writer, and sums run over j in order.
//
// A slot outside [0, row count) is skipped, so that a pair without a place
// (-1) costs nothing and no value in `slots` can lead outside the buffers.
#include "fp8q_device.h"
#include "layer_device.h"
#include "layer_launch.h"

namespace fp8q {
namespace {

constexpr int kWaves = 4;                      // waves a workgroup
constexpr uint32_t kColumns = 8 * kWave;       // elements a wave covers with one vector a lane

typedef u32x4 u32x4_el1 __attribute__((aligned(1)));

// One 1 KiB piece of a token's row (or of its scales) to its places.  Bytes
// past the last whole 16 of the row go one by one.
__device__ __forceinline__ void copy_piece(const uint8_t *src, uint8_t *dst, uint64_t row_bytes,
                                           uint64_t piece, const int *slots, uint32_t topk,
                                           uint64_t dst_rows) {
  const uint64_t b = piece * (16 * kWave) + 16 * lane_id();
  const bool whole = b + 16 <= row_bytes;
  const int n = b < row_bytes ? (int)(row_bytes - b) : 0;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (whole) {
    v = *reinterpret_cast<const u32x4_el1 *>(src + b);
  } else {
    for (int j = 0; j < n; ++j) v[j >> 2] |= (uint32_t)src[b + j] << (8 * (j & 3));
  }
  for (uint32_t j = 0; j < topk; ++j) {
    const int slot = slots[j];
    if (slot < 0 || (uint64_t)slot >= dst_rows) continue;
    uint8_t *d = dst + (uint64_t)slot * row_bytes + b;
    if (whole) {
      *reinterpret_cast<u32x4_el1 *>(d) = v;
    } else {
      for (int i = 0; i < n; ++i) d[i] = (uint8_t)(v[i >> 2] >> (8 * (i & 3)));
    }
  }
}

// One wave a (token, piece); the pieces of a token are its row's, then its
// scales'.
__global__ __launch_bounds__(64 * kWaves) void permute_kernel(MoePermute a, uint64_t row_pieces,
                                                              uint64_t pieces) {
  const uint64_t units = (uint64_t)a.tokens * pieces;
  for (uint64_t u = (uint64_t)blockIdx.x * kWaves + uniform(threadIdx.x / kWave); u < units;
       u += (uint64_t)gridDim.x * kWaves) {
    const uint64_t t = u / pieces, piece = u % pieces;
    const int *slots = a.slots + t * a.topk;
    if (piece < row_pieces)
      copy_piece(static_cast<const uint8_t *>(a.src) + t * a.row_bytes,
                 static_cast<uint8_t *>(a.dst), a.row_bytes, piece, slots, a.topk, a.dst_rows);
    else
      copy_piece(static_cast<const uint8_t *>(a.src_scales) + t * a.scale_row_bytes,
                 static_cast<uint8_t *>(a.dst_scales), a.scale_row_bytes, piece - row_pieces, slots,
                 a.topk, a.dst_rows);
  }
}

constexpr int kBf16 = 0, kE4m3 = 1, kE5m2 = 2, kMx8 = 3;   // fp8q_row_format

// Eight values of the expert row `slot`, from column e on (zeros past its end).
template <int FMT, Edge EDGE>
__device__ __forceinline__ void row_values(const MoeCombine &a, uint64_t slot, uint32_t e,
                                           uint32_t hidden, float (&f)[8]) {
  if constexpr (FMT == kBf16) {
    const uint16_t *row = static_cast<const uint16_t *>(a.rows) + slot * hidden;
    widen8(take8_bf16<EDGE>(load8_bf16<EDGE, false>(row, e, hidden), e, hidden), f);
  } else {
    const uint8_t *row = static_cast<const uint8_t *>(a.rows) + slot * hidden;
    const u32x2 q = take8_codes<EDGE>(load8_codes<EDGE, false>(row, e, hidden), e, hidden);
    const uint32_t c = e < hidden ? e : 0u;
    if constexpr (FMT == kMx8) {
      const uint32_t s = static_cast<const uint8_t *>(a.scales)[slot * (hidden / kMxBlock) + c / kMxBlock];
      const f32x2 v0 = mx_dec2<false>(q.x, s), v1 = mx_dec2<true>(q.x, s);
      const f32x2 v2 = mx_dec2<false>(q.y, s), v3 = mx_dec2<true>(q.y, s);
      f[0] = v0[0], f[1] = v0[1], f[2] = v1[0], f[3] = v1[1];
      f[4] = v2[0], f[5] = v2[1], f[6] = v3[0], f[7] = v3[1];
    } else {
      constexpr int F = FMT == kE4m3 ? 0 : 1;
      const uint64_t blocks = (hidden + kBlock - 1) / kBlock;
      const float s = static_cast<const float *>(a.scales)[slot * blocks + c / kBlock];
      const f32x2 v0 = dec2<F, false>(q.x), v1 = dec2<F, true>(q.x);
      const f32x2 v2 = dec2<F, false>(q.y), v3 = dec2<F, true>(q.y);
      f[0] = v0[0] * s, f[1] = v0[1] * s, f[2] = v1[0] * s, f[3] = v1[1] * s;
      f[4] = v2[0] * s, f[5] = v2[1] * s, f[6] = v3[0] * s, f[7] = v3[1] * s;
    }
  }
}

// One wave a (token, 512 columns).
template <int FMT, Edge EDGE>
__global__ __launch_bounds__(64 * kWaves) void combine_kernel(MoeCombine a, uint32_t pieces) {
  const uint64_t units = (uint64_t)a.tokens * pieces;
  const uint32_t hidden = (uint32_t)a.hidden;
  for (uint64_t u = (uint64_t)blockIdx.x * kWaves + uniform(threadIdx.x / kWave); u < units;
       u += (uint64_t)gridDim.x * kWaves) {
    const uint64_t t = u / pieces;
    const uint32_t e = (uint32_t)(u % pieces) * kColumns + 8 * lane_id();
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t j = 0; j < a.topk; ++j) {
      const int slot = a.slots[t * a.topk + j];
      if (slot < 0 || (uint64_t)slot >= a.row_count) continue;
      const float w = a.weights ? a.weights[t * a.topk + j] : 1.0f;
      float f[8];
      row_values<FMT, EDGE>(a, (uint64_t)slot, e, hidden, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, f[i], acc[i]);
    }
    if (e < hidden) {
      if (a.out_bf16)
        store8_bf16<EDGE, false>(static_cast<uint16_t *>(a.out) + t * hidden, e, hidden, round8_bf16(acc));
      else
        store8_f32<EDGE, false>(static_cast<float *>(a.out) + t * hidden, e, hidden, acc);
    }
  }
}

// One wave a (token, choice): the row's products with dy, and its gradient.
template <Edge EDGE>
__global__ __launch_bounds__(64 * kWaves) void combine_backward_kernel(MoeCombineBackward a) {
  const uint64_t pairs = (uint64_t)a.tokens * a.topk;
  const uint32_t hidden = (uint32_t)a.hidden;
  for (uint64_t p = (uint64_t)blockIdx.x * kWaves + uniform(threadIdx.x / kWave); p < pairs;
       p += (uint64_t)gridDim.x * kWaves) {
    const int slot = a.slots[p];
    float dot = 0.0f;
    if (slot >= 0 && (uint64_t)slot < a.row_count) {
      const float w = a.weights[p];
      const uint16_t *dy = static_cast<const uint16_t *>(a.dy) + p / a.topk * hidden;
      const uint16_t *row = static_cast<const uint16_t *>(a.rows) + (uint64_t)slot * hidden;
      uint16_t *drow = static_cast<uint16_t *>(a.drows) + (uint64_t)slot * hidden;
      for (uint32_t e = 8 * lane_id(); e < hidden; e += kColumns) {
        float g[8], r[8], d[8];
        widen8(take8_bf16<EDGE>(load8_bf16<EDGE, false>(dy, e, hidden), e, hidden), g);
        widen8(take8_bf16<EDGE>(load8_bf16<EDGE, false>(row, e, hidden), e, hidden), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot = __builtin_fmaf(g[i], r[i], dot);
          d[i] = w * g[i];
        }
        store8_bf16<EDGE, false>(drow, e, hidden, round8_bf16(d));
      }
      dot = sum_wave(dot);
    }
    if (lane_id() == 0) a.dweights[p] = dot;
  }
}

}  // namespace

hipError_t launch_moe_permute(const MoePermute &a, hipStream_t stream) {
  const uint64_t row_pieces = (a.row_bytes + 16 * kWave - 1) / (16 * kWave);
  const uint64_t pieces = row_pieces + (a.scale_row_bytes + 16 * kWave - 1) / (16 * kWave);
  hipLaunchKernelGGL(permute_kernel, dim3(grid_for((uint64_t)a.tokens * pieces, kWaves, kWaves)),
                     dim3(64 * kWaves), 0, stream, a, row_pieces, pieces);
  return hipGetLastError();
}

template <int FMT>
static void combine_launch(const MoeCombine &a, hipStream_t stream) {
  const uint32_t pieces = (uint32_t)((a.hidden + kColumns - 1) / kColumns);
  const dim3 grid(grid_for((uint64_t)a.tokens * pieces, kWaves, kWaves)), block(64 * kWaves);
  switch (edge_of(a.hidden)) {
    case kEven: hipLaunchKernelGGL((combine_kernel<FMT, kEven>), grid, block, 0, stream, a, pieces); break;
    case kOdd: hipLaunchKernelGGL((combine_kernel<FMT, kOdd>), grid, block, 0, stream, a, pieces); break;
    default: hipLaunchKernelGGL((combine_kernel<FMT, kTiny>), grid, block, 0, stream, a, pieces); break;
  }
}

hipError_t launch_moe_combine(int format, const MoeCombine &a, hipStream_t stream) {
  switch (format) {
    case kBf16: combine_launch<kBf16>(a, stream); break;
    case kE4m3: combine_launch<kE4m3>(a, stream); break;
    case kE5m2: combine_launch<kE5m2>(a, stream); break;
    default: combine_launch<kMx8>(a, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const MoeCombineBackward &a, hipStream_t stream) {
  const dim3 grid(grid_for((uint64_t)a.tokens * a.topk, kWaves, kWaves)), block(64 * kWaves);
  switch (edge_of(a.hidden)) {
    case kEven: hipLaunchKernelGGL((combine_backward_kernel<kEven>), grid, block, 0, stream, a); break;
    case kOdd: hipLaunchKernelGGL((combine_backward_kernel<kOdd>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((combine_backward_kernel<kTiny>), grid, block, 0, stream, a); break;
  }
  return hipGetLastError();
}

}  // namespace fp8q
