// grad_clip.hip -- the sum of squares over many gradient tensors, and their
// clipping in place, on gfx950.
//
// The tensors of a list are cut into chunks of equal bytes (the last of a
// tensor shorter), and workgroups walk over the chunks of up to kTensors
// tensors, whose addresses travel as kernel arguments: a call needs no table
// in device memory.  A chunk's tensor is found by bisection over the tensors'
// first chunks, which are scalar loads.
//
// Squares are exact in fp64 (of fp32 values; bf16's and the codes' fp32 ones
// as well), and so is nothing lost or overflown that an fp32 sum would; the
// conversions and fp64 multiply-adds take less than the loads.  A workgroup's
// sum goes to its own place in the workspace, and one more workgroup adds them
// up in order.
#include "fp8q_device.h"
#include "layer_device.h"
#include "model_launch.h"

namespace fp8q {
namespace {

constexpr uint32_t kTensors = 112;        // of a launch: its arguments stay under 4 KiB
constexpr int kGradWaves = 4;
constexpr uint32_t kThreads = 64 * kGradWaves;

struct Table {
  const void *data[kTensors];
  const float *scales[kTensors];
  uint64_t count[kTensors];               // values; bits 56..59 the kind, 60 one scale
  uint32_t first[kTensors + 1];           // first chunk
  uint32_t tensors;
  uint32_t chunk_bytes;                   // a multiple of 512
};

constexpr uint32_t value_bytes(int kind) { return kind == 0 ? 4 : kind == 1 ? 2 : 1; }

struct Chunk {
  const void *data;                       // the tensor's
  const float *scales;
  uint64_t begin, end;                    // values
  uint32_t kind;
  bool one_scale;
};

__device__ __forceinline__ Chunk chunk_of(const Table &t, uint32_t chunk) {
  uint32_t lo = 0, hi = t.tensors;        // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  Chunk c;
  const uint64_t packed = t.count[lo], count = packed & ((1ull << 56) - 1);
  c.kind = (uint32_t)(packed >> 56) & 15u;
  c.one_scale = (packed >> 60) & 1;
  c.data = t.data[lo];
  c.scales = t.scales[lo];
  const uint32_t values = t.chunk_bytes >> (c.kind == 0 ? 2 : c.kind == 1 ? 1 : 0);
  c.begin = (uint64_t)(chunk - t.first[lo]) * values;
  c.end = c.begin + values < count ? c.begin + values : count;
  return c;
}

__device__ __forceinline__ double square_add(double sum, float v) {
  const double d = (double)v;
  return __builtin_fma(d, d, sum);
}

// Sum of the squares of the 16 bytes of values from `at` on.
template <int KIND>
__device__ __forceinline__ double squares16(u32x4 v, float scale, double sum) {
  if constexpr (KIND == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = square_add(sum, __uint_as_float(v[i]));
  } else if constexpr (KIND == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = square_add(square_add(sum, bf16_lo(v[i])), bf16_hi(v[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 a = dec2<KIND - 2, false>(v[i]), b = dec2<KIND - 2, true>(v[i]);
      sum = square_add(square_add(sum, a.x * scale), a.y * scale);
      sum = square_add(square_add(sum, b.x * scale), b.y * scale);
    }
  }
  return sum;
}

template <int KIND>
__device__ __forceinline__ double squares1(const void *data, uint64_t i, float scale, double sum) {
  if constexpr (KIND == 0) return square_add(sum, static_cast<const float *>(data)[i]);
  if constexpr (KIND == 1) return square_add(sum, bf16_lo(static_cast<const uint16_t *>(data)[i]));
  return square_add(sum, dec2<KIND == 3 ? 1 : 0, false>(static_cast<const uint8_t *>(data)[i]).x * scale);
}

template <int KIND>
__device__ __forceinline__ double chunk_squares(const Chunk &c) {
  constexpr uint32_t kEach = 16 / value_bytes(KIND);      // values of a vector
  constexpr int kUnroll = 4;
  const uint8_t *data = static_cast<const uint8_t *>(c.data);
  double sum[2] = {0.0, 0.0};
  const uint64_t vectors = (c.end - c.begin) / kEach;     // the chunk begins at a whole one
  const auto scale_at = [&](uint64_t value) {
    if constexpr (KIND < 2) return 1.0f;
    return c.scales[c.one_scale ? 0 : value / kBlock];
  };
  for (uint64_t v0 = threadIdx.x; v0 < vectors; v0 += kUnroll * kThreads) {
    u32x4 v[kUnroll];
    float s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint64_t i = v0 + (uint64_t)u * kThreads;
      v[u] = u32x4{0u, 0u, 0u, 0u};
      s[u] = 0.0f;
      if (i < vectors) {
        v[u] = load16<true>(data + (c.begin + i * kEach) * value_bytes(KIND));
        s[u] = scale_at(c.begin + i * kEach);
      }
    }
    loads_issued();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) sum[u & 1] = squares16<KIND>(v[u], s[u], sum[u & 1]);
  }
  const uint64_t i = c.begin + vectors * kEach + threadIdx.x;
  if (i < c.end) sum[0] = squares1<KIND>(c.data, i, scale_at(i), sum[0]);
  return sum[0] + sum[1];
}

// Sum over the workgroup, on thread 0.
template <int W>
__device__ __forceinline__ double sum_workgroup(double v, double *lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  if (lane_id() == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  double all = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < W; ++w) all += lds[w];
  return all;
}

__global__ __launch_bounds__(kThreads) void sumsq_kernel(const Table t, uint32_t chunks, double *out) {
  __shared__ double lds[kGradWaves];
  double sum = 0.0;
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Chunk c = chunk_of(t, i);
    switch (c.kind) {
      case 0: sum += chunk_squares<0>(c); break;
      case 1: sum += chunk_squares<1>(c); break;
      case 2: sum += chunk_squares<2>(c); break;
      default: sum += chunk_squares<3>(c); break;
    }
  }
  sum = sum_workgroup<kGradWaves>(sum, lds);
  if (threadIdx.x == 0) out[blockIdx.x] = sum;
}

constexpr int kLastWaves = 16;
__global__ __launch_bounds__(64 * kLastWaves) void sumsq_last_kernel(const double *parts, uint64_t n, double *out) {
  __shared__ double lds[kLastWaves];
  double sum = 0.0;
#pragma unroll 4
  for (uint64_t i = threadIdx.x; i < n; i += 64 * kLastWaves) sum += parts[i];
  sum = sum_workgroup<kLastWaves>(sum, lds);
  if (threadIdx.x == 0) *out = sum;
}

template <int KIND>
__device__ __forceinline__ u32x4 scaled16(u32x4 v, float c) {
  if constexpr (KIND == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * c);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = round2_bf16(bf16_lo(v[i]) * c, bf16_hi(v[i]) * c);
  }
  return v;
}

template <int KIND>
__device__ __forceinline__ void scale_chunk(const Chunk &c, float by) {
  constexpr uint32_t kEach = 16 / value_bytes(KIND);
  constexpr int kUnroll = 4;
  uint8_t *data = static_cast<uint8_t *>(const_cast<void *>(c.data));
  const uint64_t vectors = (c.end - c.begin) / kEach;
  for (uint64_t v0 = threadIdx.x; v0 < vectors; v0 += kUnroll * kThreads) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint64_t i = v0 + (uint64_t)u * kThreads;
      if (i < vectors) v[u] = load16<true>(data + (c.begin + i * kEach) * value_bytes(KIND));
    }
    loads_issued();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint64_t i = v0 + (uint64_t)u * kThreads;
      if (i < vectors) store16<true>(data + (c.begin + i * kEach) * value_bytes(KIND), scaled16<KIND>(v[u], by));
    }
  }
  const uint64_t i = c.begin + vectors * kEach + threadIdx.x;
  if (i < c.end) {
    if constexpr (KIND == 0) {
      float *p = reinterpret_cast<float *>(data) + i;
      *p = *p * by;
    } else {
      uint16_t *p = reinterpret_cast<uint16_t *>(data) + i;
      *p = (uint16_t)round2_bf16(bf16_lo(*p) * by, 0.0f);
    }
  }
}

__global__ __launch_bounds__(kThreads) void clip_kernel(const Table t, uint32_t chunks, const double *sumsq,
                                                        double max_norm, double eps, float *norm_out) {
  const double norm = __builtin_sqrt(*sumsq);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  if (max_norm == (double)INFINITY) return;
  const double share = max_norm / (norm + eps);
  if (share >= 1.0) return;                               // not for NaN
  const float by = (float)share;
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Chunk c = chunk_of(t, i);
    if (c.kind == 0)
      scale_chunk<0>(c, by);
    else
      scale_chunk<1>(c, by);
  }
}

// Bytes of a chunk: small ones give small lists the whole chip, and large ones
// large lists few lookups.
uint32_t chunk_bytes(uint64_t bytes) { return bytes <= (8u << 20) ? 4096 : bytes <= (256u << 20) ? 16384 : 65536; }

uint64_t total_bytes(const Grad *grads, uint64_t n) {
  uint64_t bytes = 0;
  for (uint64_t i = 0; i < n; ++i) bytes += grads[i].count * value_bytes(grads[i].kind);
  return bytes;
}

constexpr uint32_t kMostWorkgroups = 2048;                // eight a CU

// Runs each(table, chunks, workgroups) over the list, kTensors tensors and at
// most 2^31 chunks at a time (a tensor has far fewer).
template <typename Each>
void each_table(const Grad *grads, uint64_t n, Each &&each) {
  constexpr uint64_t kMostChunks = 1ull << 31;
  Table t;
  t.tensors = 0;
  t.first[0] = 0;
  t.chunk_bytes = chunk_bytes(total_bytes(grads, n));
  const auto flush = [&] {
    const uint32_t chunks = t.first[t.tensors];
    if (chunks) each(t, chunks, chunks < kMostWorkgroups ? chunks : kMostWorkgroups);
    t.tensors = 0;
  };
  for (uint64_t i = 0; i < n; ++i) {
    const Grad &g = grads[i];
    if (!g.count) continue;
    const uint64_t values = t.chunk_bytes / value_bytes(g.kind), chunks = (g.count + values - 1) / values;
    if (t.tensors == kTensors || t.first[t.tensors] + chunks > kMostChunks) flush();
    t.data[t.tensors] = g.data;
    t.scales[t.tensors] = g.scales;
    t.count[t.tensors] = g.count | (uint64_t)g.kind << 56 | (g.one_scale ? 1ull << 60 : 0);
    t.first[t.tensors + 1] = t.first[t.tensors] + (uint32_t)chunks;
    ++t.tensors;
  }
  flush();
}

}  // namespace

uint64_t grad_sumsq_workspace(const Grad *grads, uint64_t n) {
  uint64_t parts = 0;
  each_table(grads, n, [&](const Table &, uint32_t, uint32_t workgroups) { parts += workgroups; });
  return parts > 1 ? 8 * parts : 0;
}

hipError_t launch_grad_sumsq(const Grad *grads, uint64_t n, double *sumsq, double *workspace, hipStream_t stream) {
  const uint64_t parts = grad_sumsq_workspace(grads, n) / 8;
  uint64_t done = 0;
  bool any = false;
  hipError_t e = hipSuccess;
  each_table(grads, n, [&](const Table &t, uint32_t chunks, uint32_t workgroups) {
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(sumsq_kernel, dim3(workgroups), dim3(kThreads), 0, stream, t, chunks,
                       parts ? workspace + done : sumsq);
    done += workgroups;
    any = true;
    e = hipGetLastError();
  });
  if (e != hipSuccess || (any && !parts)) return e;
  hipLaunchKernelGGL(sumsq_last_kernel, dim3(1), dim3(64 * kLastWaves), 0, stream, workspace, parts, sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const Grad *grads, uint64_t n, const double *sumsq, double max_norm, double eps,
                            float *norm, hipStream_t stream) {
  hipError_t e = hipSuccess;
  bool any = false;
  const auto launch = [&](const Table &t, uint32_t chunks, uint32_t workgroups) {
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(clip_kernel, dim3(workgroups), dim3(kThreads), 0, stream, t, chunks, sumsq, max_norm, eps,
                       any ? nullptr : norm);
    any = true;
    e = hipGetLastError();
  };
  each_table(grads, n, launch);
  if (!any) {
    Table none;
    none.tensors = 0;
    none.first[0] = 0;
    none.chunk_bytes = 4096;
    launch(none, 0, 1);
  }
  return e;
}

}  // namespace fp8q
