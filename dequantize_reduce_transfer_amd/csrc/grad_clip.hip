// grad_clip.hip -- the sum of squares over many gradient tensors, and their
// clipping in place, on gfx950.
//
// The tensors of a list are cut into chunks of equal bytes (the last of a
// tensor shorter), and workgroups walk over the chunks of a table of tensors,
// which travels as kernel arguments: a call needs no table in device memory, and
// a captured graph holds its own.  A chunk's tensor is found by bisection over
// the tensors' first chunks, which are scalar loads.
//
// Squares are exact in fp64 (of fp32 values; bf16's and the codes' fp32 ones
// as well), so nothing overflows or is lost that an fp32 sum would lose; the
// conversions and fp64 multiply-adds take less than the loads, and HBM bounds
// both operators.  A workgroup's sum goes to its own place in the workspace, and
// one more workgroup adds them up in order.
#include "fp8q_device.h"
#include "layer_device.h"
#include "model_launch.h"

namespace fp8q {
namespace {

constexpr int kGradWaves = 4;
constexpr uint32_t kThreads = 64 * kGradWaves;

// Tensors of a launch: as many as keep its arguments under 4 KiB (lists without
// codes need no scales; with 112 tensors a launch, 218 large ones took 2% more),
// or few, whose arguments cost less host time.
template <bool SCALED>
constexpr uint32_t kMany = SCALED ? 160 : 250;
constexpr uint32_t kFew = 32;

template <bool SCALED, uint32_t TENSORS>
struct Table {
  static constexpr uint32_t kTensors = TENSORS;
  uint64_t data[kTensors];                // the address; bits 56 .. 59 the kind, 60: one scale
  uint32_t first[kTensors + 1];           // first chunk
  uint32_t last[kTensors];                // values in the last chunk
  const float *scales[SCALED ? kTensors : 1];
  uint32_t tensors;
  uint32_t chunk_bytes;                   // a multiple of 512
};
static_assert(sizeof(Table<true, kMany<true>>) <= 4032 && sizeof(Table<false, kMany<false>>) <= 4032, "kernel arguments");

constexpr uint32_t value_bytes(int kind) { return kind == 0 ? 4 : kind == 1 ? 2 : 1; }

struct Chunk {
  const void *data;                       // the tensor's
  const float *scales;
  uint64_t begin, end;                    // values
  uint32_t kind;
  bool one_scale;
};

template <bool SCALED, uint32_t TENSORS>
__device__ __forceinline__ Chunk chunk_of(const Table<SCALED, TENSORS> &t, uint32_t chunk) {
  uint32_t lo = 0, hi = t.tensors;        // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  Chunk c;
  const uint64_t packed = t.data[lo];
  c.kind = (uint32_t)(packed >> 56) & 15u;
  c.one_scale = (packed >> 60) & 1;
  c.data = reinterpret_cast<const void *>(packed & ((1ull << 56) - 1));
  c.scales = t.scales[SCALED ? lo : 0];
  const uint32_t values = t.chunk_bytes >> (c.kind == 0 ? 2 : c.kind == 1 ? 1 : 0);
  c.begin = (uint64_t)(chunk - t.first[lo]) * values;
  c.end = c.begin + (chunk + 1 == t.first[lo + 1] ? t.last[lo] : values);
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

// Thread `tid` of THREADS' share of a chunk's sum.
template <int KIND, uint32_t THREADS>
__device__ __forceinline__ double chunk_squares(const Chunk &c, uint32_t tid) {
  constexpr uint32_t kEach = 16 / value_bytes(KIND);      // values of a vector
  constexpr int kUnroll = 8;
  const uint8_t *data = static_cast<const uint8_t *>(c.data);
  double sum[2] = {0.0, 0.0};
  const uint64_t vectors = (c.end - c.begin) / kEach;     // the chunk begins at a whole one
  const auto scale_at = [&](uint64_t value) {
    if constexpr (KIND < 2) return 1.0f;
    return c.scales[c.one_scale ? 0 : value / kBlock];
  };
  for (uint64_t v0 = tid; v0 < vectors; v0 += kUnroll * THREADS) {
    u32x4 v[kUnroll];
    float s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint64_t i = v0 + (uint64_t)u * THREADS;
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
  const uint64_t i = c.begin + vectors * kEach + tid;
  if (i < c.end) sum[0] = squares1<KIND>(c.data, i, scale_at(i), sum[0]);
  return sum[0] + sum[1];
}

template <uint32_t THREADS, bool SCALED, uint32_t TENSORS>
__device__ __forceinline__ double squares_of(const Table<SCALED, TENSORS> &t, uint32_t chunk, uint32_t tid) {
  const Chunk c = chunk_of(t, chunk);
  if (c.kind == 0) return chunk_squares<0, THREADS>(c, tid);
  if (!SCALED || c.kind == 1) return chunk_squares<1, THREADS>(c, tid);
  return c.kind == 2 ? chunk_squares<2, THREADS>(c, tid) : chunk_squares<3, THREADS>(c, tid);
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

template <bool SCALED>
__global__ __launch_bounds__(kThreads) void sumsq_kernel(const Table<SCALED, kMany<SCALED>> t, uint32_t chunks,
                                                         double *out) {
  __shared__ double lds[kGradWaves];
  double sum = 0.0;
  for (uint32_t i = block_position<16>(); i < chunks; i += gridDim.x) sum += squares_of<kThreads>(t, i, threadIdx.x);
  sum = sum_workgroup<kGradWaves>(sum, lds);
  if (threadIdx.x == 0) out[blockIdx.x] = sum;
}

constexpr int kLastWaves = 16;

// A small list by one workgroup, a wave a chunk.
template <bool SCALED>
__global__ __launch_bounds__(64 * kLastWaves) void sumsq_small_kernel(const Table<SCALED, kFew> t, uint32_t chunks,
                                                                      double *out) {
  __shared__ double lds[kLastWaves];
  double sum = 0.0;
  for (uint32_t i = uniform(threadIdx.x / kWave); i < chunks; i += kLastWaves)
    sum += squares_of<kWave>(t, i, lane_id());
  sum = sum_workgroup<kLastWaves>(sum, lds);
  if (threadIdx.x == 0) *out = sum;
}

__global__ __launch_bounds__(64 * kLastWaves) void sumsq_last_kernel(const double *parts, uint64_t n, double *out) {
  __shared__ double lds[kLastWaves];
  double sum = 0.0;
#pragma unroll 4
  for (uint64_t i = threadIdx.x; i < n; i += 64 * kLastWaves) sum += parts[i];
  sum = sum_workgroup<kLastWaves>(sum, lds);
  if (threadIdx.x == 0) *out = sum;
}

// Bytes of a chunk of the clipping: what its workgroup's threads load at once.
// One chunk a workgroup, and runs of them an XCD (block_position), took 757 us
// for 6.0e8 fp32 values (6.4 TB/s); chunks of 4 KiB 773, of 16 KiB 774, of 64
// KiB 850, 8 KiB with cached loads about a fifth more, and 2048 workgroups that
// walk over chunks of 64 KiB 921.
constexpr uint32_t kClipChunk = 8192;

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
  constexpr int kUnroll = kClipChunk / 16 / kThreads;
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

template <uint32_t TENSORS>
__global__ __launch_bounds__(kThreads) void clip_kernel(const Table<false, TENSORS> t, uint32_t chunks,
                                                        const double *sumsq, double max_norm, double eps,
                                                        float *norm_out) {
  const double norm = __builtin_sqrt(*sumsq);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  if (max_norm == (double)INFINITY) return;
  const double share = max_norm / (norm + eps);
  if (share >= 1.0) return;                               // not for NaN
  const float by = (float)share;
  for (uint32_t i = block_position<64>(); i < chunks; i += gridDim.x) {
    const Chunk c = chunk_of(t, i);
    if (c.kind == 0)
      scale_chunk<0>(c, by);
    else
      scale_chunk<1>(c, by);
  }
}

// Bytes of a chunk of the sum: small ones give small lists the whole chip, and
// large ones large lists few lookups (3.5e9 bf16 values: 64 KiB 1165 us, 32 KiB
// 1169, 16 KiB 1205).
uint32_t sum_chunk(const Grad *grads, uint64_t n) {
  uint64_t bytes = 0;
  for (uint64_t i = 0; i < n; ++i) bytes += grads[i].count * value_bytes(grads[i].kind);
  return bytes <= (8u << 20) ? 4096 : bytes <= (256u << 20) ? 16384 : 65536;
}

constexpr uint32_t kMostWorkgroups = 2048;                // of a sum: eight a CU
constexpr uint32_t kSmallChunks = 64;                     // chunks up to which one workgroup sums, a launch less

// Runs each(table, chunks) over the list, a table of tensors and at most 2^31
// chunks at a time (a tensor has far fewer).
template <bool SCALED, uint32_t TENSORS, typename Each>
void each_table(const Grad *grads, uint64_t n, uint32_t chunk, Each &&each) {
  constexpr uint64_t kMostChunks = 1ull << 31;
  Table<SCALED, TENSORS> t;
  t.tensors = 0;
  t.first[0] = 0;
  t.scales[0] = nullptr;
  t.chunk_bytes = chunk;
  const auto flush = [&] {
    if (t.tensors) each(t, t.first[t.tensors]);
    t.tensors = 0;
  };
  for (uint64_t i = 0; i < n; ++i) {
    const Grad &g = grads[i];
    if (!g.count) continue;
    const uint64_t values = chunk / value_bytes(g.kind), chunks = (g.count + values - 1) / values;
    if (t.tensors == t.kTensors || t.first[t.tensors] + chunks > kMostChunks) flush();
    t.data[t.tensors] = reinterpret_cast<uint64_t>(g.data) | (uint64_t)g.kind << 56 | (g.one_scale ? 1ull << 60 : 0);
    if (SCALED) t.scales[t.tensors] = g.scales;
    t.last[t.tensors] = (uint32_t)(g.count - (chunks - 1) * values);
    t.first[t.tensors + 1] = t.first[t.tensors] + (uint32_t)chunks;
    ++t.tensors;
  }
  flush();
}

bool any_codes(const Grad *grads, uint64_t n) {
  for (uint64_t i = 0; i < n; ++i)
    if (grads[i].count && grads[i].kind >= 2) return true;
  return false;
}

uint32_t workgroups_of(uint32_t chunks) { return chunks < kMostWorkgroups ? chunks : kMostWorkgroups; }

// A list that one workgroup sums.
bool small_sum(const Grad *grads, uint64_t n) {
  const uint32_t chunk = sum_chunk(grads, n);
  uint64_t chunks = 0, tensors = 0;
  for (uint64_t i = 0; i < n; ++i) {
    tensors += grads[i].count != 0;
    chunks += (grads[i].count * value_bytes(grads[i].kind) + chunk - 1) / chunk;
  }
  return tensors <= kFew && chunks <= kSmallChunks;
}

// Workgroups of a sum's launches: 0 where one workgroup does it all.
template <bool SCALED>
uint64_t sum_parts(const Grad *grads, uint64_t n) {
  uint64_t parts = 0;
  if (!small_sum(grads, n))
    each_table<SCALED, kMany<SCALED>>(grads, n, sum_chunk(grads, n),
                                      [&](const auto &, uint32_t chunks) { parts += workgroups_of(chunks); });
  return parts;
}

template <bool SCALED>
hipError_t sumsq_launch(const Grad *grads, uint64_t n, double *sumsq, double *workspace, hipStream_t stream) {
  hipError_t e = hipSuccess;
  uint64_t parts = 0;
  if (small_sum(grads, n)) {
    bool any = false;
    each_table<SCALED, kFew>(grads, n, sum_chunk(grads, n), [&](const auto &t, uint32_t chunks) {
      hipLaunchKernelGGL(sumsq_small_kernel<SCALED>, dim3(1), dim3(64 * kLastWaves), 0, stream, t, chunks, sumsq);
      any = true;
      e = hipGetLastError();
    });
    if (any) return e;
  } else {
    each_table<SCALED, kMany<SCALED>>(grads, n, sum_chunk(grads, n), [&](const auto &t, uint32_t chunks) {
      if (e != hipSuccess) return;
      hipLaunchKernelGGL(sumsq_kernel<SCALED>, dim3(workgroups_of(chunks)), dim3(kThreads), 0, stream, t, chunks,
                         workspace + parts);
      parts += workgroups_of(chunks);
      e = hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  // the parts' sum: 0 where the list holds nothing
  hipLaunchKernelGGL(sumsq_last_kernel, dim3(1), dim3(64 * kLastWaves), 0, stream, workspace, parts, sumsq);
  return hipGetLastError();
}

template <uint32_t TENSORS>
hipError_t clip_launch(const Grad *grads, uint64_t n, const double *sumsq, double max_norm, double eps, float *norm,
                       hipStream_t stream) {
  hipError_t e = hipSuccess;
  bool any = false;
  const auto launch = [&](const Table<false, TENSORS> &t, uint32_t chunks) {
    if (e != hipSuccess) return;
    const uint32_t most = (uint32_t)(FP8Q_MODEL_MAX_WAVES < kGradWaves ? 1 : FP8Q_MODEL_MAX_WAVES / kGradWaves);
    hipLaunchKernelGGL(clip_kernel<TENSORS>, dim3(chunks < 1 ? 1 : chunks < most ? chunks : most), dim3(kThreads), 0,
                       stream, t, chunks, sumsq, max_norm, eps, any ? nullptr : norm);
    any = true;
    e = hipGetLastError();
  };
  each_table<false, TENSORS>(grads, n, kClipChunk, launch);
  if (!any) {                                             // the norm all the same
    Table<false, TENSORS> none;
    none.tensors = 0;
    none.first[0] = 0;
    none.chunk_bytes = kClipChunk;
    launch(none, 0);
  }
  return e;
}

}  // namespace

uint64_t grad_sumsq_workspace(const Grad *grads, uint64_t n) {
  return 8 * (any_codes(grads, n) ? sum_parts<true>(grads, n) : sum_parts<false>(grads, n));
}

hipError_t launch_grad_sumsq(const Grad *grads, uint64_t n, double *sumsq, double *workspace, hipStream_t stream) {
  return any_codes(grads, n) ? sumsq_launch<true>(grads, n, sumsq, workspace, stream)
                             : sumsq_launch<false>(grads, n, sumsq, workspace, stream);
}

hipError_t launch_grad_clip(const Grad *grads, uint64_t n, const double *sumsq, double max_norm, double eps,
                            float *norm, hipStream_t stream) {
  return n <= kFew ? clip_launch<kFew>(grads, n, sumsq, max_norm, eps, norm, stream)
                   : clip_launch<kMany<false>>(grads, n, sumsq, max_norm, eps, norm, stream);
}

}  // namespace fp8q
