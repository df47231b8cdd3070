// moe_sort.hip -- (token, choice) pairs sorted by expert, stable, on gfx950.
//
// A counting sort.  The pairs are cut into one run per workgroup and, inside
// it, one per wave, in order, so a pair's place is
//   pairs of lower experts
//   + pairs of its expert in earlier workgroups, earlier waves, and earlier
//     in its own wave's run,
// all of them counts, which integer atomics give in any order.  Up to
// kOneWorkgroup pairs one workgroup does it all in one launch; beyond that a
// first kernel writes each workgroup's counts to the workspace and a second
// one adds up those before its own.  The work is a few bytes a pair: launches
// and the serial chain inside a wave bound it, not HBM.
//
// Inside a wave, the lanes that hold the same expert are found with one
// ballot per bit of the expert's number; the count of such lanes below a lane
// is its rank, and the lowest of them moves the wave's counter on.
#include "fp8q_device.h"
#include "layer_launch.h"

namespace fp8q {
namespace {

constexpr int kSortWaves = 16;
constexpr uint32_t kSortThreads = 64 * kSortWaves;
constexpr uint32_t kMaxExperts = 1024;         // FP8Q_MAX_EXPERTS
constexpr uint32_t kOneWorkgroup = 16384;      // pairs up to which one workgroup sorts
constexpr uint32_t kChunkPairs = 4096;         // pairs a workgroup, at least
constexpr uint32_t kMaxChunks = 256;           // workgroups, at most

// Pairs a workgroup takes (a multiple of 64 * kSortWaves so that every wave's
// run is whole 64s).
uint32_t chunk_pairs(uint32_t pairs) {
  uint32_t per = (uint32_t)(((uint64_t)pairs + kMaxChunks - 1) / kMaxChunks);
  if (per < kChunkPairs) per = kChunkPairs;
  return (per + kSortThreads - 1) / kSortThreads * kSortThreads;
}

uint32_t chunks_for(uint32_t pairs) {
  if (pairs <= kOneWorkgroup) return 1;
  const uint32_t per = chunk_pairs(pairs);
  return (uint32_t)(((uint64_t)pairs + per - 1) / per);
}

template <typename Id>
__device__ __forceinline__ uint32_t expert_of(const Id *ids, uint32_t p, uint32_t experts) {
  const Id v = ids[p];
  return v >= 0 && v < (Id)experts ? (uint32_t)v : 0xFFFFFFFFu;
}

// counts[chunk][expert].
template <typename Id>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const Id *ids, uint32_t pairs,
                                                                  uint32_t experts, uint32_t per,
                                                                  uint32_t *counts) {
  __shared__ uint32_t hist[kMaxExperts];
  for (uint32_t e = threadIdx.x; e < experts; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const uint32_t first = blockIdx.x * per;
  const uint32_t left = pairs - first, n = left < per ? left : per;
  for (uint32_t i = threadIdx.x; i < n; i += kSortThreads) {
    const uint32_t e = expert_of(ids, first + i, experts);
    if (e != 0xFFFFFFFFu) atomicAdd(&hist[e], 1u);
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < experts; e += kSortThreads)
    counts[(uint64_t)blockIdx.x * experts + e] = hist[e];
}

// LDS: before[experts] (this expert's pairs in earlier workgroups, then its
// first place), total[experts], and place[waves][experts].
template <typename Id>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const Id *ids, uint32_t pairs,
                                                                  uint32_t experts, uint32_t bits,
                                                                  uint32_t per,
                                                                  const uint32_t *counts, int *slots,
                                                                  int *pairs_out, int *offsets) {
  __shared__ uint32_t lds[(2 + kSortWaves) * kMaxExperts];
  __shared__ uint32_t wave_sum[kSortWaves];
  uint32_t *before = lds, *total = lds + experts, *place = lds + 2 * experts;
  const uint32_t tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const uint32_t chunk = blockIdx.x, chunks = gridDim.x;
  const uint32_t first = chunk * per;
  const uint32_t left = pairs - first, n = left < per ? left : per;
  const uint32_t run = per / kSortWaves;                 // a wave's pairs, a multiple of 64
  const uint32_t w0 = wid * run < n ? wid * run : n;
  const uint32_t w1 = w0 + run < n ? w0 + run : n;

  for (uint32_t i = tid; i < (2 + kSortWaves) * experts; i += kSortThreads) lds[i] = 0;
  __syncthreads();
  // the wave's counts, and every workgroup's
  uint32_t *mine = place + wid * experts;
  for (uint32_t i = w0 + lane; i < w1; i += kWave) {
    const uint32_t e = expert_of(ids, first + i, experts);
    if (e != 0xFFFFFFFFu) atomicAdd(&mine[e], 1u);
  }
  if (counts) {
    const uint32_t cells = chunks * experts;
    for (uint32_t i = tid; i < cells; i += kSortThreads) {
      const uint32_t c = counts[i];
      if (c) {
        const uint32_t e = i % experts;
        atomicAdd(&total[e], c);
        if (i < chunk * experts) atomicAdd(&before[e], c);
      }
    }
  }
  __syncthreads();
  // one thread an expert: places inside the expert, then the experts' starts
  uint32_t sum = 0, at = 0;
  if (tid < experts) {
    if (!counts)
      for (int w = 0; w < kSortWaves; ++w) total[tid] += place[w * experts + tid];
    sum = total[tid];
  }
  uint32_t scan = sum;                                   // inclusive over the wave's experts
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)scan, d);
    if (lane >= (uint32_t)d) scan += o;
  }
  if (lane == kWave - 1) wave_sum[wid] = scan;
  __syncthreads();
  uint32_t all = 0;
  for (uint32_t w = 0; w < (uint32_t)kSortWaves; ++w) {
    if (w < wid) at += wave_sum[w];
    all += wave_sum[w];
  }
  if (tid < experts) {
    const uint32_t start = at + scan - sum;
    if (chunk == 0) offsets[tid] = (int)start;
    uint32_t next = start + before[tid];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = place[w * experts + tid];
      place[w * experts + tid] = next;
      next += c;
    }
  }
  if (chunk == 0 && tid == 0) offsets[experts] = (int)all;
  __syncthreads();
  // places, 64 pairs at a time
  for (uint32_t i0 = w0; i0 < w1; i0 += kWave) {
    const uint32_t i = i0 + lane;
    const uint32_t p = first + i;
    const uint32_t e = i < w1 ? expert_of(ids, p, experts) : 0xFFFFFFFFu;
    const bool held = e != 0xFFFFFFFFu;
    uint64_t same = __builtin_amdgcn_ballot_w64(held);
    for (uint32_t b = 0; b < bits; ++b) {
      const bool one = (e >> b) & 1u;
      const uint64_t m = __builtin_amdgcn_ballot_w64(one);
      same &= one ? m : ~m;
    }
    int slot = -1;
    uint32_t old = 0;
    const uint32_t rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32),
                                                    __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    const int leader = held ? (int)__builtin_ctzll(same) : 0;
    if (held && rank == 0) old = atomicAdd(&mine[e], (uint32_t)__builtin_popcountll(same));
    old = (uint32_t)__shfl((int)old, leader);
    if (held) {
      slot = (int)(old + rank);
      pairs_out[slot] = (int)p;
    }
    if (i < w1) {
      slots[p] = slot;
      if (p >= all) pairs_out[p] = -1;
    }
  }
}

template <typename Id>
hipError_t sort_launch(const MoeSort &a, hipStream_t stream) {
  const Id *ids = static_cast<const Id *>(a.ids);
  const uint32_t chunks = chunks_for(a.pairs);
  uint32_t bits = 0;
  while ((1u << bits) < a.experts) ++bits;
  uint32_t per = chunks == 1 ? (a.pairs + kSortThreads - 1) / kSortThreads * kSortThreads
                             : chunk_pairs(a.pairs);
  if (per == 0) per = kSortThreads;
  if (chunks > 1) {
    hipLaunchKernelGGL((sort_count_kernel<Id>), dim3(chunks), dim3(kSortThreads), 0,
                       stream, ids, a.pairs, a.experts, per, a.workspace);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((sort_place_kernel<Id>), dim3(chunks), dim3(kSortThreads), 0,
                     stream, ids, a.pairs, a.experts, bits, per,
                     chunks > 1 ? a.workspace : nullptr, a.slots, a.pairs_out, a.offsets);
  return hipGetLastError();
}

}  // namespace

uint64_t moe_sort_workspace(uint32_t pairs, uint32_t experts) {
  const uint32_t chunks = chunks_for(pairs);
  return chunks > 1 ? 4ull * chunks * experts : 0;
}

hipError_t launch_moe_sort(const MoeSort &a, hipStream_t stream) {
  return a.ids64 ? sort_launch<int64_t>(a, stream) : sort_launch<int32_t>(a, stream);
}

}  // namespace fp8q
