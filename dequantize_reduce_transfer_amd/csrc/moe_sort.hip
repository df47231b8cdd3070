// moe_sort.hip -- (token, choice) pairs sorted by expert, stable, on gfx950.
//
// A counting sort.  The pairs are cut into one run per workgroup and, inside
// it, one per wave, in order, so a pair's place is
//   pairs of lower experts
//   + pairs of its expert in earlier workgroups, earlier waves, and earlier
//     in its own wave's run,
// all of them counts, which integer atomics in LDS give in any order.  Up to
// kOneWorkgroup pairs one workgroup does it all in one launch; beyond that a
// first kernel writes each workgroup's counts to the workspace and a second
// one adds up those before its own.
//
// Inside a wave, the lanes that hold the same expert are found with one
// ballot per bit of the expert's number; the count of such lanes below a lane
// is its rank, and the lowest of them moves the wave's counter on.
//
// The bytes are few (12 a pair, 1.6 MB at 16384 x 8: a quarter of a
// microsecond); launches and the serial chain (load, count, scan over the
// experts, place) bound it.  So a wave's run is short (64 pairs where the
// workgroups suffice), the next 64 ids are loaded ahead, and small sorts run
// in small workgroups, whose barriers and LDS to clear are fewer.
#include "fp8q_device.h"
#include "layer_launch.h"

namespace fp8q {
namespace {

constexpr uint32_t kMaxExperts = 1024;         // FP8Q_MAX_EXPERTS
constexpr uint32_t kNone = 0xFFFFFFFFu;
constexpr int kSortWaves = 16;                 // of the large workgroups
constexpr uint32_t kSortThreads = 64 * kSortWaves;
static_assert(kSortThreads >= kMaxExperts, "a thread an expert adds up the counts and writes them");
constexpr uint32_t kOneWorkgroup = 4096;       // pairs up to which one workgroup sorts

// Pairs a workgroup takes in a sort by two kernels.  Each workgroup adds up
// every workgroup's counts, so there are no more of them than keep the counts
// (workgroups x experts) at kMostCounts, and runs of two pairs a thread at
// least: at 131072 pairs and 128 experts on MI355X 64 workgroups take 10.3 us,
// 128 take 11.6 and 32 take 10.8-11.2; at 1048576 pairs 256 workgroups take 22,
// 64 take 27.
constexpr uint32_t kMostCounts = 32768, kChunkPairs = 2 * kSortThreads;
uint32_t chunk_pairs(uint32_t pairs, uint32_t experts) {
  uint32_t most = kMostCounts / experts;
  most = most < 16 ? 16 : most > 256 ? 256 : most;
  const uint32_t per = (uint32_t)(((uint64_t)pairs + most - 1) / most);
  return (per + kChunkPairs - 1) / kChunkPairs * kChunkPairs;
}

uint32_t chunks_for(uint32_t pairs, uint32_t experts) {
  if (pairs <= kOneWorkgroup) return 1;
  const uint32_t per = chunk_pairs(pairs, experts);
  return (uint32_t)(((uint64_t)pairs + per - 1) / per);
}

// The pair's expert, kNone where it has none (an id outside the experts, or
// no pair).
template <typename Id>
__device__ __forceinline__ uint32_t expert_of(const Id *ids, uint32_t p, bool exists, uint32_t experts) {
  if (!exists) return kNone;
  const Id v = ids[p];
  return v >= 0 && v < (Id)experts ? (uint32_t)v : kNone;
}

// counts[chunk][expert].
template <typename Id>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const Id *ids, uint32_t pairs,
                                                                  uint32_t experts, uint32_t per,
                                                                  uint32_t *counts) {
  __shared__ uint32_t hist[kMaxExperts];
  const uint32_t first = blockIdx.x * per;
  const uint32_t left = pairs - first, n = left < per ? left : per;
  uint32_t e = expert_of(ids, first + threadIdx.x, threadIdx.x < n, experts);
  if (threadIdx.x < experts) hist[threadIdx.x] = 0;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < n; i += kSortThreads) {
    const uint32_t next = expert_of(ids, first + i + kSortThreads, i + kSortThreads < n, experts);
    if (e != kNone) atomicAdd(&hist[e], 1u);
    e = next;
  }
  __syncthreads();
  if (threadIdx.x < experts) counts[(uint64_t)blockIdx.x * experts + threadIdx.x] = hist[threadIdx.x];
}

// The places of one workgroup's pairs.  `counts` is null where the workgroup
// has them all.  `lanes` is the power of two from `experts` up.
template <typename Id, int W>
__global__ __launch_bounds__(64 * W) void sort_place_kernel(const Id *ids, uint32_t pairs,
                                                            uint32_t experts, uint32_t lanes,
                                                            uint32_t per, const uint32_t *counts,
                                                            int *slots, int *pairs_out, int *offsets) {
  constexpr uint32_t kThreads = 64 * W;
  // place[w][e]: pairs of e in wave w's run, then the place of its next one;
  // before[e], total[e]: its pairs in earlier workgroups, and in all
  __shared__ uint32_t place[W * kMaxExperts];
  __shared__ uint32_t before[kMaxExperts], total[kMaxExperts];
  __shared__ uint32_t wave_sum[2][W];
  const uint32_t tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const uint32_t chunk = blockIdx.x, chunks = gridDim.x;
  const uint32_t first = chunk * per;
  const uint32_t left = pairs - first, n = left < per ? left : per;
  const uint32_t run = per / W;                          // a wave's pairs, a multiple of 64
  const uint32_t w0 = wid * run < n ? wid * run : n;
  const uint32_t w1 = w0 + run < n ? w0 + run : n;
  uint32_t *mine = place + wid * experts;

  const uint32_t e_first = expert_of(ids, first + w0 + lane, w0 + lane < w1, experts);
  for (uint32_t i = tid; i < W * experts; i += kThreads) place[i] = 0;
  for (uint32_t i = tid; i < experts; i += kThreads) before[i] = total[i] = 0;
  __syncthreads();
  uint32_t e = e_first;
  for (uint32_t i = w0 + lane; i < w1; i += kWave) {
    const uint32_t next = expert_of(ids, first + i + kWave, i + kWave < w1, experts);
    if (e != kNone) atomicAdd(&mine[e], 1u);
    e = next;
  }
  if (W == kSortWaves && counts) {                       // a thread adds up one expert's, every few workgroups'
    const uint32_t x = tid & (lanes - 1);
    if (x < experts) {
      uint32_t all = 0, early = 0;
#pragma unroll 8
      for (uint32_t c = tid / lanes; c < chunks; c += kThreads / lanes) {
        const uint32_t v = counts[(uint64_t)c * experts + x];
        all += v;
        early += c < chunk ? v : 0u;
      }
      atomicAdd(&total[x], all);
      atomicAdd(&before[x], early);
    }
  }
  __syncthreads();
  // the experts' first places, kThreads experts at a time
  uint32_t carry = 0;
  for (uint32_t e0 = 0, turn = 0; e0 < experts; e0 += kThreads, turn ^= 1) {
    const uint32_t x = e0 + tid;
    uint32_t sum = 0;
    if (x < experts) {
      sum = total[x];
      if (!counts)
        for (int w = 0; w < W; ++w) sum += place[w * experts + x];
    }
    uint32_t scan = sum;                                 // inclusive over the wave
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const uint32_t o = (uint32_t)__shfl_up((int)scan, d);
      if (lane >= (uint32_t)d) scan += o;
    }
    uint32_t at = carry;
    if constexpr (W > 1) {
      if (lane == kWave - 1) wave_sum[turn][wid] = scan;
      __syncthreads();
      for (uint32_t w = 0; w < (uint32_t)W; ++w) {
        if (w < wid) at += wave_sum[turn][w];
        carry += wave_sum[turn][w];
      }
    } else {
      carry += (uint32_t)__builtin_amdgcn_readlane((int)scan, kWave - 1);
    }
    if (x < experts) {
      const uint32_t start = at + scan - sum;
      if (chunk == 0) offsets[x] = (int)start;
      uint32_t next = start + before[x], c[W];
#pragma unroll
      for (int w = 0; w < W; ++w) c[w] = place[w * experts + x];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        place[w * experts + x] = next;
        next += c[w];
      }
    }
  }
  if (chunk == 0 && tid == 0) offsets[experts] = (int)carry;
  __syncthreads();
  // places, 64 pairs at a time
  e = e_first;
  for (uint32_t i0 = w0; i0 < w1; i0 += kWave) {
    const uint32_t i = i0 + lane, p = first + i;
    const uint32_t next = expert_of(ids, p + kWave, i + kWave < w1, experts);
    const bool held = e != kNone;
    uint64_t same = __builtin_amdgcn_ballot_w64(held);
    for (uint32_t b = 1; b < lanes; b <<= 1) {
      const bool one = (e & b) != 0;
      const uint64_t m = __builtin_amdgcn_ballot_w64(one);
      same &= one ? m : ~m;
    }
    const uint32_t rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32),
                                                    __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    uint32_t old = 0;
    if (held && rank == 0) old = atomicAdd(&mine[e], (uint32_t)__builtin_popcountll(same));
    old = (uint32_t)__shfl((int)old, held ? (int)__builtin_ctzll(same) : 0);
    int slot = -1;
    if (held) {
      slot = (int)(old + rank);
      pairs_out[slot] = (int)p;
    }
    if (i < w1) {
      slots[p] = slot;
      if (p >= carry) pairs_out[p] = -1;
    }
    e = next;
  }
}

template <typename Id, int W>
void place_launch(const MoeSort &a, uint32_t chunks, uint32_t per, hipStream_t stream) {
  uint32_t lanes = 1;
  while (lanes < a.experts) lanes <<= 1;
  hipLaunchKernelGGL((sort_place_kernel<Id, W>), dim3(chunks), dim3(64 * W), 0, stream,
                     static_cast<const Id *>(a.ids), a.pairs, a.experts, lanes, per,
                     chunks > 1 ? a.workspace : nullptr, a.slots, a.pairs_out, a.offsets);
}

// Waves of a lone workgroup: one for up to 64 pairs (a few tokens), four up to
// 512, sixteen beyond.  On MI355X, in a graph: 8 pairs 2.8 us with one wave,
// 3.6 with sixteen; 512 pairs 3.6 with four, 3.8 with sixteen; 2048 pairs 5.0
// with sixteen, 8.0 with four; 4096 pairs 7.0, which is what two kernels take
// as well.
template <typename Id>
hipError_t sort_launch(const MoeSort &a, hipStream_t stream) {
  const uint32_t chunks = chunks_for(a.pairs, a.experts);
  if (chunks > 1) {
    const uint32_t per = chunk_pairs(a.pairs, a.experts);
    hipLaunchKernelGGL((sort_count_kernel<Id>), dim3(chunks), dim3(kSortThreads), 0, stream,
                       static_cast<const Id *>(a.ids), a.pairs, a.experts, per, a.workspace);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    place_launch<Id, kSortWaves>(a, chunks, per, stream);
    return hipGetLastError();
  }
  const uint32_t groups = (a.pairs + 63) / 64 < 1 ? 1 : (a.pairs + 63) / 64;   // of 64 pairs
  if (groups <= 1)
    place_launch<Id, 1>(a, 1, 64 * groups, stream);
  else if (groups <= 8)
    place_launch<Id, 4>(a, 1, 64 * 4 * ((groups + 3) / 4), stream);
  else
    place_launch<Id, kSortWaves>(a, 1, kSortThreads * ((groups + kSortWaves - 1) / kSortWaves), stream);
  return hipGetLastError();
}

}  // namespace

uint64_t moe_sort_workspace(uint32_t pairs, uint32_t experts) {
  const uint32_t chunks = chunks_for(pairs, experts);
  return chunks > 1 ? 4ull * chunks * experts : 0;
}

hipError_t launch_moe_sort(const MoeSort &a, hipStream_t stream) {
  return a.ids64 ? sort_launch<int64_t>(a, stream) : sort_launch<int32_t>(a, stream);
}

}  // namespace fp8q
