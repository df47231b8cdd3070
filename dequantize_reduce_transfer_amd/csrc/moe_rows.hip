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
// A token's slots (and weights) are one load, lane j holding slot j; the ones
// that lead to a row are then broadcast to scalar registers, so that a row's
// base is scalar.  Rows are taken up to eight at a time, all their loads issued
// before the first is used and without a branch between them: where fewer are
// left the last one's is repeated (from the caches) and dropped.  A slot
// outside [0, row count) is skipped, so no value in `slots` can lead outside
// the buffers.
//
// Measured on MI355X at 16384 tokens, topk 8, hidden 2048 (median, rotating
// inputs): permute of E4M3 rows with scales 52 us, 6.0 TB/s; combine of bf16
// rows 102 us, 5.9 TB/s, of E4M3 rows 55 us, 6.3 TB/s; combine's backward 207
// us, 5.5 TB/s (a plain copy reaches 6.2-6.5, one stream read and eight written
// 5.2).  What the choices are worth there: the four waves of a workgroup side
// by side on one token's columns, so that whole 4 KiB rows move at once, 102 us
// against 136 with a wave a token; a wave's eight rows in flight together 105
// against 123 us one after another; non-temporal row loads 105 against 112 us;
// the permute's token rows loaded through the caches 10% over non-temporal (the
// waves with the other places read them too).  Fewer rows in flight, other runs
// of workgroups an XCD (8 to 256) and fewer resident workgroups all measured
// within 1% or slower: what is left is scattered rows' share of HBM's rate.
#include <type_traits>

#include "fp8q_device.h"
#include "layer_device.h"
#include "layer_launch.h"

namespace fp8q {
namespace {

constexpr int kWaves = 4;                      // waves a workgroup
constexpr uint32_t kColumns = 8 * kWave;       // columns a wave covers with one vector a lane
constexpr uint32_t kBackwardChoices = 8;       // choices a workgroup of the backward pass takes

__device__ __forceinline__ uint32_t broadcast(uint32_t v, uint32_t from) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, (int)from);
}

// The token's slots, one a lane; a slot that leads to no row is negative.
__device__ __forceinline__ int load_slots(const int *slots, uint64_t token, uint32_t topk,
                                          uint64_t row_count) {
  const uint32_t lane = lane_id();
  if (lane >= topk) return -1;
  const int s = slots[token * topk + lane];
  return s >= 0 && (uint64_t)s < row_count ? s : -1;
}

// The next G of the choices in `held` (bit j: choice j has a row), ascending;
// fewer than G are filled up with the last one.  `held` is not 0.
template <int G>
struct Choices {
  uint32_t lane[G];            // the choice: the lane that holds its slot and weight
  bool real[G];                // not a repetition
  __device__ __forceinline__ uint64_t take(uint64_t held) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      real[j] = held != 0;
      lane[j] = held ? (uint32_t)__builtin_ctzll(held) : lane[j ? j - 1 : 0];
      held &= held - 1;        // 0 stays 0
    }
    return held;
  }
};

// ---------------------------------------------------------------------------
// permute
// ---------------------------------------------------------------------------

// 16 bytes of the vector `i` of a row of `bytes` (at least 16): where the row
// ends inside it, the row's last 16, so that two lanes may hold (and write)
// the same bytes twice.
__device__ __forceinline__ uint32_t vector_at(uint32_t i, uint32_t bytes) {
  return 16u * i + 16u <= bytes ? 16u * i : bytes - 16u;
}

// Bytes [first, first + 1 KiB) of a row to every place.
__device__ __forceinline__ void copy_run(const uint8_t *src, uint8_t *dst, uint32_t bytes,
                                         uint32_t first, int slots, uint32_t topk) {
  const uint32_t lane = lane_id();
  if (bytes < 16) {                                      // fewer bytes than lanes: one each
    const uint8_t v = lane < bytes ? src[lane] : 0;
    for (uint32_t j = 0; j < topk; ++j) {
      const int slot = (int)broadcast((uint32_t)slots, j);
      if (slot >= 0 && lane < bytes) dst[(uint64_t)slot * bytes + lane] = v;
    }
    return;
  }
  const uint32_t i = first / 16 + lane;
  const bool in = 16 * i < bytes;
  const uint32_t at = vector_at(in ? i : 0, bytes);
  const u32x4 v = load16<false>(src + at);
  for (uint32_t j = 0; j < topk; ++j) {
    const int slot = (int)broadcast((uint32_t)slots, j);
    if (slot >= 0 && in) store16<true>(dst + (uint64_t)slot * bytes + at, v);
  }
}

// One wave a token, U KiB of its row (blockIdx.y) and `per` of its places
// (`groups` waves side by side, so that what they all read comes from the
// caches); the waves that have the row's start have its scales too.
template <int U>
__global__ __launch_bounds__(64 * kWaves) void permute_kernel(MoePermute a, uint32_t per, uint32_t groups) {
  const uint32_t unit = blockIdx.x * kWaves + uniform(threadIdx.x / kWave);
  const uint32_t group = unit % groups;
  const uint64_t t = unit / groups;
  if (t >= a.tokens) return;
  const uint32_t lane = lane_id(), bytes = (uint32_t)a.row_bytes, sbytes = (uint32_t)a.scale_row_bytes;
  const uint32_t first = blockIdx.y * (1024 * U);
  const uint8_t *src = static_cast<const uint8_t *>(a.src) + t * bytes;
  const uint8_t *ssrc = static_cast<const uint8_t *>(a.src_scales) + t * sbytes;
  uint8_t *dst = static_cast<uint8_t *>(a.dst), *sdst = static_cast<uint8_t *>(a.dst_scales);
  const int slots = load_slots(a.slots, t, a.topk, a.dst_rows);
  const bool lead = blockIdx.y == 0 && group == 0;
  if (bytes < 16) {
    if (lead) copy_run(src, dst, bytes, 0, slots, a.topk);
  } else {
    const bool scales = sbytes >= 16 && sbytes <= 1024 && blockIdx.y == 0;
    u32x4 v[U], s = {0u, 0u, 0u, 0u};
    uint32_t at[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = first / 16 + u * kWave + lane;
      in[u] = 16 * i < bytes;
      at[u] = vector_at(in[u] ? i : 0, bytes);
      v[u] = load16<false>(src + at[u]);
    }
    const bool sin = scales && 16 * lane < sbytes;
    const uint32_t sat = sin ? vector_at(lane, sbytes) : 0;
    if (sin) s = load16<false>(ssrc + sat);
    loads_issued();
    const uint32_t j0 = group * per, left = a.topk - j0, j1 = j0 + (left < per ? left : per);
    for (uint32_t j = j0; j < j1; ++j) {
      const int slot = (int)broadcast((uint32_t)slots, j);
      if (slot < 0) continue;
      uint8_t *d = dst + (uint64_t)slot * bytes, *sd = sdst + (uint64_t)slot * sbytes;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (in[u]) store16<true>(d + at[u], v[u]);
      if (sin) store16<true>(sd + sat, s);
    }
  }
  if (lead && sbytes && (bytes < 16 || sbytes < 16 || sbytes > 1024))
    for (uint32_t b = 0; b < sbytes; b += 1024) copy_run(ssrc, sdst, sbytes, b, slots, a.topk);
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------

constexpr int kBf16 = 0, kE4m3 = 1, kE5m2 = 2, kMx8 = 3;   // fp8q_row_format

// Eight columns of an expert row in a lane, as they are in memory.
template <int FMT, Edge EDGE>
struct RowPiece {
  u32x4 v;
  uint32_t scale;
  __device__ __forceinline__ void load(const MoeCombine &a, uint32_t slot, uint32_t e, uint32_t hidden) {
    const uint64_t base = (uint64_t)slot * hidden;
    if constexpr (FMT == kBf16) {
      v = load8_bf16<EDGE, true>(static_cast<const uint16_t *>(a.rows) + base, e, hidden);
    } else {
      const u32x2 q = load8_codes<EDGE, true>(static_cast<const uint8_t *>(a.rows) + base, e, hidden);
      v = u32x4{q.x, q.y, 0u, 0u};
      const uint32_t c = e < hidden ? e : 0u;
      if constexpr (FMT == kMx8) {
        const uint8_t *s = static_cast<const uint8_t *>(a.scales) + (uint64_t)slot * (hidden / kMxBlock);
        scale = s[c / kMxBlock];
      } else {
        const uint32_t *s = static_cast<const uint32_t *>(a.scales) +
                            (uint64_t)slot * ((hidden + kBlock - 1) / kBlock);
        scale = s[c / kBlock];
      }
    }
  }
  __device__ __forceinline__ void clear() {
    v = u32x4{0u, 0u, 0u, 0u};
    scale = 0;
  }
  __device__ __forceinline__ void values(uint32_t e, uint32_t hidden, float (&f)[8]) const {
    if constexpr (FMT == kBf16) {
      widen8(take8_bf16<EDGE>(v, e, hidden), f);
    } else {
      const u32x2 q = take8_codes<EDGE>(u32x2{v.x, v.y}, e, hidden);
      f32x2 d[4];
      if constexpr (FMT == kMx8) {
        d[0] = mx_dec2<false>(q.x, scale), d[1] = mx_dec2<true>(q.x, scale);
        d[2] = mx_dec2<false>(q.y, scale), d[3] = mx_dec2<true>(q.y, scale);
      } else {
        constexpr int F = FMT == kE4m3 ? 0 : 1;
        d[0] = dec2<F, false>(q.x), d[1] = dec2<F, true>(q.x);
        d[2] = dec2<F, false>(q.y), d[3] = dec2<F, true>(q.y);
      }
      const float s = FMT == kMx8 ? 1.0f : __uint_as_float(scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = FMT == kMx8 ? d[i / 2][i % 2] : d[i / 2][i % 2] * s;
    }
  }
};

// One wave a token and 512 columns, G of its rows at a time; a workgroup has
// W column pieces of 4 / W tokens.
template <int FMT, Edge EDGE, int G, int W>
__global__ __launch_bounds__(64 * kWaves) void combine_kernel(MoeCombine a) {
  const uint32_t wid = uniform(threadIdx.x / kWave);
  const uint64_t t = (uint64_t)block_position() * (kWaves / W) + wid / W;
  const uint32_t piece = blockIdx.y * W + wid % W, hidden = (uint32_t)a.hidden;
  if (t >= a.tokens || piece * kColumns >= hidden) return;
  const uint32_t lane = lane_id(), e = piece * kColumns + 8 * lane;
  const int slots = load_slots(a.slots, t, a.topk, a.row_count);
  const float weights = lane < a.topk && a.weights ? a.weights[t * a.topk + lane] : 1.0f;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (uint64_t held = __builtin_amdgcn_ballot_w64(slots >= 0); held;) {
    Choices<G> c;
    RowPiece<FMT, EDGE> row[G];
    held = c.take(held);
#pragma unroll
    for (int j = 0; j < G; ++j) row[j].load(a, broadcast((uint32_t)slots, c.lane[j]), e, hidden);
    loads_issued();
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float w = __uint_as_float(broadcast(__float_as_uint(weights), c.lane[j]));
      float f[8];
      if (!c.real[j]) row[j].clear();
      row[j].values(e, hidden, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(c.real[j] ? w : 0.0f, f[i], acc[i]);
    }
  }
  if (e < hidden) {
    if (a.out_bf16)
      store8_bf16<EDGE, false>(static_cast<uint16_t *>(a.out) + t * hidden, e, hidden, round8_bf16(acc));
    else
      store8_f32<EDGE, false>(static_cast<float *>(a.out) + t * hidden, e, hidden, acc);
  }
}

// W waves a token, each every W-th 512 columns; workgroups of 4 waves, and
// blockIdx.y names eight of the token's choices.  A row's products with dy are
// summed over the lanes, then over the waves.
template <Edge EDGE, int G, int W>
__global__ __launch_bounds__(64 * kWaves) void combine_backward_kernel(MoeCombineBackward a) {
  __shared__ float part[kWaves][kWave];
  const uint32_t wid = uniform(threadIdx.x / kWave), sub = wid % W;
  const uint64_t t0 = (uint64_t)block_position() * (kWaves / W) + wid / W;
  const bool live = t0 < a.tokens;                       // the same for the token's waves
  const uint64_t t = live ? t0 : 0;
  const uint32_t lane = lane_id(), hidden = (uint32_t)a.hidden;
  const uint16_t *dy = static_cast<const uint16_t *>(a.dy) + t * hidden;
  const int slots = live ? load_slots(a.slots, t, a.topk, a.row_count) : -1;
  const float weights = lane < a.topk ? a.weights[t * a.topk + lane] : 0.0f;
  float mine = 0.0f;                                     // lane j's is choice j's sum
  const bool ours = lane / kBackwardChoices == blockIdx.y;
  if (const uint64_t held = __builtin_amdgcn_ballot_w64(slots >= 0 && ours)) {
    Choices<G> c;
    c.take(held);
    float dot[G];
#pragma unroll
    for (int j = 0; j < G; ++j) dot[j] = 0.0f;
    for (uint32_t first = sub * kColumns; first < hidden; first += W * kColumns) {
      const uint32_t e = first + 8 * lane;
      u32x4 gv = load8_bf16<EDGE, false>(dy, e, hidden), rv[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const uint64_t base = (uint64_t)broadcast((uint32_t)slots, c.lane[j]) * hidden;
        rv[j] = load8_bf16<EDGE, true>(static_cast<const uint16_t *>(a.rows) + base, e, hidden);
      }
      loads_issued();
      float g[8];
      widen8(take8_bf16<EDGE>(gv, e, hidden), g);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float r[8], d[8];
        widen8(take8_bf16<EDGE>(rv[j], e, hidden), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(g[i], r[i], dot[j]);
        if (!c.real[j]) continue;
        const float w = __uint_as_float(broadcast(__float_as_uint(weights), c.lane[j]));
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = w * g[i];
        const uint64_t base = (uint64_t)broadcast((uint32_t)slots, c.lane[j]) * hidden;
        if (e < hidden)
          store8_bf16<EDGE, true>(static_cast<uint16_t *>(a.drows) + base, e, hidden, round8_bf16(d));
      }
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float sum = sum_wave(dot[j]);
      mine = c.lane[j] == lane ? sum : mine;
    }
  }
  if constexpr (W > 1) {
    part[wid][lane] = mine;
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int w = 1; w < W; ++w) mine += part[wid + w][lane];
  }
  if (live && ours && lane < a.topk) a.dweights[t * a.topk + lane] = mine;
}

// Waves that share a token by its 512-column pieces.
template <Edge EDGE, typename Launch>
void by_pieces(uint64_t hidden, Launch &&launch) {
  const uint64_t pieces = (hidden + kColumns - 1) / kColumns;
  if (EDGE == kTiny || pieces <= 1) return launch(std::integral_constant<int, 1>());
  if constexpr (EDGE != kTiny) {
    if (pieces == 2) return launch(std::integral_constant<int, 2>());
    launch(std::integral_constant<int, 4>());
  }
}

// Rows at a time: topk, up to eight.
template <typename Launch>
void by_choices(uint32_t topk, Launch &&launch) {
  if (topk <= 1)
    launch(std::integral_constant<int, 1>());
  else if (topk == 2)
    launch(std::integral_constant<int, 2>());
  else if (topk <= 4)
    launch(std::integral_constant<int, 4>());
  else
    launch(std::integral_constant<int, 8>());
}

template <typename Launch>
void by_edge(uint64_t hidden, Launch &&launch) {
  switch (edge_of(hidden)) {
    case kEven: return launch(std::integral_constant<Edge, kEven>());
    case kOdd: return launch(std::integral_constant<Edge, kOdd>());
    default: return launch(std::integral_constant<Edge, kTiny>());
  }
}

template <int FMT, Edge EDGE>
void combine_launch(const MoeCombine &a, hipStream_t stream) {
  by_choices(a.topk, [&](auto g) {
    by_pieces<EDGE>(a.hidden, [&](auto w) {
      constexpr int W = decltype(w)::value;
      const uint32_t pieces = (uint32_t)((a.hidden + kColumns - 1) / kColumns);
      const dim3 grid((a.tokens + kWaves / W - 1) / (kWaves / W), (pieces + W - 1) / W);
      hipLaunchKernelGGL((combine_kernel<FMT, EDGE, decltype(g)::value, W>), grid, dim3(64 * kWaves), 0,
                         stream, a);
    });
  });
}

template <int FMT>
void combine_rows(const MoeCombine &a, hipStream_t stream) {
  if constexpr (FMT == kMx8)                             // hidden % 32 == 0
    combine_launch<kMx8, kEven>(a, stream);
  else
    by_edge(a.hidden, [&](auto edge) { combine_launch<FMT, decltype(edge)::value>(a, stream); });
}

// Runs `launch` over the tokens in steps that keep a grid inside its limit.
template <typename Args, typename Step>
hipError_t over_tokens(Args a, uint32_t pieces, Step &&step) {
  const uint64_t fit = max_workgroups(kWaves) / pieces, most = fit < 1 ? 1 : fit;
  for (uint32_t left = a.tokens; left;) {
    const uint32_t n = left < most ? left : (uint32_t)most;
    a.tokens = n;
    step(a);
    left -= n;
    a.slots += (uint64_t)n * a.topk;
    a.advance(n);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_permute(const MoePermute &a, hipStream_t stream) {
  const uint32_t kib = (uint32_t)((a.row_bytes + 1023) / 1024);
  const uint32_t U = kib <= 1 ? 1 : kib <= 2 ? 2 : 4;
  // Places a wave writes to: one for rows of a KiB and more, so that as many
  // waves as places store at once (16384 tokens, topk 8: 2 KiB rows 52.3 us
  // against 56.2 with eight, 1 KiB rows 30.3 against 33.7); eight for shorter
  // rows, where waves would be many and small (512 bytes 19.6 against 25.5, 256
  // bytes 10.3 against 28.3), and for two choices (1 KiB rows 9.9 against 10.7).
  const uint32_t per = a.row_bytes >= 1024 && a.topk > 2 ? 1 : 8, groups = (a.topk + per - 1) / per;
  return over_tokens(a, (kib + U - 1) / U * groups, [&](const MoePermute &s) {
    const dim3 grid((s.tokens * groups + kWaves - 1) / kWaves, (kib + U - 1) / U), block(64 * kWaves);
    if (U == 1)
      hipLaunchKernelGGL((permute_kernel<1>), grid, block, 0, stream, s, per, groups);
    else if (U == 2)
      hipLaunchKernelGGL((permute_kernel<2>), grid, block, 0, stream, s, per, groups);
    else
      hipLaunchKernelGGL((permute_kernel<4>), grid, block, 0, stream, s, per, groups);
  });
}

hipError_t launch_moe_combine(int format, const MoeCombine &a, hipStream_t stream) {
  return over_tokens(a, (uint32_t)((a.hidden + kColumns - 1) / kColumns), [&](const MoeCombine &s) {
    switch (format) {
      case kBf16: combine_rows<kBf16>(s, stream); break;
      case kE4m3: combine_rows<kE4m3>(s, stream); break;
      case kE5m2: combine_rows<kE5m2>(s, stream); break;
      default: combine_rows<kMx8>(s, stream); break;
    }
  });
}

hipError_t launch_moe_combine_backward(const MoeCombineBackward &a, hipStream_t stream) {
  return over_tokens(a, 1, [&](const MoeCombineBackward &s) {
    by_edge(s.hidden, [&](auto edge) {
      by_choices(s.topk, [&](auto g) {
        by_pieces<decltype(edge)::value>(s.hidden, [&](auto w) {
          constexpr int W = decltype(w)::value;
          hipLaunchKernelGGL((combine_backward_kernel<decltype(edge)::value, decltype(g)::value, W>),
                             dim3((s.tokens + kWaves / W - 1) / (kWaves / W), (s.topk + kBackwardChoices - 1) / kBackwardChoices), dim3(64 * kWaves), 0,
                             stream, s);
        });
      });
    });
  });
}

}  // namespace fp8q
