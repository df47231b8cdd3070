// moe_experts.hip -- a whole MoE layer for a few tokens, from weights in the
// codec's formats, on gfx950.
//
//   gate_up_kernel  h[p] = silu(gate_e x_t) * (up_e x_t) of every pair p
//   down_kernel     out_t = sum over the token's pairs of weight * (down_e h[p])
//
// Both read the rows of the experts that a token chose once, and little else:
// at 8 of 128 experts of 2048 x 768 a token's MXFP8 rows are 39 MB, so HBM
// bounds them for as long as an expert has few tokens.
//
// Products are 16x16x32 bf16 matrix instructions: the tokens' rows are operand
// A, 16 weight rows operand B, and both may take the k's of a chunk of 64 in
// any order, as long as it is the same.  Lane (r, q) = (lane % 16, lane / 16)
// holds k = 16 q .. 16 q + 15 of row r: one 16-byte load of codes, whose first
// and last eight are two instructions' operands.  A code becomes a bf16 exactly
// (E4M3 and E5M2 have at most 4 significant bits; times a power of two, MXFP8's
// scale, too).  An fp32 scale is not put into a bf16: it multiplies the chunk's
// fp32 sums, which it can because a lane's sums are all of weight row r.
#include "fp8q_device.h"
#include "layer_device.h"
#include "model_launch.h"

namespace fp8q {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum RowFormat : int { kBf16 = 0, kE4M3 = 1, kE5M2 = 2, kMx8 = 3 };   // fp8q_row_format

constexpr uint32_t kMaxExperts = 1024;   // FP8Q_MAX_EXPERTS
constexpr uint32_t kMaxPairs = 1024;     // FP8Q_EXPERTS_MAX_PAIRS
constexpr uint32_t kChunk = 64;          // k's of a chunk
constexpr int kGateUpWaves = 4;          // of a gate_up workgroup: they share the k's
constexpr int kDownWaves = 16;           // of a down workgroup: they share the experts

__device__ __forceinline__ int expert_of(const void *ids, bool ids64, uint32_t p, uint32_t experts) {
  const int64_t v = ids64 ? static_cast<const int64_t *>(ids)[p] : static_cast<const int *>(ids)[p];
  return v >= 0 && v < (int64_t)experts ? (int)v : -1;
}

// Sixteen elements of a weight row and what their scale is.
template <int F>
struct Piece {
  u32x4 v[F == kBf16 ? 2 : 1];
  uint32_t scale;                        // fp32 bits, or an E8M0 code
};

// A lane's piece of chunk c, all of it inside the row.  `row` is the lane's
// row, `scales` the row's scales.
template <int F>
__device__ __forceinline__ Piece<F> load_piece(const uint8_t *row, const uint8_t *scales, uint32_t c, uint32_t q) {
  Piece<F> p;
  const uint32_t kk = c * kChunk + q * 16u;
  if constexpr (F == kBf16) {
    p.v[0] = load16<false>(row + 2u * kk);
    p.v[1] = load16<false>(row + 2u * kk + 16u);
    p.scale = 0;
  } else {
    p.v[0] = load16<false>(row + kk);
    p.scale = F == kMx8 ? scales[kk / kMxBlock] : reinterpret_cast<const uint32_t *>(scales)[c / 2u];
  }
  return p;
}

// The same where the row ends inside the chunk: zeros past its end.
template <int F>
__device__ __forceinline__ Piece<F> load_last_piece(const uint8_t *row, const uint8_t *scales, uint32_t c,
                                                    uint32_t q, uint32_t k) {
  Piece<F> p;
  const uint32_t kk = c * kChunk + q * 16u;
  if constexpr (F == kBf16) {
#pragma unroll
    for (uint32_t j = 0; j < 16; ++j) {
      const bool in = kk + j < k;
      const uint32_t v = in ? reinterpret_cast<const uint16_t *>(row)[kk + j] : 0u;
      p.v[j / 8][j % 8 / 2] = j % 2 ? p.v[j / 8][j % 8 / 2] | v << 16 : v;
    }
    p.scale = 0;
  } else {
#pragma unroll
    for (uint32_t j = 0; j < 16; ++j) {
      const bool in = kk + j < k;
      const uint32_t v = in ? row[kk + j] : 0u;
      p.v[0][j / 4] = j % 4 ? p.v[0][j / 4] | v << (8 * (j % 4)) : v;
    }
    if constexpr (F == kMx8)
      p.scale = kk < k ? scales[kk / kMxBlock] : 127u;
    else
      p.scale = reinterpret_cast<const uint32_t *>(scales)[c / 2u];
  }
  return p;
}

// Eight codes as bf16 values, times 2^(e8m0 - 127) where they are MXFP8's.
template <int F>
__device__ __forceinline__ bf16x8 widen_codes(uint32_t lo, uint32_t hi, uint32_t scale) {
  bf16x2 a, b, c, d;
  if constexpr (F == kE5M2) {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
  } else {
    const float s = F == kMx8 ? __uint_as_float(scale << 23) : 1.0f;
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
  }
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

template <int F>
__device__ __forceinline__ bf16x8 half_of(const Piece<F> &p, int half) {
  if constexpr (F == kBf16) return __builtin_bit_cast(bf16x8, p.v[half]);
  return widen_codes<F>(p.v[0][2 * half], p.v[0][2 * half + 1], p.scale);
}

// A lane's sixteen elements of a token's row, two operands.
struct Token {
  u32x4 v[2];
};

// sums[i] += (token row 4 q + i) . (weight row r), over one chunk.
template <int F, int PARTS>
__device__ __forceinline__ void multiply(f32x4 &sums, const Token (&a)[PARTS], const Piece<F> &w) {
  const bf16x8 w0 = half_of<F>(w, 0), w1 = half_of<F>(w, 1);
  constexpr bool kScaled = F == kE4M3 || F == kE5M2;
  f32x4 d = kScaled ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sums;
#pragma unroll
  for (int i = PARTS - 1; i >= 0; --i) {        // the smallest parts first
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[i].v[0]), w0, d, 0, 0, 0);
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[i].v[1]), w1, d, 0, 0, 0);
  }
  if constexpr (kScaled) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[i] = __builtin_fmaf(__uint_as_float(w.scale), d[i], sums[i]);
  } else {
    sums = d;
  }
}

// What a wave multiplies: N matrices' rows (the lane's), and the rows of M x 16
// tokens (the lane's ones, `parts` apart).  `k` is the rows' length; `padded`:
// token rows are zero from k to the next multiple of 16.
template <int F, int N, int M, int PARTS, int UNROLL>
struct Dot {
  const uint8_t *row[N], *scales[N];
  const uint16_t *token[M];
  uint64_t parts;
  uint32_t k;

  __device__ __forceinline__ void load_token(Token (&t)[PARTS], int m, uint32_t c, uint32_t q) const {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const uint16_t *p = token[m] + i * parts + c * kChunk + q * 16u;
      t[i].v[0] = load16<false>(p);
      t[i].v[1] = load16<false>(p + 8);
    }
  }

  template <bool PADDED>
  __device__ __forceinline__ void load_last_token(Token (&t)[PARTS], int m, uint32_t c, uint32_t q) const {
    const uint32_t kk = c * kChunk + q * 16u;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const uint16_t *p = token[m] + i * parts;
      if constexpr (PADDED) {
        const u32x4 zero = {0u, 0u, 0u, 0u};
        t[i].v[0] = kk < k ? load16<false>(p + kk) : zero;
        t[i].v[1] = kk < k ? load16<false>(p + kk + 8) : zero;
      } else {
#pragma unroll
        for (uint32_t j = 0; j < 16; ++j) {
          const uint32_t v = kk + j < k ? p[kk + j] : 0u;
          t[i].v[j / 8][j % 8 / 2] = j % 2 ? t[i].v[j / 8][j % 8 / 2] | v << 16 : v;
        }
      }
    }
  }

  // sums += over chunks [c0, c1), the last of which may be the row's partial one.
  template <bool PADDED>
  __device__ __forceinline__ void run(f32x4 (&sums)[N][M], uint32_t c0, uint32_t c1, uint32_t q) const {
    const uint32_t full = k / kChunk < c1 ? k / kChunk : c1;
    for (uint32_t c = c0; c < full; c += UNROLL) {
      Piece<F> w[UNROLL][N];
      Token t[UNROLL][M][PARTS];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        if (c + u < full) {
#pragma unroll
          for (int n = 0; n < N; ++n) w[u][n] = load_piece<F>(row[n], scales[n], c + u, q);
#pragma unroll
          for (int m = 0; m < M; ++m) load_token(t[u][m], m, c + u, q);
        }
      }
      loads_issued();
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        if (c + u < full) {
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int n = 0; n < N; ++n) multiply<F, PARTS>(sums[n][m], t[u][m], w[u][n]);
        }
      }
    }
    if (full < c1 && c0 < c1) {
      Token t[PARTS];
      Piece<F> w[N];
#pragma unroll
      for (int n = 0; n < N; ++n) w[n] = load_last_piece<F>(row[n], scales[n], full, q, k);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        load_last_token<PADDED>(t, m, full, q);
#pragma unroll
        for (int n = 0; n < N; ++n) multiply<F, PARTS>(sums[n][m], t, w[n]);
      }
    }
  }
};

template <int F>
__host__ __device__ __forceinline__ uint64_t row_bytes(uint32_t k) {
  return F == kBf16 ? 2ull * k : k;
}
template <int F>
__host__ __device__ __forceinline__ uint64_t scale_bytes(uint32_t k) {
  return F == kBf16 ? 0 : F == kMx8 ? k / kMxBlock : 4ull * ((k + kBlock - 1) / kBlock);
}

// First chunk of part i of n: a multiple of two, so that the fp32 scales'
// blocks are whole.
__device__ __forceinline__ uint32_t part_start(uint32_t chunks, uint32_t i, uint32_t n) {
  return (chunks + 1u) / 2u * i / n * 2u;
}

struct GateUp {
  const uint16_t *x;
  const void *ids;
  bool ids64, by_pair;
  uint32_t pairs, topk, experts, hidden, inter, tiles;
  uint32_t padded;                       // inter, up to a multiple of 16
  int parts;                             // bf16 numbers that make an h: 2 or 3
  ExpertMatrix gate, up;
  uint16_t *h;                           // [parts][pairs][padded]
};

// h of up to 16 M pairs of one expert, for 16 of its rows.
template <int F, int M>
__device__ __forceinline__ void gate_up_tile(const GateUp &a, uint32_t e, uint32_t n0, const uint16_t *list,
                                             uint32_t count, float *sums_lds) {
  const uint32_t lane = lane_id(), r = lane % 16u, q = lane / 16u, wid = uniform(threadIdx.x / kWave);
  const uint32_t n = n0 + r < a.inter ? n0 + r : a.inter - 1;
  Dot<F, 2, M, 1, M == 1 ? 8 : M == 2 ? 4 : 2> dot;
  dot.k = a.hidden;
  dot.parts = 0;
  dot.row[0] = a.gate.rows + (a.gate.expert_rows * e + n) * row_bytes<F>(a.hidden);
  dot.row[1] = a.up.rows + (a.up.expert_rows * e + n) * row_bytes<F>(a.hidden);
  dot.scales[0] = a.gate.scales + (a.gate.expert_rows * e + n) * scale_bytes<F>(a.hidden);
  dot.scales[1] = a.up.scales + (a.up.expert_rows * e + n) * scale_bytes<F>(a.hidden);
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const uint32_t c = 16u * m + r < count ? 16u * m + r : count - 1;
    dot.token[m] = a.x + (uint64_t)(list[c] / a.topk) * a.hidden;
  }
  f32x4 sums[2][M];
#pragma unroll
  for (int m = 0; m < M; ++m) sums[0][m] = sums[1][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t chunks = (a.hidden + kChunk - 1) / kChunk;
  const uint32_t c1 = part_start(chunks, wid + 1, kGateUpWaves);
  dot.template run<false>(sums, part_start(chunks, wid, kGateUpWaves), c1 < chunks ? c1 : chunks, q);
  // [wave][gate, up][token 16 m + 4 q + i][row r]
  float *mine = sums_lds + wid * (2u * M * 256u);
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[(g * M + m) * 256 + (4 * q + i) * 16 + r] = sums[g][m][i];
  __syncthreads();
  for (uint32_t at = threadIdx.x; at < M * 256u; at += 64u * kGateUpWaves) {
    const uint32_t c = at / 16u, col = n0 + at % 16u;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kGateUpWaves; ++w) {
      g += sums_lds[w * (2u * M * 256u) + at];
      u += sums_lds[w * (2u * M * 256u) + M * 256u + at];
    }
    if (c >= count) continue;
    float h = g / (1.0f + expf(-g)) * u;
    if (col >= a.inter) h = 0.0f;        // the padding
    // h as a sum of bf16 numbers: its leading bits, and the rest's.  (An inf
    // or NaN has no rest.)
    uint16_t *to = a.h + (uint64_t)list[c] * a.padded + col;
    const uint64_t part = (uint64_t)a.pairs * a.padded;
    const uint32_t bits = __float_as_uint(h);
    const bool finite = (bits & 0x7F800000u) != 0x7F800000u;
    to[0] = (uint16_t)(h != h ? 0x7FC0u : bits >> 16);
    const float rest = finite ? h - __uint_as_float(bits & 0xFFFF0000u) : 0.0f;
    if (a.parts == 2) {
      to[part] = (uint16_t)round2_bf16(rest, 0.0f);
    } else {
      const uint32_t b = __float_as_uint(rest);
      to[part] = (uint16_t)(b >> 16);
      to[2 * part] = (uint16_t)round2_bf16(rest - __uint_as_float(b & 0xFFFF0000u), 0.0f);
    }
  }
}

template <int F>
__global__ __launch_bounds__(64 * kGateUpWaves) void gate_up_kernel(const GateUp a) {
  __shared__ uint16_t list[kMaxPairs];
  __shared__ float sums[kGateUpWaves * 2 * 4 * 256];
  const uint32_t lane = lane_id(), wid = uniform(threadIdx.x / kWave);
  const uint32_t which = blockIdx.x / a.tiles, n0 = blockIdx.x % a.tiles * 16u;
  // the expert: number `which`, or the one of pair `which` if no pair before it
  // has the same
  int e = (int)which;
  if (a.by_pair) {
    e = expert_of(a.ids, a.ids64, which, a.experts);
    if (e < 0) return;
  }
  uint32_t count = 0;
  for (uint32_t p0 = 0; p0 < a.pairs; p0 += kWave) {
    const uint32_t p = p0 + lane;
    const bool same = p < a.pairs && expert_of(a.ids, a.ids64, p, a.experts) == e;
    const uint64_t mask = __builtin_amdgcn_ballot_w64(same);
    if (a.by_pair && count == 0 && mask && p0 + (uint32_t)__builtin_ctzll(mask) != which) return;
    if (same && wid == 0)
      list[count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] =
          (uint16_t)p;
    count += (uint32_t)__builtin_popcountll(mask);
  }
  if (count == 0) return;
  __syncthreads();
  for (uint32_t m0 = 0; m0 < count; m0 += 64u) {
    const uint32_t left = count - m0;
    if (m0) __syncthreads();
    if (left <= 16u)
      gate_up_tile<F, 1>(a, (uint32_t)e, n0, list + m0, left, sums);
    else if (left <= 32u)
      gate_up_tile<F, 2>(a, (uint32_t)e, n0, list + m0, left, sums);
    else
      gate_up_tile<F, 4>(a, (uint32_t)e, n0, list + m0, left < 64u ? left : 64u, sums);
  }
}

struct Down {
  const uint16_t *h;
  const void *ids;
  const float *weights;
  bool ids64, out_bf16;
  uint32_t tokens, topk, experts, hidden, inter, padded;
  ExpertMatrix down;
  void *out;
};

// y of up to 16 M pairs of one expert, for 16 of its rows, over chunks [c0, c1).
template <int F, int M, int PARTS>
__device__ __forceinline__ void down_tile(const Down &a, uint32_t e, uint32_t n0, const uint16_t *list,
                                          uint32_t count, uint32_t c0, uint32_t c1, float *y) {
  const uint32_t lane = lane_id(), r = lane % 16u, q = lane / 16u;
  const uint32_t n = n0 + r < a.hidden ? n0 + r : a.hidden - 1;
  Dot<F, 1, M, PARTS, M == 1 ? 4 : 1> dot;
  dot.k = a.inter;
  dot.parts = (uint64_t)a.tokens * a.topk * a.padded;
  dot.row[0] = a.down.rows + (a.down.expert_rows * e + n) * row_bytes<F>(a.inter);
  dot.scales[0] = a.down.scales + (a.down.expert_rows * e + n) * scale_bytes<F>(a.inter);
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const uint32_t c = 16u * m + r < count ? 16u * m + r : count - 1;
    dot.token[m] = a.h + (uint64_t)list[c] * a.padded;
  }
  f32x4 sums[1][M];
#pragma unroll
  for (int m = 0; m < M; ++m) sums[0][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  dot.template run<true>(sums, c0, c1, q);
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = 16u * m + 4u * q + i;
      if (c < count) y[(uint32_t)list[c] * 16u + r] = sums[0][m][i];
    }
}

template <int F, int PARTS>
__global__ __launch_bounds__(64 * kDownWaves) void down_kernel(const Down a) {
  __shared__ float y[kMaxPairs * 16];              // [split][pair][row]
  __shared__ uint32_t counts[kMaxExperts], active[kMaxExperts], first[kMaxExperts];
  __shared__ uint16_t list[kMaxPairs];
  __shared__ uint32_t wave_sum[kDownWaves];
  const uint32_t tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const uint32_t pairs = a.tokens * a.topk, n0 = blockIdx.x * 16u;
  // the pairs by expert, and the experts that have some
  const int e = tid < pairs ? expert_of(a.ids, a.ids64, tid, a.experts) : -1;
  counts[tid] = 0;
  __syncthreads();
  uint32_t rank = 0;
  if (e >= 0) rank = atomicAdd(&counts[e], 1u);
  __syncthreads();
  const uint32_t mine = counts[tid], one = (mine ? 1u << 16 : 0u) + mine;   // both scans in one
  uint32_t scan = one;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)scan, d);
    if (lane >= (uint32_t)d) scan += o;
  }
  if (lane == kWave - 1) wave_sum[wid] = scan;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (uint32_t w = 0; w < (uint32_t)kDownWaves; ++w) {
    if (w < wid) before += wave_sum[w];
    all += wave_sum[w];
  }
  const uint32_t at = before + scan - one;
  if (mine) active[at >> 16] = tid;
  first[tid] = at & 0xFFFFu;
  __syncthreads();
  if (e >= 0) list[first[e] + rank] = (uint16_t)tid;
  __syncthreads();
  // where experts are fewer than waves, several waves share one's k's
  const uint32_t experts = all >> 16, chunks = (a.inter + kChunk - 1) / kChunk;
  uint32_t splits = 1;
  while (experts * splits * 2 <= (uint32_t)kDownWaves && pairs * splits * 2 <= kMaxPairs &&
         splits * 4 <= chunks)
    splits *= 2;
  for (uint32_t item = wid; item < experts * splits; item += kDownWaves) {
    const uint32_t x = uniform(active[item / splits]), s = item % splits;
    const uint32_t n = uniform(counts[x]), f = uniform(first[x]);
    const uint32_t c0 = part_start(chunks, s, splits), end = part_start(chunks, s + 1, splits);
    const uint32_t c1 = end < chunks ? end : chunks;
    float *to = y + s * pairs * 16u;
    for (uint32_t m0 = 0; m0 < n; m0 += 32u) {
      const uint32_t left = n - m0;
      if (left <= 16u)
        down_tile<F, 1, PARTS>(a, x, n0, list + f + m0, left, c0, c1, to);
      else
        down_tile<F, 2, PARTS>(a, x, n0, list + f + m0, left < 32u ? left : 32u, c0, c1, to);
    }
  }
  __syncthreads();
  for (uint32_t i = tid; i < a.tokens * 16u; i += 64u * kDownWaves) {
    const uint32_t t = i / 16u, r = i % 16u;
    if (n0 + r >= a.hidden) continue;
    float sum = 0.0f;
    for (uint32_t j = 0; j < a.topk; ++j) {
      const uint32_t p = t * a.topk + j;
      if (expert_of(a.ids, a.ids64, p, a.experts) < 0) continue;
      float v = 0.0f;
      for (uint32_t s = 0; s < splits; ++s) v += y[(s * pairs + p) * 16u + r];
      sum = __builtin_fmaf(a.weights[p], v, sum);
    }
    const uint64_t o = (uint64_t)t * a.hidden + n0 + r;
    if (a.out_bf16)
      static_cast<uint16_t *>(a.out)[o] = (uint16_t)round2_bf16(sum, 0.0f);
    else
      static_cast<float *>(a.out)[o] = sum;
  }
}

uint32_t padded(uint32_t inter) { return (inter + 15u) / 16u * 16u; }

template <int F>
hipError_t experts_launch(const MoeExperts &a, hipStream_t stream) {
  const uint32_t pairs = a.tokens * a.topk;
  if (a.inter) {
    const bool by_pair = pairs < a.experts;
    const uint32_t tiles = (a.inter + 15u) / 16u;
    const GateUp g{a.x, a.ids, a.ids64, by_pair, pairs, a.topk, a.experts, a.hidden, a.inter, tiles,
                   padded(a.inter), a.out_bf16 ? 2 : 3, a.gate, a.up, a.workspace};
    hipLaunchKernelGGL((gate_up_kernel<F>), dim3((by_pair ? pairs : a.experts) * tiles),
                       dim3(64 * kGateUpWaves), 0, stream, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const Down d{a.workspace, a.ids, a.weights, a.ids64, a.out_bf16, a.tokens, a.topk, a.inter ? a.experts : 0,
               a.hidden, a.inter, padded(a.inter), a.down, a.out};
  const dim3 grid((a.hidden + 15u) / 16u), block(64 * kDownWaves);
  if (a.out_bf16)
    hipLaunchKernelGGL((down_kernel<F, 2>), grid, block, 0, stream, d);
  else
    hipLaunchKernelGGL((down_kernel<F, 3>), grid, block, 0, stream, d);
  return hipGetLastError();
}

}  // namespace

uint64_t moe_experts_workspace(uint32_t pairs, uint32_t inter, bool out_bf16) {
  return 2ull * (out_bf16 ? 2 : 3) * pairs * padded(inter);
}

hipError_t launch_moe_experts(int format, const MoeExperts &a, hipStream_t stream) {
  switch (format) {
    case kBf16: return experts_launch<kBf16>(a, stream);
    case kE4M3: return experts_launch<kE4M3>(a, stream);
    case kE5M2: return experts_launch<kE5M2>(a, stream);
    default: return experts_launch<kMx8>(a, stream);
  }
}

}  // namespace fp8q
