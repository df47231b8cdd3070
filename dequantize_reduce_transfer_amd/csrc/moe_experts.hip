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
// holds k = 16 q .. 16 q + 15 of row r: 16 bytes of codes, whose first and last
// eight are two instructions' operands (of bf16 rows, 8 k's of 32: one).  A code
// becomes a bf16 exactly (E4M3 and E5M2 have at most 4 significant bits; times a
// power of two, MXFP8's scale, too).  An fp32 scale is not put into a bf16: it
// multiplies the chunk's fp32 sums, which it can because a lane's sums are all
// of weight row r.
#include "fp8q_device.h"
#include "layer_device.h"
#include "model_launch.h"

namespace fp8q {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum RowFormat : int { kBf16 = 0, kE4M3 = 1, kE5M2 = 2, kMx8 = 3 };   // fp8q_row_format

constexpr uint32_t kMaxPairs = 1024;     // FP8Q_EXPERTS_MAX_PAIRS
constexpr int kGateUpWaves = 4;          // of a gate_up workgroup: they share the k's
constexpr int kDownWaves = 8;            // of a down workgroup: they share the experts
constexpr int kRowsWaves = 4;            // of a down_rows workgroup: 16 rows each
constexpr uint32_t kFewPairs = 32;       // pairs up to which one kernel multiplies and adds up

__device__ __forceinline__ int expert_of(const void *ids, bool ids64, uint32_t p, uint32_t experts) {
  const int64_t v = ids64 ? static_cast<const int64_t *>(ids)[p] : static_cast<const int *>(ids)[p];
  return v >= 0 && v < (int64_t)experts ? (int)v : -1;
}

// A wave's tile of weights in LDS: R rows of 256 bytes, as 16-byte pieces, which
// are a lane's operands.  Lanes 0 .. 15 of a load take one row's pieces, so it
// reads whole lines; a matrix instruction's lane (r, q) wants piece 4 c + q of
// row r, which straight from memory would be 16 rows a load, 64 bytes of each: a
// quarter of the rate at which a CU's addresses are worked off.  Piece p of row
// v lies in place p ^ v, so that a read's rows fall into different banks.  Tiles
// of 8 rows give lanes 8 .. 15 of an operand the rows of lanes 0 .. 7 again.
constexpr uint32_t kRowBytes = 256;

typedef const void __attribute__((address_space(1))) *GlobalPtr;
typedef void __attribute__((address_space(3))) *LdsPtr;

// Everything the wave has issued is there.
__device__ __forceinline__ void all_loaded() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// The wave's LDS reads and writes are done.
__device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int F>
constexpr uint32_t kPiece = F == kBf16 ? 8 : 16;    // elements of a piece

template <int F>
__host__ __device__ __forceinline__ uint64_t row_bytes(uint32_t k) {
  return F == kBf16 ? 2ull * k : k;
}
template <int F>
__host__ __device__ __forceinline__ uint64_t scale_bytes(uint32_t k) {
  return F == kBf16 ? 0 : F == kMx8 ? k / kMxBlock : 4ull * ((k + kBlock - 1) / kBlock);
}

// The last bytes [at, at + 16) of a row that ends inside them, zeros behind.
__device__ __forceinline__ u32x4 load_row_end(const uint8_t *row, uint32_t at, uint32_t bytes) {
  if (bytes >= 16) return shift_down(load16<false>(row + bytes - 16), at + 16 - bytes, 8);
  u32x4 v = {0u, 0u, 0u, 0u};
  for (uint32_t j = 0; at + j < bytes; ++j) v[j / 4] |= (uint32_t)row[at + j] << (8 * (j % 4));
  return v;
}

// Loads the tile of rows [0, R) (those from `rows` on: the last row again) and
// bytes [at, at + 256) into LDS, all inside the rows; `width` bytes a row.
//   ALIGNED  rows and their length are multiples of 16 bytes: straight into LDS
template <int R, bool ALIGNED>
__device__ __forceinline__ void load_tile(uint8_t *tile, const uint8_t *base, uint32_t rows, uint32_t width,
                                          uint32_t at, uint32_t lane) {
  u32x4 v[ALIGNED ? 1 : R / 4];
#pragma unroll
  for (uint32_t i = 0; i < R / 4; ++i) {
    const uint32_t row = i * 4 + lane / 16u, p = (lane % 16u) ^ row;
    const uint32_t n = row < rows ? row : rows - 1;
    const uint8_t *from = base + (uint64_t)n * width + (at + p * 16u);
    if constexpr (ALIGNED)
      __builtin_amdgcn_global_load_lds((GlobalPtr)from, (LdsPtr)(tile + i * 1024), 16, 0, 0);
    else
      v[i] = load16<false>(from);
  }
  if constexpr (!ALIGNED) {
#pragma unroll
    for (uint32_t i = 0; i < R / 4; ++i) *reinterpret_cast<u32x4 *>(tile + i * 1024 + lane * 16u) = v[i];
  }
}

// The lane's piece of chunk c (four pieces a row).
template <int R>
__device__ __forceinline__ u32x4 read_piece(const uint8_t *tile, uint32_t c, uint32_t r, uint32_t q) {
  return *reinterpret_cast<const u32x4 *>(tile + (r % R) * kRowBytes + (((c * 4u + q) ^ (r % R)) * 16u));
}

// Eight codes as bf16 values, times 2^(e8m0 - 127) where they are MXFP8's.
template <int F>
__device__ __forceinline__ bf16x8 widen_codes(uint32_t lo, uint32_t hi, float scale) {
  bf16x2 a, b, c, d;
  if constexpr (F == kE5M2) {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
  } else {
    const float s = F == kMx8 ? scale : 1.0f;
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
  }
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Sixteen bytes of a token's row (eight k's): an operand.
__device__ __forceinline__ f32x4 matrix_step(u32x4 a, bf16x8 b, f32x4 d) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), b, d, 0, 0, 0);
}

// The scale's factor of the lane's 16 k's: an fp32, or E8M0's 2^(code - 127) in
// the exponent's place.
template <int F>
__device__ __forceinline__ float scale_of(uint32_t w) {
  return __uint_as_float(F == kMx8 ? (w & 0xFFu) << 23 : w);
}

// Scales of a lane's row over four chunks (256 k's): fp32 a block of 128, or
// E8M0 codes of four blocks of 32 a word.
template <int F>
struct Scales {
  uint32_t w[2];

  __device__ __forceinline__ void load(const uint8_t *row, uint32_t e) {
    if constexpr (F == kBf16) return;
    const u32x2 v = load8<false>(F == kMx8 ? row + e / kMxBlock : row + e / kBlock * 4u);
    w[0] = v.x;
    w[1] = v.y;
  }
  __device__ __forceinline__ float of(int c, uint32_t q) const {
    return scale_of<F>(F == kMx8 ? w[c / 2] >> (16 * (c % 2) + 8 * (q / 2u)) : w[c / 2]);
  }
};

// What a wave multiplies: N matrices' rows, and the rows of 16 tokens (the
// lane's one; `parts` elements from one part of a row to the next).
//   R       rows of a tile
//   TILES   tiles of each matrix that are loaded at once
//   PADDED  token rows are zeros from k to the next multiple of 16
template <int F, int N, int R, int TILES, int PARTS, bool PADDED, bool ALIGNED>
struct Dot {
  static constexpr int kVectors = F == kBf16 ? 1 : 2;    // operands of a piece
  static constexpr uint32_t kTile = 16 * kPiece<F>;      // elements of a tile's row
  static constexpr uint32_t kLds = N * TILES * R * kRowBytes;
  const uint8_t *rows[N];                                // the tile's first row (uniform)
  const uint8_t *row[N], *scales[N];                     // the lane's
  const uint16_t *token;
  uint64_t parts;
  uint32_t count;                                        // rows there are
  uint32_t k;
  uint8_t *lds;                                          // kLds bytes

  struct Operand {
    u32x4 v[PARTS][kVectors];
  };

  // sums += the chunk whose weights are w.
  __device__ __forceinline__ void multiply(f32x4 &sums, const Operand &t, u32x4 w, float scale) const {
    constexpr bool kScaled = F == kE4M3 || F == kE5M2;
    const bf16x8 b0 = F == kBf16 ? __builtin_bit_cast(bf16x8, w) : widen_codes<F>(w.x, w.y, scale);
    bf16x8 b1 = b0;
    if constexpr (F != kBf16) b1 = widen_codes<F>(w.z, w.w, scale);
    f32x4 d = kScaled ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sums;
#pragma unroll
    for (int i = PARTS - 1; i >= 0; --i) {               // the smallest parts first
      d = matrix_step(t.v[i][0], b0, d);
      if constexpr (kVectors == 2) d = matrix_step(t.v[i][kVectors - 1], b1, d);
    }
    if constexpr (kScaled) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[i] = __builtin_fmaf(scale, d[i], sums[i]);
    } else {
      sums = d;
    }
  }

  __device__ __forceinline__ void load_tokens(Operand (&t)[4], uint32_t e, uint32_t q) const {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int v = 0; v < kVectors; ++v)
          t[c].v[i][v] = load16<false>(token + i * parts + e + (c * 4u + q) * kPiece<F> + 8u * v);
  }

  // sums[n] += over W whole tiles' k's from element e on.
  template <int W>
  __device__ __forceinline__ void stage(f32x4 (&sums)[N], uint32_t e, uint32_t lane) const {
    const uint32_t r = lane % 16u, q = lane / 16u, width = (uint32_t)row_bytes<F>(k);
    Scales<F> s[N][W];
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        load_tile<R, ALIGNED>(lds + (w * N + n) * (R * kRowBytes), rows[n], count, width,
                              (uint32_t)row_bytes<F>(e + w * kTile), lane);
        s[n][w].load(scales[n], e + w * kTile);
      }
    // the tokens' rows, two tiles of them in registers
    Operand t[2][4];
    load_tokens(t[0], e, q);
    if constexpr (W > 1) load_tokens(t[1], e + kTile, q);
    loads_issued();
    all_loaded();
    if (!ALIGNED) lds_done();
#pragma unroll
    for (int w = 0; w < W; ++w) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int n = 0; n < N; ++n)
          multiply(sums[n], t[w % 2][c], read_piece<R>(lds + (w * N + n) * (R * kRowBytes), c, r, q), s[n][w].of(c, q));
        loads_issued();
      }
      if (w + 2 < W) load_tokens(t[w % 2], e + (w + 2) * kTile, q);
    }
    lds_done();                                          // before the next tiles overwrite these
  }

  // sums[n] += over the k's from element e on, fewer than a tile's.
  __device__ __forceinline__ void tail(f32x4 (&sums)[N], uint32_t e, uint32_t lane) const {
    const uint32_t q = lane / 16u, width = (uint32_t)row_bytes<F>(k);
#pragma unroll 1
    for (; e < k; e += 4 * kPiece<F>) {
      const uint32_t kk = e + q * kPiece<F>, b = (uint32_t)row_bytes<F>(kk);
      const u32x4 zero = {0u, 0u, 0u, 0u};
      Operand t;
#pragma unroll
      for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int v = 0; v < kVectors; ++v) {
          const uint16_t *p = token + i * parts;
          const uint32_t at = kk + 8u * v, end = PADDED ? (k + 15u) / 16u * 16u : k;
          t.v[i][v] = at + 8u <= end ? load16<false>(p + at)
                      : at < end     ? load_row_end(reinterpret_cast<const uint8_t *>(p), 2u * at, 2u * end)
                                     : zero;
        }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const u32x4 w = b + 16u <= width ? load16<false>(row[n] + b) : b < width ? load_row_end(row[n], b, width) : zero;
        uint32_t s = 0;
        if constexpr (F == kMx8)
          s = kk < k ? scales[n][kk / kMxBlock] : 127u;
        else if constexpr (F != kBf16)
          s = reinterpret_cast<const uint32_t *>(scales[n])[e / kBlock];
        multiply(sums[n], t, w, scale_of<F>(s));
      }
    }
  }

  // Tiles of a row's k's, the last one partial.
  static __host__ __device__ __forceinline__ uint32_t tiles(uint32_t k) { return (k + kTile - 1) / kTile; }

  // sums += over tiles [t0, t1).
  __device__ __forceinline__ void run(f32x4 (&sums)[N], uint32_t t0, uint32_t t1, uint32_t lane) const {
    const uint32_t whole = k / kTile < t1 ? k / kTile : t1;
    uint32_t i = t0;
    for (; i + TILES <= whole; i += TILES) stage<TILES>(sums, i * kTile, lane);
    if constexpr (TILES > 1)
      for (; i < whole; ++i) stage<1>(sums, i * kTile, lane);
    if (whole < t1 && t0 < t1) tail(sums, whole * kTile, lane);
  }
};

// The pairs of the workgroup's expert (number `which`, or by_pair the one of
// pair `which` if no pair before it has the same) into `list`, by wave 0; how
// many there are, 0 where there is nothing to do.
__device__ __forceinline__ uint32_t expert_pairs(const void *ids, bool ids64, bool by_pair, uint32_t pairs,
                                                 uint32_t experts, uint32_t which, uint16_t *list, int &e) {
  const uint32_t lane = lane_id(), wid = uniform(threadIdx.x / kWave);
  e = (int)which;
  if (by_pair) {
    e = expert_of(ids, ids64, which, experts);
    if (e < 0) return 0;
  }
  uint32_t count = 0;
  for (uint32_t p0 = 0; p0 < pairs; p0 += kWave) {
    const uint32_t p = p0 + lane;
    const bool same = p < pairs && expert_of(ids, ids64, p, experts) == e;
    const uint64_t mask = __builtin_amdgcn_ballot_w64(same);
    if (by_pair && count == 0 && mask && p0 + (uint32_t)__builtin_ctzll(mask) != which) return 0;
    if (same && wid == 0)
      list[count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] =
          (uint16_t)p;
    count += (uint32_t)__builtin_popcountll(mask);
  }
  __syncthreads();
  return count;
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

template <int F, bool ALIGNED>
using GateUpDot = Dot<F, 2, 16, 1, 1, false, ALIGNED>;

// h of up to 16 pairs of one expert, for 16 of its rows.
template <int F, bool ALIGNED>
__device__ __forceinline__ void gate_up_tile(const GateUp &a, uint32_t e, uint32_t n0, const uint16_t *list,
                                             uint32_t count, uint8_t *lds) {
  const uint32_t lane = lane_id(), r = lane % 16u, q = lane / 16u, wid = uniform(threadIdx.x / kWave);
  const uint32_t n = n0 + r < a.inter ? n0 + r : a.inter - 1;
  GateUpDot<F, ALIGNED> dot;
  dot.k = a.hidden;
  dot.parts = 0;
  dot.count = a.inter - n0;
  dot.lds = lds + wid * dot.kLds;
  dot.rows[0] = a.gate.rows + (a.gate.expert_rows * e + n0) * row_bytes<F>(a.hidden);
  dot.rows[1] = a.up.rows + (a.up.expert_rows * e + n0) * row_bytes<F>(a.hidden);
  dot.scales[0] = a.gate.scales + (a.gate.expert_rows * e + n) * scale_bytes<F>(a.hidden);
  dot.scales[1] = a.up.scales + (a.up.expert_rows * e + n) * scale_bytes<F>(a.hidden);
  dot.token = a.x + (uint64_t)(list[r < count ? r : count - 1] / a.topk) * a.hidden;
  dot.row[0] = dot.rows[0] + (n - n0) * row_bytes<F>(a.hidden);
  dot.row[1] = dot.rows[1] + (n - n0) * row_bytes<F>(a.hidden);
  f32x4 sums[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
  const uint32_t tiles = dot.tiles(a.hidden);
  dot.run(sums, tiles * wid / kGateUpWaves, tiles * (wid + 1) / kGateUpWaves, lane);
  __syncthreads();                       // the tiles' memory is the sums' now
  float *sums_lds = reinterpret_cast<float *>(lds);
  // [wave][gate, up][token 4 q + i][row r]
  float *mine = sums_lds + wid * 512u;
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[g * 256 + (4 * q + i) * 16 + r] = sums[g][i];
  __syncthreads();
  {
    const uint32_t at = threadIdx.x, c = at / 16u, col = n0 + at % 16u;
    if (c >= count) return;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kGateUpWaves; ++w) {
      g += sums_lds[w * 512u + at];
      u += sums_lds[w * 512u + 256u + at];
    }
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

template <int F, bool ALIGNED>
__global__ __launch_bounds__(64 * kGateUpWaves) void gate_up_kernel(const GateUp a) {
  __shared__ uint16_t list[kMaxPairs];
  __shared__ alignas(16) uint8_t lds[kGateUpWaves * GateUpDot<F, ALIGNED>::kLds];
  const uint32_t n0 = blockIdx.x % a.tiles * 16u;
  int e;
  const uint32_t count = expert_pairs(a.ids, a.ids64, a.by_pair, a.pairs, a.experts, blockIdx.x / a.tiles, list, e);
  if (count == 0) return;
  for (uint32_t m0 = 0; m0 < count; m0 += 16u) {
    if (m0) __syncthreads();
    gate_up_tile<F, ALIGNED>(a, (uint32_t)e, n0, list + m0, count - m0 < 16u ? count - m0 : 16u, lds);
  }
}

struct Down {
  const uint16_t *h;
  const void *ids;
  const float *weights;
  bool ids64, by_pair, out_bf16;
  uint32_t tokens, topk, experts, hidden, inter, padded, groups;
  ExpertMatrix down;
  float *y;                              // [pairs][hidden], of down_rows_kernel
  void *out;
};

template <int F, int R, int TILES, int PARTS, bool ALIGNED>
using DownDot = Dot<F, 1, R, TILES, PARTS, true, ALIGNED>;

// The product of up to 16 pairs of one expert with R of its rows, over tiles
// [t0, t1) of the k's.
template <int F, int R, int TILES, int PARTS, bool ALIGNED>
__device__ __forceinline__ f32x4 down_tile(const Down &a, uint32_t e, uint32_t n0, uint32_t pair, uint32_t t0,
                                           uint32_t t1, uint8_t *lds) {
  const uint32_t lane = lane_id(), r = lane % 16u;
  const uint32_t n = n0 + r % R < a.hidden ? n0 + r % R : a.hidden - 1;
  DownDot<F, R, TILES, PARTS, ALIGNED> dot;
  dot.k = a.inter;
  dot.parts = (uint64_t)a.tokens * a.topk * a.padded;
  dot.count = a.hidden - n0;
  dot.lds = lds;
  dot.rows[0] = a.down.rows + (a.down.expert_rows * e + n0) * row_bytes<F>(a.inter);
  dot.scales[0] = a.down.scales + (a.down.expert_rows * e + n) * scale_bytes<F>(a.inter);
  dot.token = a.h + (uint64_t)pair * a.padded;
  dot.row[0] = dot.rows[0] + (n - n0) * row_bytes<F>(a.inter);
  f32x4 sums[1] = {{0.0f, 0.0f, 0.0f, 0.0f}};
  dot.run(sums, t0, t1, lane);
  return sums[0];
}

__device__ __forceinline__ void store_out(const Down &a, uint64_t at, float v) {
  if (a.out_bf16)
    static_cast<uint16_t *>(a.out)[at] = (uint16_t)round2_bf16(v, 0.0f);
  else
    static_cast<float *>(a.out)[at] = v;
}

// Up to 64 pairs: a workgroup takes R rows of every expert that a pair names,
// the waves an expert (or a part of its k's) each, and adds the pairs up.
template <int F, int R, int PARTS, bool ALIGNED>
__global__ __launch_bounds__(64 * kDownWaves) void down_kernel(const Down a) {
  constexpr int kTiles = 3;
  __shared__ float y[kDownWaves * kFewPairs * R];  // [split][pair][row]
  __shared__ alignas(16) uint8_t tiles[kDownWaves * DownDot<F, R, kTiles, PARTS, ALIGNED>::kLds];
  const uint32_t tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const uint32_t pairs = a.tokens * a.topk, n0 = blockIdx.x * (uint32_t)R, r = lane % 16u, q = lane / 16u;
  // lane p's pair: the others of its expert, and whether it is their first
  const int e = lane < pairs ? expert_of(a.ids, a.ids64, lane, a.experts) : -1;
  uint64_t same = __builtin_amdgcn_ballot_w64(e >= 0);
  const uint64_t held = same;
  for (uint32_t b = 1; b < a.experts; b <<= 1) {
    const bool one = (e & b) != 0;
    const uint64_t m = __builtin_amdgcn_ballot_w64(one);
    same &= one ? m : ~m;
  }
  uint64_t first = __builtin_amdgcn_ballot_w64(e >= 0 && (uint32_t)__builtin_ctzll(same) == lane);
  // where experts are fewer than waves, several waves share one's k's
  const uint32_t experts = (uint32_t)__builtin_popcountll(first);
  const uint32_t whole = DownDot<F, R, kTiles, PARTS, ALIGNED>::tiles(a.inter);
  uint32_t splits = 1;
  while (experts * splits * 2 <= (uint32_t)kDownWaves && splits * 2 <= whole) splits *= 2;
  for (uint32_t item = 0; item < experts * splits; ++item) {
    const uint32_t leader = uniform((uint32_t)__builtin_ctzll(first)), s = item % splits;
    if (s == splits - 1) first &= first - 1;
    if (item % kDownWaves != wid) continue;
    uint64_t mine = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)same, leader) |
                    (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(same >> 32), leader) << 32;
    const uint32_t x = (uint32_t)__builtin_amdgcn_readlane(e, leader);
    while (mine) {                       // 16 pairs at a time: the j-th of them is lane j's
      uint32_t pair = 0, c = 0;
      for (; c < 16 && mine; ++c, mine &= mine - 1) {
        const uint32_t p = (uint32_t)__builtin_ctzll(mine);
        pair = r >= c ? p : pair;
      }
      const f32x4 sums = down_tile<F, R, kTiles, PARTS, ALIGNED>(
          a, x, n0, pair, whole * s / splits, whole * (s + 1) / splits, tiles + wid * DownDot<F, R, kTiles, PARTS, ALIGNED>::kLds);
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t to = (uint32_t)__shfl((int)pair, (int)(4u * q + i));
        if (4u * q + i < c && r < R) y[(s * pairs + to) * R + r] = sums[i];
      }
    }
  }
  __syncthreads();
  for (uint32_t i = tid; i < a.tokens * R; i += 64u * kDownWaves) {
    const uint32_t t = i / R, c = i % R;
    if (n0 + c >= a.hidden) continue;
    float sum = 0.0f;
    for (uint32_t j = 0; j < a.topk; ++j) {
      const uint32_t p = t * a.topk + j;
      if (!(held >> p & 1)) continue;
      float v = 0.0f;
      for (uint32_t s = 0; s < splits; ++s) v += y[(s * pairs + p) * R + c];
      sum = __builtin_fmaf(a.weights[p], v, sum);
    }
    store_out(a, (uint64_t)t * a.hidden + n0 + c, sum);
  }
}

// y of the pairs of one expert, 16 rows a wave.
template <int F, int PARTS, bool ALIGNED>
__global__ __launch_bounds__(64 * kRowsWaves) void down_rows_kernel(const Down a) {
  constexpr int kTiles = 3;
  __shared__ uint16_t list[kMaxPairs];
  __shared__ alignas(16) uint8_t tiles[kRowsWaves * DownDot<F, 16, kTiles, PARTS, ALIGNED>::kLds];
  const uint32_t lane = lane_id(), wid = uniform(threadIdx.x / kWave), r = lane % 16u, q = lane / 16u;
  int e;
  const uint32_t count = expert_pairs(a.ids, a.ids64, a.by_pair, a.tokens * a.topk, a.experts, blockIdx.x / a.groups,
                                      list, e);
  const uint32_t n0 = (blockIdx.x % a.groups * kRowsWaves + wid) * 16u;
  if (count == 0 || n0 >= a.hidden) return;
  for (uint32_t m0 = 0; m0 < count; m0 += 16u) {
    const uint32_t n = count - m0 < 16u ? count - m0 : 16u;
    const f32x4 sums = down_tile<F, 16, kTiles, PARTS, ALIGNED>(
        a, (uint32_t)e, n0, list[m0 + (r < n ? r : n - 1)], 0, ~0u, tiles + wid * DownDot<F, 16, kTiles, PARTS, ALIGNED>::kLds);
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      if (4u * q + i < n && n0 + r < a.hidden) a.y[(uint64_t)list[m0 + 4u * q + i] * a.hidden + n0 + r] = sums[i];
  }
}

// out_t = sum of the token's y.
__global__ __launch_bounds__(256) void combine_kernel(const Down a) {
  const uint32_t column = blockIdx.x * 256u + threadIdx.x, t = blockIdx.y;
  if (column >= a.hidden) return;
  float sum = 0.0f;
#pragma unroll 4
  for (uint32_t j = 0; j < a.topk; ++j) {
    const uint32_t p = t * a.topk + j;
    if (expert_of(a.ids, a.ids64, p, a.experts) < 0) continue;
    sum = __builtin_fmaf(a.weights[p], a.y[(uint64_t)p * a.hidden + column], sum);
  }
  store_out(a, (uint64_t)t * a.hidden + column, sum);
}

uint32_t padded(uint32_t inter) { return (inter + 15u) / 16u * 16u; }

template <int F>
bool aligned_rows(const ExpertMatrix &m, uint32_t k) {
  return reinterpret_cast<uintptr_t>(m.rows) % 16 == 0 && row_bytes<F>(k) % 16 == 0;
}

template <int F, bool ALIGNED>
void gate_up_launch(const GateUp &g, hipStream_t stream) {
  hipLaunchKernelGGL((gate_up_kernel<F, ALIGNED>), dim3((g.by_pair ? g.pairs : g.experts) * g.tiles),
                     dim3(64 * kGateUpWaves), 0, stream, g);
}

template <int F, int R, bool ALIGNED>
void down_launch(const Down &d, hipStream_t stream) {
  const dim3 grid((d.hidden + R - 1) / R), block(64 * kDownWaves);
  if (d.out_bf16)
    hipLaunchKernelGGL((down_kernel<F, R, 2, ALIGNED>), grid, block, 0, stream, d);
  else
    hipLaunchKernelGGL((down_kernel<F, R, 3, ALIGNED>), grid, block, 0, stream, d);
}

template <int F, bool ALIGNED>
void down_rows_launch(const Down &d, hipStream_t stream) {
  const dim3 grid((d.by_pair ? d.tokens * d.topk : d.experts) * d.groups), block(64 * kRowsWaves);
  if (d.out_bf16)
    hipLaunchKernelGGL((down_rows_kernel<F, 2, ALIGNED>), grid, block, 0, stream, d);
  else
    hipLaunchKernelGGL((down_rows_kernel<F, 3, ALIGNED>), grid, block, 0, stream, d);
}

// Bytes of the workspace's h, a multiple of 16.
uint64_t h_bytes(uint32_t pairs, uint32_t inter, bool out_bf16) {
  return 2ull * (out_bf16 ? 2 : 3) * pairs * padded(inter);
}

template <int F>
hipError_t experts_launch(const MoeExperts &a, hipStream_t stream) {
  const uint32_t pairs = a.tokens * a.topk;
  if (a.inter) {
    const GateUp g{a.x, a.ids, a.ids64, pairs < a.experts, pairs, a.topk, a.experts, a.hidden, a.inter,
                   (a.inter + 15u) / 16u, padded(a.inter), a.out_bf16 ? 2 : 3, a.gate, a.up, a.workspace};
    if (aligned_rows<F>(a.gate, a.hidden) && aligned_rows<F>(a.up, a.hidden))
      gate_up_launch<F, true>(g, stream);
    else
      gate_up_launch<F, false>(g, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const Down d{a.workspace, a.ids, a.weights, a.ids64, pairs < a.experts, a.out_bf16, a.tokens, a.topk,
               a.inter ? a.experts : 0, a.hidden, a.inter, padded(a.inter), (a.hidden + 16 * kRowsWaves - 1) / (16 * kRowsWaves),
               a.down, reinterpret_cast<float *>(a.workspace + h_bytes(pairs, a.inter, a.out_bf16) / 2), a.out};
  const bool aligned = aligned_rows<F>(a.down, a.inter);
  if (pairs <= kFewPairs || a.inter == 0) {
    if (aligned)
      d.hidden < 4096 ? down_launch<F, 8, true>(d, stream) : down_launch<F, 16, true>(d, stream);
    else
      d.hidden < 4096 ? down_launch<F, 8, false>(d, stream) : down_launch<F, 16, false>(d, stream);
    return hipGetLastError();
  }
  aligned ? down_rows_launch<F, true>(d, stream) : down_rows_launch<F, false>(d, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(combine_kernel, dim3((a.hidden + 255u) / 256u, a.tokens), dim3(256), 0, stream, d);
  return hipGetLastError();
}

}  // namespace

uint64_t moe_experts_workspace(uint32_t pairs, uint32_t hidden, uint32_t inter, bool out_bf16) {
  if (!inter) return 0;
  return h_bytes(pairs, inter, out_bf16) + (pairs <= kFewPairs ? 0 : 4ull * pairs * hidden);
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
