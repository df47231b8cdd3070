// moe_experts.hip -- a whole MoE layer for a few tokens, from weights in the
// codec's formats, on gfx950.
//
//   up to 24 pairs (kFewPairs):
//     gate_up_kernel  h[p] = silu(gate_e x_t) * (up_e x_t) of every pair p
//     down_kernel     out_t = sum over the token's pairs of weight * (down_e h[p])
//   more:
//     wide_kernel     h[p], and again y[p] = down_e h[p]
//     combine_kernel  out_t = sum over the token's pairs of weight * y[p]
//   inter == 0: combine_kernel alone, of any number of pairs and no expert
//
// The rows of the experts that a token chose are read once, and little else is:
// at 8 of 128 experts of 2048 x 768 a token's MXFP8 rows are 39 MB, so HBM
// bounds all of them for as long as an expert has few tokens.  Rows that go
// straight into LDS (TileLoad) come in non-temporally, which took 10% off 32
// tokens (119 us to 107) and left one token where it was.  Measured on MI355X,
// whole calls: that layer in MXFP8, one token 17 us (its bytes at 6.5 TB/s: 6), 2
// 26 (12), 5 42 (26), 32 99 to 104 (84), 128 130 (96); 128 tokens through 2 of 8
// experts of 4096 x 14336 in bf16 504 to 525 (434).
//
// Products are 16x16x32 bf16 matrix instructions: the tokens' rows are operand
// A, 16 weight rows operand B, and both may take the k's of a chunk of 64 in
// any order, as long as it is the same.  Lane (r, q) = (lane % 16, lane / 16)
// holds k = 16 q .. 16 q + 15 of row r: 16 bytes of codes, whose first and last
// eight are two instructions' operands (of bf16 rows, 8 k's of 32: one).  A code
// becomes a bf16 exactly (E4M3 and E5M2 have at most 4 significant bits; times a
// power of two, MXFP8's scale, too).  An fp32 scale's power of two goes into the
// bf16s as well, so that sums are in fp32's range where the weights' products
// are; its significand multiplies the chunk's fp32 sums, which it can because a
// lane's sums are all of weight row r.
#include "fp8q_device.h"
#include "layer_device.h"
#include "model_launch.h"

namespace fp8q {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum RowFormat : int { kBf16 = 0, kE4M3 = 1, kE5M2 = 2, kMx8 = 3 };   // fp8q_row_format

constexpr int kGateUpWaves = 4;          // of a gate_up workgroup: they share the k's
constexpr int kDownWaves = 8;            // of a down workgroup: they share the experts
// Pairs up to which one kernel multiplies by down and adds up.  At 8 of 128
// experts of 2048 x 768 in MXFP8, 16 pairs take 27 us this way and 32 the other,
// which is a launch more; 24 pairs 38 and 34 (in bf16 49 and 50), 32 pairs 44 and
// 36 (58 and 58), since a workgroup's waves walk over four experts each here.
constexpr uint32_t kFewPairs = 24;

// The experts of pairs p[0 .. N), -1 where they have none (an id outside the
// experts, or a pair that does not exist).  The ids' loads are on their way
// together: a branch on their type for each would wait for each.
template <int N>
__device__ __forceinline__ void experts_of(const void *ids, bool ids64, const uint32_t (&p)[N], uint32_t pairs,
                                           uint32_t experts, int (&e)[N]) {
  if (ids64) {
    int64_t v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = static_cast<const int64_t *>(ids)[p[i] < pairs ? p[i] : 0u];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = p[i] < pairs && v[i] >= 0 && v[i] < (int64_t)experts ? (int)v[i] : -1;
  } else {
    int v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = static_cast<const int *>(ids)[p[i] < pairs ? p[i] : 0u];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = p[i] < pairs && v[i] >= 0 && v[i] < (int)experts ? v[i] : -1;
  }
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
constexpr uint32_t kTile = 16 * kPiece<F>;          // elements of a tile's row
template <int F>
constexpr int kVectors = F == kBf16 ? 1 : 2;        // operands of a piece

template <int F>
__host__ __device__ __forceinline__ uint64_t row_bytes(uint32_t k) {
  return F == kBf16 ? 2ull * k : k;
}
template <int F>
__host__ __device__ __forceinline__ uint64_t scale_bytes(uint32_t k) {
  return F == kBf16 ? 0 : F == kMx8 ? k / kMxBlock : 4ull * ((k + kBlock - 1) / kBlock);
}

// Bytes [at, at + 16) of a row, zeros past its end, in two steps: the load, from
// inside the row, and what it takes afterwards (so that several loads are on
// their way before the first is waited for).
__device__ __forceinline__ u32x4 load_end(const uint8_t *row, uint32_t at, uint32_t bytes) {
  if (bytes >= 16u) return load16<false>(row + (at + 16u <= bytes ? at : bytes - 16u));
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll 1
  for (uint32_t j = 0; at + j < bytes; ++j) {
    const uint32_t byte = (uint32_t)row[at + j] << (8 * (j % 4));
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) v[i] |= j / 4 == i ? byte : 0u;
  }
  return v;
}
__device__ __forceinline__ u32x4 take_end(u32x4 v, uint32_t at, uint32_t bytes) {
  return shift_down(v, bytes < 16u || at + 16u <= bytes ? 0u : at + 16u - bytes, 8);
}
__device__ __forceinline__ u32x4 load_up_to(const uint8_t *row, uint32_t at, uint32_t bytes) {
  return take_end(load_end(row, at, bytes), at, bytes);
}

// The loads of a tile: rows [0, R) (those from `rows` on: the last row again) and
// bytes [at, at + 256) of them; `width` bytes a row.
//   DIRECT  rows and their length are multiples of 16 bytes: straight into LDS;
//           otherwise through registers, which `commit` writes to LDS, so that
//           several tiles' loads may be on their way together (78 choices
//           among 60 E4M3 experts of 1411 x 1000: 74 us, 2.2 TB/s)
template <int R, bool DIRECT>
struct TileLoad {
  u32x4 v[DIRECT ? 1 : R / 4];

  // All of them inside the rows.
  __device__ __forceinline__ void issue(uint8_t *tile, const uint8_t *base, uint32_t rows, uint32_t width,
                                        uint32_t at, uint32_t lane) {
#pragma unroll
    for (uint32_t i = 0; i < R / 4; ++i) {
      const uint32_t row = i * 4 + lane / 16u, p = (lane % 16u) ^ row;
      const uint32_t n = row < rows ? row : rows - 1;
      const uint8_t *from = base + (uint64_t)n * width + (at + p * 16u);
      if constexpr (DIRECT)
        __builtin_amdgcn_global_load_lds((GlobalPtr)from, (LdsPtr)(tile + i * 1024), 16, 0, 2);
      else
        v[i] = load16<false>(from);
    }
  }

  // Rows that end before at + 256: zeros behind (DIRECT: the last piece again,
  // which the reader replaces).
  __device__ __forceinline__ void issue_end(uint8_t *tile, const uint8_t *base, uint32_t rows, uint32_t width,
                                            uint32_t at, uint32_t lane) {
#pragma unroll
    for (uint32_t i = 0; i < R / 4; ++i) {
      const uint32_t row = i * 4 + lane / 16u, b = at + ((lane % 16u) ^ row) * 16u;
      const uint8_t *from = base + (uint64_t)(row < rows ? row : rows - 1) * width;
      if constexpr (DIRECT)
        __builtin_amdgcn_global_load_lds((GlobalPtr)(from + (b < width ? b : width - 16u)), (LdsPtr)(tile + i * 1024),
                                         16, 0, 2);
      else
        v[i] = load_end(from, b, width);
    }
  }

  // END: after issue_end, of the same rows and bytes.
  template <bool END>
  __device__ __forceinline__ void commit(uint8_t *tile, uint32_t width, uint32_t at, uint32_t lane) const {
    if constexpr (!DIRECT) {
#pragma unroll
      for (uint32_t i = 0; i < R / 4; ++i) {
        const uint32_t b = at + ((lane % 16u) ^ (i * 4 + lane / 16u)) * 16u;
        *reinterpret_cast<u32x4 *>(tile + i * 1024 + lane * 16u) = END ? take_end(v[i], b, width) : v[i];
      }
    }
  }
};

// The lane's piece of chunk c (four pieces a row).
template <int R>
__device__ __forceinline__ u32x4 read_piece(const uint8_t *tile, uint32_t c, uint32_t r, uint32_t q) {
  return *reinterpret_cast<const u32x4 *>(tile + (r % R) * kRowBytes + (((c * 4u + q) ^ (r % R)) * 16u));
}

// Eight codes as bf16 values, times the scale's power of two.
template <int F>
__device__ __forceinline__ bf16x8 widen_codes(uint32_t lo, uint32_t hi, float scale) {
  bf16x2 a, b, c, d;
  if constexpr (F == kE5M2) {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, true);
  } else {
    a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  }
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// An fp32 scale in two factors, both exact: a power of two that leaves every
// code a normal bf16 (2^-110 to 2^111: E5M2's codes go from 2^-16 to under
// 2^16), and the rest, the significand of scales in that range.  An infinite or
// NaN scale's rest is infinite or NaN.
struct SplitScale {
  float power, rest;

  __device__ __forceinline__ explicit SplitScale(float scale) {
    constexpr uint32_t kLeast = 17u << 23, kMost = 238u << 23;
    const uint32_t e = __float_as_uint(scale) & 0x7F800000u, p = e < kLeast ? kLeast : e > kMost ? kMost : e;
    power = __uint_as_float(p);
    rest = scale * __uint_as_float((254u << 23) - p);
  }
};

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

// Scales of a lane's row over a tile of codes (256 k's): fp32 a block of 128, or
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

  // Where the row ends inside the tile: what is behind is not used.
  __device__ __forceinline__ void load_end(const uint8_t *row, uint32_t e, uint32_t k) {
    if constexpr (F == kMx8) {
      const uint32_t blocks = k / kMxBlock, at = e / kMxBlock;
      uint64_t v = 0;
      if (blocks >= 8) {
        const u32x2 u = load8<false>(row + blocks - 8);
        v = (u.x | (uint64_t)u.y << 32) >> (8 * (at + 8 - blocks));
      } else {
#pragma unroll 1
        for (uint32_t i = 0; i < blocks; ++i) v |= (uint64_t)row[i] << (8 * i);
      }
      w[0] = (uint32_t)v;
      w[1] = (uint32_t)(v >> 32);
    } else if constexpr (F != kBf16) {
      const uint32_t *p = reinterpret_cast<const uint32_t *>(row);
      w[0] = p[e / kBlock];
      w[1] = p[(k - 1) / kBlock];
    }
  }

  __device__ __forceinline__ float of(int c, uint32_t q) const {
    return scale_of<F>(F == kMx8 ? w[c / 2] >> (16 * (c % 2) + 8 * (q / 2u)) : w[c / 2]);
  }

  // Of a tile at element e in which the row ends: 0 for a chunk behind it, whose
  // products' sum, 0 too, an infinite scale would make a NaN.
  __device__ __forceinline__ float of_end(int c, uint32_t q, uint32_t e, uint32_t k) const {
    return (F == kE4M3 || F == kE5M2) && e + c * 4u * kPiece<F> >= k ? 0.0f : of(c, q);
  }
};

// A lane's k's of a token's row that one piece of weights meets.
template <int F, int PARTS>
struct Operand {
  u32x4 v[PARTS][kVectors<F>];
};

// A piece of weights as operands, and what their products' sum is multiplied by.
template <int F>
struct Weights {
  bf16x8 b[kVectors<F>];
  float scale;

  __device__ __forceinline__ Weights(u32x4 w, float s) : scale(s) {
    if constexpr (F == kBf16) {
      b[0] = __builtin_bit_cast(bf16x8, w);
    } else {
      float power = s;
      if constexpr (F != kMx8) {
        const SplitScale split(s);
        power = split.power;
        scale = split.rest;
      }
      b[0] = widen_codes<F>(w.x, w.y, power);
      b[kVectors<F> - 1] = widen_codes<F>(w.z, w.w, power);
    }
  }
};

// sums += one chunk's products.
template <int F, int PARTS>
__device__ __forceinline__ void multiply(f32x4 &sums, const Operand<F, PARTS> &t, const Weights<F> &w) {
  constexpr bool kScaled = F == kE4M3 || F == kE5M2;
  f32x4 d = kScaled ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sums;
#pragma unroll
  for (int i = PARTS - 1; i >= 0; --i)                   // the smallest parts first
#pragma unroll
    for (int v = 0; v < kVectors<F>; ++v) d = matrix_step(t.v[i][v], w.b[v], d);
  if constexpr (kScaled) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[i] = __builtin_fmaf(w.scale, d[i], sums[i]);
  } else {
    sums = d;
  }
}

// What a wave multiplies by itself: N matrices' rows, and the rows of 16 tokens
// (the lane's one; `parts` elements from one part of a row to the next), which
// it loads straight into registers: few tokens are few lines.
//   R       rows of a tile
//   TILES   tiles of each matrix that are loaded at once
//   PADDED  token rows are zeros from k to the next multiple of 16
template <int F, int N, int R, int TILES, int PARTS, bool PADDED, bool DIRECT>
struct Dot {
  static constexpr uint32_t kLds = N * TILES * R * kRowBytes;
  const uint8_t *rows[N];                                // the tile's first row (uniform)
  const uint8_t *scales[N];                              // the lane's row's
  const uint16_t *token;
  uint64_t parts;
  uint32_t count;                                        // rows there are
  uint32_t k;
  uint8_t *lds;                                          // kLds bytes

  __device__ __forceinline__ void load_tokens(Operand<F, PARTS> (&t)[4], uint32_t e, uint32_t q) const {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int v = 0; v < kVectors<F>; ++v)
          t[c].v[i][v] = load16<false>(token + i * parts + e + (c * 4u + q) * kPiece<F> + 8u * v);
  }

  // Zeros past the row's end.
  __device__ __forceinline__ void load_tokens_end(Operand<F, PARTS> (&t)[4], uint32_t e, uint32_t q) const {
    const uint32_t end = PADDED ? (k + 15u) / 16u * 16u : k;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int v = 0; v < kVectors<F>; ++v) {
          const uint32_t at = e + (c * 4u + q) * kPiece<F> + 8u * v;
          const uint16_t *row = token + i * parts;
          if constexpr (PADDED || DIRECT) {              // end is a multiple of 8
            const u32x4 x = load16<false>(row + (at < end ? at : 0u)), zero = {0u, 0u, 0u, 0u};
            t[c].v[i][v] = at < end ? x : zero;
          } else {
            t[c].v[i][v] = load_up_to(reinterpret_cast<const uint8_t *>(row), 2u * at, 2u * end);
          }
        }
  }

  // sums[n] += over W tiles' k's from element e on; END: the row ends in the last.
  template <int W, bool END>
  __device__ __forceinline__ void stage(f32x4 (&sums)[N], uint32_t e, uint32_t lane) const {
    const uint32_t r = lane % 16u, q = lane / 16u, width = (uint32_t)row_bytes<F>(k);
    const auto tile = [&](int w, int n) { return lds + (w * N + n) * (R * kRowBytes); };
    TileLoad<R, DIRECT> loads[W][N];
    Scales<F> s[N][W];
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint32_t at = (uint32_t)row_bytes<F>(e + w * kTile<F>);
        if constexpr (END) {
          loads[w][n].issue_end(tile(w, n), rows[n], count, width, at, lane);
          s[n][w].load_end(scales[n], e, k);
        } else {
          loads[w][n].issue(tile(w, n), rows[n], count, width, at, lane);
          s[n][w].load(scales[n], e + w * kTile<F>);
        }
      }
    // the tokens' rows, two tiles of them in registers
    Operand<F, PARTS> t[W > 1 ? 2 : 1][4];
    if constexpr (END)
      load_tokens_end(t[0], e, q);
    else
      load_tokens(t[0], e, q);
    if constexpr (W > 1) load_tokens(t[1], e + kTile<F>, q);
    loads_issued();
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int n = 0; n < N; ++n)
        loads[w][n].template commit<END>(tile(w, n), width, (uint32_t)row_bytes<F>(e + w * kTile<F>), lane);
    all_loaded();
    if (!DIRECT) lds_done();
#pragma unroll
    for (int w = 0; w < W; ++w) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
          u32x4 v = read_piece<R>(tile(w, n), c, r, q);
          if (END && DIRECT && (uint32_t)row_bytes<F>(e) + (c * 4u + q) * 16u >= width) v = u32x4{0u, 0u, 0u, 0u};
          multiply<F, PARTS>(sums[n], t[W > 1 ? w % 2 : 0][c], Weights<F>(v, END ? s[n][w].of_end(c, q, e, k) : s[n][w].of(c, q)));
        }
        loads_issued();
      }
      if (w + 2 < W) load_tokens(t[w % 2], e + (w + 2) * kTile<F>, q);
    }
    lds_done();                                          // before the next tiles overwrite these
  }

  // sums += over tiles [t0, t1).
  __device__ __forceinline__ void run(f32x4 (&sums)[N], uint32_t t0, uint32_t t1, uint32_t lane) const {
    const uint32_t whole = k / kTile<F> < t1 ? k / kTile<F> : t1;
    uint32_t i = t0;
    for (; i + TILES <= whole; i += TILES) stage<TILES, false>(sums, i * kTile<F>, lane);
    if constexpr (TILES > 1)
      for (; i < whole; ++i) stage<1, false>(sums, i * kTile<F>, lane);
    if (whole < t1 && t0 < t1 && whole * kTile<F> < k) stage<1, true>(sums, whole * kTile<F>, lane);
  }
};

// Tiles of a row's k's, the last one partial.
template <int F>
__host__ __device__ __forceinline__ uint32_t tiles_of(uint32_t k) {
  return (k + kTile<F> - 1) / kTile<F>;
}

struct Layer {
  const uint16_t *x;
  const void *ids;
  const float *weights;
  bool ids64, out_bf16;
  bool by_pair;                          // a workgroup's expert is a pair's
  uint32_t tokens, topk, pairs, experts, hidden, inter;
  uint32_t padded;                       // inter, up to a multiple of 16
  uint32_t groups;                       // workgroups an expert
  uint32_t splits;                       // parts of down's k's, a workgroup and a y each
  ExpertMatrix gate, up, down;
  uint16_t *h;                           // [parts][pairs][padded]: 2 or 3 bf16 numbers an h
  float *y;                              // [splits][pairs][hidden]
  void *out;
};

// The pairs of a workgroup's expert: expert `which`, or (by_pair) the one of pair
// `which` if no pair before it has the same.
struct Pairs {
  int e;
  uint32_t count;                        // 0 where there is nothing to do

  // Every wave scans all pairs; wave 0 writes those of rank [m0, m0 + most) to
  // `list`, which a barrier has to follow.
  __device__ __forceinline__ Pairs(const Layer &a, uint32_t which, uint32_t m0, uint32_t most, uint16_t *list) {
    constexpr uint32_t kAtOnce = 4;      // loads of 64 ids on their way together
    const uint32_t lane = lane_id(), wid = uniform(threadIdx.x / kWave);
    e = (int)which;
    count = 0;
    for (uint32_t p0 = 0; p0 < a.pairs; p0 += kAtOnce * kWave) {
      uint32_t p[kAtOnce + 1];
      int id[kAtOnce + 1];
#pragma unroll
      for (uint32_t i = 0; i < kAtOnce; ++i) p[i] = p0 + i * kWave + lane;
      p[kAtOnce] = which;
      experts_of(a.ids, a.ids64, p, a.pairs, a.experts, id);
      if (a.by_pair) e = (int)uniform((uint32_t)id[kAtOnce]);
#pragma unroll
      for (uint32_t i = 0; i < kAtOnce; ++i) {
        const bool same = id[i] == e && e >= 0;
        const uint64_t mask = __builtin_amdgcn_ballot_w64(same);
        if (a.by_pair && count == 0 && mask && p0 + i * kWave + (uint32_t)__builtin_ctzll(mask) != which) {
          e = -1;                        // another workgroup's
          return;
        }
        const uint32_t rank = count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                                __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
        if (same && wid == 0 && rank - m0 < most) list[rank - m0] = (uint16_t)p[i];
        count += (uint32_t)__builtin_popcountll(mask);
      }
    }
  }
};

// silu(g) * u.
__device__ __forceinline__ float gated(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// h of a pair at a column of its padded row (zeros from inter on), as a sum of
// bf16 numbers: its leading bits, and the rest's.  Two hold 16 of its bits, which
// is far past what a bf16 output shows; three hold them all.  (An inf or NaN has
// no rest.)
__device__ __forceinline__ void store_h(const Layer &a, uint32_t pair, uint32_t column, float h) {
  if (column >= a.padded) return;
  if (column >= a.inter) h = 0.0f;
  uint16_t *to = a.h + (uint64_t)pair * a.padded + column;
  const uint64_t part = (uint64_t)a.pairs * a.padded;
  const uint32_t bits = __float_as_uint(h);
  to[0] = (uint16_t)(h != h ? 0x7FC0u : bits >> 16);
  const bool finite = (bits & 0x7F800000u) != 0x7F800000u;
  const float rest = finite ? h - __uint_as_float(bits & 0xFFFF0000u) : 0.0f;
  if (a.out_bf16) {
    to[part] = (uint16_t)round2_bf16(rest, 0.0f);
  } else {
    const uint32_t b = __float_as_uint(rest);
    to[part] = (uint16_t)(b >> 16);
    to[2 * part] = (uint16_t)round2_bf16(rest - __uint_as_float(b & 0xFFFF0000u), 0.0f);
  }
}

// One tile of each at a time: two of each (64 KiB of LDS a workgroup, so two of
// them a CU) took 90 us where this took 69, for 256 pairs; and eight waves that
// share the k's 48 us where four took 40, for 2 pairs of rows of 4096.
template <int F, bool DIRECT>
using GateUpDot = Dot<F, 2, 16, 1, 1, false, DIRECT>;

// h of up to 16 pairs of one expert, for 16 of its rows, whose k's the waves
// share.
template <int F, bool DIRECT>
__device__ __forceinline__ void gate_up_tile(const Layer &a, uint32_t e, uint32_t n0, const uint16_t *list,
                                             uint32_t count, uint8_t *lds) {
  const uint32_t lane = lane_id(), r = lane % 16u, q = lane / 16u, wid = uniform(threadIdx.x / kWave);
  const uint32_t n = n0 + r < a.inter ? n0 + r : a.inter - 1;
  GateUpDot<F, DIRECT> dot;
  dot.k = a.hidden;
  dot.parts = 0;
  dot.count = a.inter - n0;
  dot.lds = lds + wid * dot.kLds;
  dot.rows[0] = a.gate.rows + (a.gate.expert_rows * e + n0) * row_bytes<F>(a.hidden);
  dot.rows[1] = a.up.rows + (a.up.expert_rows * e + n0) * row_bytes<F>(a.hidden);
  dot.scales[0] = a.gate.scales + (a.gate.expert_rows * e + n) * scale_bytes<F>(a.hidden);
  dot.scales[1] = a.up.scales + (a.up.expert_rows * e + n) * scale_bytes<F>(a.hidden);
  dot.token = a.x + (uint64_t)(list[r < count ? r : count - 1] / a.topk) * a.hidden;
  f32x4 sums[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
  const uint32_t tiles = tiles_of<F>(a.hidden);
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
    store_h(a, list[c], col, gated(g, u));
  }
}

template <int F, bool DIRECT>
__global__ __launch_bounds__(64 * kGateUpWaves) void gate_up_kernel(const Layer a) {
  __shared__ uint16_t list[kFewPairs];
  __shared__ alignas(16) uint8_t lds[kGateUpWaves * GateUpDot<F, DIRECT>::kLds];
  const uint32_t n0 = blockIdx.x % a.groups * 16u;
  const Pairs pairs(a, blockIdx.x / a.groups, 0, kFewPairs, list);
  if (pairs.count == 0) return;
  __syncthreads();
  for (uint32_t m0 = 0; m0 < pairs.count; m0 += 16u) {
    if (m0) __syncthreads();
    gate_up_tile<F, DIRECT>(a, (uint32_t)pairs.e, n0, list + m0, pairs.count - m0 < 16u ? pairs.count - m0 : 16u, lds);
  }
}

template <int F, int R, int TILES, int PARTS, bool DIRECT>
using DownDot = Dot<F, 1, R, TILES, PARTS, true, DIRECT>;

// The product of up to 16 pairs of one expert with R of its rows, over tiles
// [t0, t1) of the k's.
template <int F, int R, int TILES, int PARTS, bool DIRECT>
__device__ __forceinline__ f32x4 down_tile(const Layer &a, uint32_t e, uint32_t n0, uint32_t pair, uint32_t t0,
                                           uint32_t t1, uint8_t *lds) {
  const uint32_t lane = lane_id(), r = lane % 16u;
  const uint32_t n = n0 + r % R < a.hidden ? n0 + r % R : a.hidden - 1;
  DownDot<F, R, TILES, PARTS, DIRECT> dot;
  dot.k = a.inter;
  dot.parts = (uint64_t)a.pairs * a.padded;
  dot.count = a.hidden - n0;
  dot.lds = lds;
  dot.rows[0] = a.down.rows + (a.down.expert_rows * e + n0) * row_bytes<F>(a.inter);
  dot.scales[0] = a.down.scales + (a.down.expert_rows * e + n) * scale_bytes<F>(a.inter);
  dot.token = a.h + (uint64_t)pair * a.padded;
  f32x4 sums[1] = {{0.0f, 0.0f, 0.0f, 0.0f}};
  dot.run(sums, t0, t1, lane);
  return sums[0];
}

__device__ __forceinline__ void store_out(const Layer &a, uint64_t at, float v) {
  if (a.out_bf16)
    static_cast<uint16_t *>(a.out)[at] = (uint16_t)round2_bf16(v, 0.0f);
  else
    static_cast<float *>(a.out)[at] = v;
}

// Up to kFewPairs pairs, no more: a workgroup takes R rows of every expert that a pair
// names, the waves an expert (or a part of its k's) each, and adds the pairs up.
// R is 8 where 16 would leave CUs without a workgroup (hidden < 4096).
template <int F, int R, int PARTS, bool DIRECT>
__global__ __launch_bounds__(64 * kDownWaves) void down_kernel(const Layer a) {
  constexpr int kTiles = PARTS == 3 ? 1 : 3;       // what the registers hold
  __shared__ float y[kDownWaves * kFewPairs * R];  // [split][pair][row]
  __shared__ float weights[kFewPairs];
  __shared__ alignas(16) uint8_t tiles[kDownWaves * DownDot<F, R, kTiles, PARTS, DIRECT>::kLds];
  const uint32_t tid = threadIdx.x, lane = lane_id(), wid = uniform(tid / kWave);
  const uint32_t pairs = a.pairs, n0 = blockIdx.x * (uint32_t)R, r = lane % 16u, q = lane / 16u;
  // lane p's pair: the others of its expert, and whether it is their first
  if (tid < pairs) weights[tid] = a.weights[tid];
  int es[1];
  experts_of(a.ids, a.ids64, {lane}, pairs, a.experts, es);
  const int e = es[0];
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
  const uint32_t whole = tiles_of<F>(a.inter);
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
      const f32x4 sums = down_tile<F, R, kTiles, PARTS, DIRECT>(
          a, x, n0, pair, whole * s / splits, whole * (s + 1) / splits,
          tiles + wid * DownDot<F, R, kTiles, PARTS, DIRECT>::kLds);
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
      sum = __builtin_fmaf(weights[p], v, sum);
    }
    store_out(a, (uint64_t)t * a.hidden + n0 + c, sum);
  }
}

// out_t = sum of the token's y: lane j has the token's j-th expert and weight.
__global__ __launch_bounds__(256) void combine_kernel(const Layer a) {
  const uint32_t column = blockIdx.x * 256u + threadIdx.x, p0 = blockIdx.y * a.topk, lane = lane_id();
  const float weight = a.weights[p0 + (lane < a.topk ? lane : 0u)];
  int e[1];
  experts_of(a.ids, a.ids64, {p0 + lane}, lane < a.topk ? a.pairs : 0u, a.experts, e);
  uint64_t held = __builtin_amdgcn_ballot_w64(e[0] >= 0);
  const float *y = a.y + (uint64_t)p0 * a.hidden + (column < a.hidden ? column : 0u);
  const uint64_t split = (uint64_t)a.pairs * a.hidden;
  float sum = 0.0f;
  constexpr int kAtOnce = 8;             // loads on their way together
  while (held) {
    float v[kAtOnce], w[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint32_t j = held ? (uint32_t)__builtin_ctzll(held) : 0u;
      w[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), (int)j));
      v[i] = held ? y[(uint64_t)j * a.hidden] : 0.0f;
      if (!held) w[i] = 0.0f;
      for (uint32_t s = 1; s < a.splits; ++s) v[i] += held ? y[s * split + (uint64_t)j * a.hidden] : 0.0f;
      held &= held - 1;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) sum = __builtin_fmaf(w[i], v[i], sum);
  }
  if (column < a.hidden) store_out(a, (uint64_t)blockIdx.y * a.hidden + column, sum);
}

// More pairs: the workgroup's waves take 16 rows each of gate and of up (or twice
// 16 of down), over all of the k's, and share the tokens' rows, which go through
// LDS as the weights do: straight from memory into registers, 16 tokens are 16
// rows a load.  For 128 tokens of 2 of 8 wide bf16 experts the kernels above,
// which do that, took 1239 us, and 639 went through these; 32 tokens of 8 of 128,
// two an expert, 135 and 119.
//
// While a workgroup multiplies, its loads' place in LDS is taken, and the CU's
// other workgroups load: small ones do better than large ones (eight waves that
// share the tokens: 142 us for 119, 759 for 639).
constexpr int kWideWaves = 4;

// Of 16 M tokens, 16 times those whose rows are in LDS at once.  Where half of
// them leave room for a workgroup more a CU, and their registers do too, the
// weights are multiplied with one half after the other (gate and up of wide bf16
// experts, 128 tokens: 375 us whole, 350 in halves; down 190 and 212, MXFP8 212
// and 219).
template <int F, int M, int PARTS>
constexpr int kHeldTiles = M > 2 && F == kBf16 && PARTS == 1 ? 2 : M;

template <int F, int M, int PARTS>
constexpr uint32_t kTokenBytes = PARTS * kHeldTiles<F, M, PARTS> * 16 * 2 * kTile<F>;

// sums[n][m] = products of the wave's rows (rows[n]: the first one's, scales[n]:
// the lane's one's) with 16 M tokens' rows.
template <int F, int M, int PARTS, bool PADDED, bool DIRECT>
struct WideDot {
  const uint8_t *rows[2], *scales[2];
  uint32_t count[2];                                     // rows there are
  uint32_t k;
  const uint8_t *tokens;
  uint8_t *weights_lds;                                  // the wave's: 2 tiles
  uint8_t *tokens_lds;                                   // kTokenBytes

  // A token's 256 or 512 bytes of a tile are pieces of 16; a load takes whole
  // rows of them, and piece p of token c lies in place p ^ (c % 16).
  static constexpr uint32_t kPieces = 2 * kTile<F> / 16;
  static constexpr uint32_t kUnits = kTokenBytes<F, M, PARTS> / 1024;
  static constexpr uint32_t kLoads = (kUnits + kWideWaves - 1) / kWideWaves;   // a wave's
  static constexpr int kHeld = kHeldTiles<F, M, PARTS>, kRounds = M / kHeld;
  uint32_t from[kRounds][kLoads];                        // the lane's rows' bytes into `tokens`, one a load

  // list: the pairs (all 16 M); a pair's row is pair / per * stride bytes into
  // `tokens`, its parts part_bytes apart.
  __device__ __forceinline__ void find(const uint16_t *list, uint32_t count, uint32_t per, uint32_t stride,
                                       uint32_t part_bytes, uint32_t lane, uint32_t wid) {
#pragma unroll
    for (int h = 0; h < kRounds; ++h)
#pragma unroll
      for (uint32_t i = 0; i < kLoads; ++i) {
        const uint32_t row = ((wid * kLoads + i) * 64u + lane) / kPieces, c = h * 16u * kHeld + row % (16u * kHeld);
        from[h][i] = list[c < count ? c : count - 1] / per * stride + row / (16u * kHeld) * part_bytes;
      }
  }

  template <bool END>
  __device__ __forceinline__ void stage(f32x4 (&sums)[2][M], uint32_t e, uint32_t lane, uint32_t wid) const {
    const uint32_t r = lane % 16u, q = lane / 16u, width = (uint32_t)row_bytes<F>(k), at = (uint32_t)row_bytes<F>(e);
    TileLoad<16, DIRECT> loads[2];
    Scales<F> s[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      if constexpr (END) {
        loads[n].issue_end(weights_lds + n * 4096, rows[n], count[n], width, at, lane);
        s[n].load_end(scales[n], e, k);
      } else {
        loads[n].issue(weights_lds + n * 4096, rows[n], count[n], width, at, lane);
        s[n].load(scales[n], e);
      }
    }
    constexpr bool kTokensDirect = PADDED || DIRECT;     // rows are multiples of 16 bytes
    const uint32_t end = 2u * (PADDED ? (k + 15u) / 16u * 16u : k);
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int h = 0; h < kRounds; ++h) {
      u32x4 v[kTokensDirect ? 1 : kLoads];
#pragma unroll
      for (uint32_t i = 0; i < kLoads; ++i) {
        if (kUnits % kWideWaves && wid * kLoads + i >= kUnits) break;
        const uint32_t unit = (wid * kLoads + i) * 64u + lane;
        const uint32_t p = (unit % kPieces) ^ (unit / kPieces % 16u), b = 2u * e + p * 16u;
        const uint8_t *row_at = tokens + from[h][i];
        if constexpr (kTokensDirect)
          __builtin_amdgcn_global_load_lds((GlobalPtr)(row_at + (!END || b < end ? b : 0u)),
                                           (LdsPtr)(tokens_lds + (wid * kLoads + i) * 1024u), 16, 0, 0);
        else
          v[i] = END ? load_end(row_at, b, end) : load16<false>(row_at + b);
      }
      loads_issued();
      if (h == 0) {
#pragma unroll
        for (int n = 0; n < 2; ++n) loads[n].template commit<END>(weights_lds + n * 4096, width, at, lane);
      }
      if constexpr (!kTokensDirect) {
#pragma unroll
        for (uint32_t i = 0; i < kLoads; ++i) {
          const uint32_t unit = (wid * kLoads + i) * 64u + lane;
          const uint32_t b = 2u * e + ((unit % kPieces) ^ (unit / kPieces % 16u)) * 16u;
          if (kUnits % kWideWaves == 0 || wid * kLoads + i < kUnits)
            *reinterpret_cast<u32x4 *>(tokens_lds + unit * 16u) = END ? take_end(v[i], b, end) : v[i];
        }
      }
      all_loaded();
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        u32x4 x[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          x[n] = read_piece<16>(weights_lds + n * 4096, c, r, q);
          if (END && DIRECT && at + (c * 4u + q) * 16u >= width) x[n] = zero;
        }
        const Weights<F> w[2] = {{x[0], END ? s[0].of_end(c, q, e, k) : s[0].of(c, q)},
                                 {x[1], END ? s[1].of_end(c, q, e, k) : s[1].of(c, q)}};
#pragma unroll
        for (int m = 0; m < kHeld; ++m) {
          Operand<F, PARTS> t;
#pragma unroll
          for (int i = 0; i < PARTS; ++i)
#pragma unroll
            for (int j = 0; j < kVectors<F>; ++j) {
              const uint32_t p = (c * 4u + q) * kVectors<F> + j;
              t.v[i][j] = *reinterpret_cast<const u32x4 *>(
                  tokens_lds + ((i * kHeld + m) * 16u + r) * (kPieces * 16u) + ((p ^ r) * 16u));
              if (END && kTokensDirect && 2u * e + p * 16u >= end) t.v[i][j] = zero;
            }
#pragma unroll
          for (int n = 0; n < 2; ++n) multiply<F, PARTS>(sums[n][h * kHeld + m], t, w[n]);
        }
        loads_issued();
      }
      __syncthreads();                                   // before the next loads overwrite these
    }
  }

  // over tiles [t0, t1) of the rows
  __device__ __forceinline__ void run(f32x4 (&sums)[2][M], uint32_t t0, uint32_t t1, uint32_t lane, uint32_t wid) const {
    for (uint32_t t = t0; t < t1; ++t) {
      if ((t + 1) * kTile<F> <= k)
        stage<false>(sums, t * kTile<F>, lane, wid);
      else
        stage<true>(sums, t * kTile<F>, lane, wid);
    }
  }
};

// h of `count` pairs of one expert, up to 16 M, for the workgroup's 64 rows of
// gate and up from n0 on, or their y for its 128 rows of down, over part `split`
// of the k's.  `list`, which holds them, is in tokens_lds.
template <int F, bool DOWN, int M, int PARTS, bool DIRECT>
__device__ __forceinline__ void wide_tile(const Layer &a, uint32_t e, uint32_t n0, uint32_t split, uint16_t *list,
                                          uint32_t count, uint8_t *weights_lds, uint8_t *tokens_lds) {
  const uint32_t lane = lane_id(), r = lane % 16u, q = lane / 16u, wid = uniform(threadIdx.x / kWave);
  const uint32_t rows = DOWN ? a.hidden : a.inter, k = DOWN ? a.inter : a.hidden;
  WideDot<F, M, PARTS, DOWN, DIRECT> dot;
  dot.k = k;
  uint32_t first[2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const ExpertMatrix &w = DOWN ? a.down : n ? a.up : a.gate;
    first[n] = n0 + (DOWN ? (wid * 2u + n) * 16u : wid * 16u);
    // a wave past the last row takes that one
    const uint32_t from = first[n] < rows ? first[n] : rows - 1, row = from + r < rows ? from + r : rows - 1;
    dot.count[n] = rows - from;
    dot.rows[n] = w.rows + (w.expert_rows * e + from) * row_bytes<F>(k);
    dot.scales[n] = w.scales + (w.expert_rows * e + row) * scale_bytes<F>(k);
  }
  dot.tokens = reinterpret_cast<const uint8_t *>(DOWN ? a.h : a.x);
  dot.find(list, count, DOWN ? 1u : a.topk, 2u * (DOWN ? a.padded : a.hidden), a.pairs * a.padded * 2u, lane, wid);
  dot.weights_lds = weights_lds + wid * 8192u;
  dot.tokens_lds = tokens_lds;
  // a thread's pair, kept while the list's memory is the tokens'
  const uint16_t mine = list[threadIdx.x < count ? threadIdx.x : 0u];
  __syncthreads();
  f32x4 sums[2][M];
#pragma unroll
  for (int m = 0; m < M; ++m) sums[0][m] = sums[1][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const uint32_t tiles = tiles_of<F>(k), splits = DOWN ? a.splits : 1u;
  dot.run(sums, tiles * split / splits, tiles * (split + 1) / splits, lane, wid);
  if (threadIdx.x < 16 * M) list[threadIdx.x] = mine;
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t c = 16u * m + 4u * q + i;
      if (c >= count) continue;
      const uint32_t p = list[c];
      if constexpr (DOWN) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
          if (first[n] + r < rows) a.y[((uint64_t)split * a.pairs + p) * a.hidden + first[n] + r] = sums[n][m][i];
      } else {
        store_h(a, p, first[0] + r, gated(sums[0][m][i], sums[1][m][i]));
      }
    }
}

template <int F, bool DOWN, int M, int PARTS, bool DIRECT>
__global__ __launch_bounds__(64 * kWideWaves) void wide_kernel(const Layer a) {
  __shared__ alignas(16) uint8_t weights[kWideWaves * 8192];
  __shared__ alignas(16) uint8_t tokens[kTokenBytes<F, M, PARTS>];
  uint16_t *list = reinterpret_cast<uint16_t *>(tokens);
  // of a split's workgroups, those of one expert follow one another
  const uint32_t splits = DOWN ? a.splits : 1u, group = blockIdx.x % (a.groups * splits);
  const uint32_t n0 = group % a.groups * (kWideWaves * (DOWN ? 32u : 16u)), split = group / a.groups;
  for (uint32_t m0 = 0;; m0 += 16u * M) {
    const Pairs pairs(a, blockIdx.x / (a.groups * splits), m0, 16u * M, list);
    if (pairs.count <= m0) return;
    const uint32_t left = pairs.count - m0, e = (uint32_t)pairs.e;
    __syncthreads();
    if (M > 1 && left <= 16u)
      wide_tile<F, DOWN, 1, PARTS, DIRECT>(a, e, n0, split, list, left, weights, tokens);
    else if (M > 2 && left <= 32u)
      wide_tile<F, DOWN, 2, PARTS, DIRECT>(a, e, n0, split, list, left, weights, tokens);
    else
      wide_tile<F, DOWN, M, PARTS, DIRECT>(a, e, n0, split, list, left < 16u * M ? left : 16u * M, weights, tokens);
    if (left <= 16u * M) return;
    __syncthreads();
  }
}

uint32_t padded(uint32_t inter) { return (inter + 15u) / 16u * 16u; }

template <int F>
bool aligned_rows(const ExpertMatrix &m, uint32_t k) {
  return reinterpret_cast<uintptr_t>(m.rows) % 16 == 0 && row_bytes<F>(k) % 16 == 0;
}

// Parts of down's k's.  Where the experts' rows alone would not give every CU
// four workgroups, parts of 1024 k's or more do (256 workgroups of 14336 k's,
// 128 tokens: one part 246 us, four 189, and 4 more in the sum).
uint32_t splits_of(uint32_t pairs, uint32_t experts, uint32_t hidden, uint32_t inter) {
  const uint32_t workgroups = (pairs < experts ? pairs : experts) * ((hidden + 127u) / 128u);
  const uint32_t want = 1024u / workgroups, most = inter / 1024u;
  const uint32_t n = want < most ? want : most;
  return n < 1 ? 1 : n < 8 ? n : 8;
}

// Bytes of the workspace's h, a multiple of 16.
uint64_t h_bytes(uint32_t pairs, uint32_t inter, bool out_bf16) {
  return 2ull * (out_bf16 ? 2 : 3) * pairs * padded(inter);
}

// A launch of `groups` workgroups an expert and split.
template <typename Kernel>
hipError_t by_expert(Kernel kernel, Layer a, uint32_t groups, uint32_t splits, uint32_t waves, hipStream_t stream) {
  a.groups = groups;
  hipLaunchKernelGGL(kernel, dim3((a.by_pair ? a.pairs : a.experts) * groups * splits), dim3(64 * waves), 0, stream, a);
  return hipGetLastError();
}

// The wide kernel for `m` x 16 tokens an expert.
template <int F, bool DOWN, int PARTS, bool DIRECT>
hipError_t wide_launch(const Layer &a, int m, hipStream_t stream) {
  const uint32_t groups = DOWN ? (a.hidden + 127u) / 128u : (a.inter + 63u) / 64u;
  const uint32_t splits = DOWN ? a.splits : 1u;
  return m == 1   ? by_expert(wide_kernel<F, DOWN, 1, PARTS, DIRECT>, a, groups, splits, kWideWaves, stream)
         : m == 2 ? by_expert(wide_kernel<F, DOWN, 2, PARTS, DIRECT>, a, groups, splits, kWideWaves, stream)
                  : by_expert(wide_kernel<F, DOWN, 4, PARTS, DIRECT>, a, groups, splits, kWideWaves, stream);
}

template <int F, bool DIRECT>
hipError_t gate_up(const Layer &a, int wide, hipStream_t stream) {
  if (wide) return wide_launch<F, false, 1, DIRECT>(a, wide, stream);
  return by_expert(gate_up_kernel<F, DIRECT>, a, (a.inter + 15u) / 16u, 1, kGateUpWaves, stream);
}

hipError_t combine(const Layer &a, hipStream_t stream) {
  hipLaunchKernelGGL(combine_kernel, dim3((a.hidden + 255u) / 256u, a.tokens), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <int F, int PARTS, bool DIRECT>
hipError_t down(const Layer &a, int wide, hipStream_t stream) {
  if (!wide) {
    const dim3 block(64 * kDownWaves);
    if (a.hidden < 4096)
      hipLaunchKernelGGL((down_kernel<F, 8, PARTS, DIRECT>), dim3((a.hidden + 7u) / 8u), block, 0, stream, a);
    else
      hipLaunchKernelGGL((down_kernel<F, 16, PARTS, DIRECT>), dim3((a.hidden + 15u) / 16u), block, 0, stream, a);
    return hipGetLastError();
  }
  const hipError_t e = wide_launch<F, true, PARTS, DIRECT>(a, wide, stream);
  return e != hipSuccess ? e : combine(a, stream);
}

// 0: few pairs; else how many times 16 tokens the wide kernels hold, which have
// to be few for an expert's share of the pairs, since room for more takes LDS and
// registers from the loads: at 8 pairs an expert 16 take 134 us, 32 138 and 64
// 171; at 16 pairs of wide MXFP8 experts 419, 294 and 345; at 32 (bf16) 1229, 795
// and 551.  The share is pairs / experts, which the host knows; where few experts
// have most of the pairs it is too low (64 tokens that all choose the same 8 of
// 128: 151 us, and 71 if 64 were held).
int wide_of(uint32_t pairs, uint32_t experts) {
  if (pairs <= kFewPairs) return 0;
  const uint32_t each = (pairs + experts - 1) / experts;
  return each <= 10 ? 1 : each <= 20 ? 2 : 4;
}

template <int F>
hipError_t experts_launch(const MoeExperts &m, hipStream_t stream) {
  const uint32_t pairs = m.tokens * m.topk;
  const Layer a{m.x, m.ids, m.weights, m.ids64, m.out_bf16, pairs < m.experts, m.tokens, m.topk, pairs,
                m.inter ? m.experts : 0, m.hidden, m.inter, padded(m.inter), 0,
                splits_of(pairs, m.experts, m.hidden, m.inter), m.gate, m.up, m.down, m.workspace,
                reinterpret_cast<float *>(m.workspace + h_bytes(pairs, m.inter, m.out_bf16) / 2), m.out};
  if (!m.inter) return combine(a, stream);                // of no experts: zeros, and no y is read
  const int wide = wide_of(pairs, m.experts);
  const bool gate_up_direct = aligned_rows<F>(m.gate, m.hidden) && aligned_rows<F>(m.up, m.hidden);
  const hipError_t e = gate_up_direct ? gate_up<F, true>(a, wide, stream) : gate_up<F, false>(a, wide, stream);
  if (e != hipSuccess) return e;
  const bool direct = aligned_rows<F>(m.down, m.inter);
  if (m.out_bf16) return direct ? down<F, 2, true>(a, wide, stream) : down<F, 2, false>(a, wide, stream);
  return direct ? down<F, 3, true>(a, wide, stream) : down<F, 3, false>(a, wide, stream);
}

}  // namespace

uint64_t moe_experts_workspace(uint32_t pairs, uint32_t experts, uint32_t hidden, uint32_t inter, bool out_bf16) {
  if (!inter || !hidden) return 0;
  return h_bytes(pairs, inter, out_bf16) +
         (pairs <= kFewPairs ? 0 : 4ull * splits_of(pairs, experts, hidden, inter) * pairs * hidden);
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
