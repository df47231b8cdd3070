/*
 * fp8q_layer.h -- C ABI of the MoE layer's activation path on MI355X
 * (gfx950): rows of the residual stream normed straight into 8 bits, sent to
 * their experts in the codec's formats, and brought back, with the gradients
 * that training needs.  The library is libfp8q_layer.so; formats, status
 * codes and the scale rules are those of fp8q.h (libfp8q.so), whose
 * dequantize and reduce entry points read what these write.
 *
 * Conventions: those of fp8q.h.  Data pointers are device pointers on the
 * current HIP device; calls enqueue on `stream` and return without
 * synchronising; the caller owns every buffer, workspaces included, and the
 * library allocates nothing and keeps no state; every argument is checked on
 * the host before any launch, and a rejected call writes nothing; every entry
 * point can be captured in a HIP graph.  Data pointers are 16-byte aligned,
 * except: fp32 scales, rstd, slots, pairs, offsets, weights of rows and their
 * gradients 4 bytes, int64 ids 8 bytes, int32 ids 4 bytes, E8M0 scales any.
 * No output may overlap an input or another output, except where an entry
 * point says that a buffer may be updated in place.  Rows need no alignment
 * of their own: any `hidden` is allowed, and a row starts where the one
 * before it ends.
 *
 * "Rows" below are [count, hidden], row-major.  Rows in 8 bits carry scales:
 *   E4M3 / E5M2  fp32 [count, ceil(hidden / 128)], one per 128 elements of a
 *                row, the row's last block partial where hidden % 128 != 0
 *                (with hidden % 128 == 0 this is fp8q.h's flat layout);
 *   MXFP8        E8M0 [count, hidden / 32], hidden a multiple of 32.
 */
#ifndef FP8Q_LAYER_H
#define FP8Q_LAYER_H

#include "fp8q.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8Q_NORM_MAX_HIDDEN 32768   /* longest row of the norm entry points      */
#define FP8Q_MAX_HIDDEN (((size_t)1) << 20) /* longest row of the moe entry points */
#define FP8Q_MAX_TOPK 64             /* most experts a token                      */
#define FP8Q_MAX_EXPERTS 1024        /* most experts                              */
#define FP8Q_MAX_PAIRS (((size_t)1) << 30)  /* tokens * topk: pairs are int32     */

typedef enum {
    FP8Q_WEIGHT_F32 = 0,
    FP8Q_WEIGHT_BF16 = 1
} fp8q_weight_dtype;

typedef enum {
    FP8Q_ROWS_BF16 = 0,              /* bf16, no scales                           */
    FP8Q_ROWS_E4M3 = 1,              /* E4M3 codes, fp32 scales per 128           */
    FP8Q_ROWS_E5M2 = 2,              /* E5M2 codes, fp32 scales per 128           */
    FP8Q_ROWS_MX8 = 3                /* E4M3 codes, E8M0 scales per 32            */
} fp8q_row_format;

/*
 * Root-mean-square norm of the residual stream, into 8 bits with scales.
 * Per row, all in fp32:
 *   h    = x + residual                      (x where there is no residual)
 *   rstd = 1 / sqrt(sum(h * h) / hidden + eps)
 *   y    = (h * rstd) * weight
 * and y is quantized by the rule of fp8q_quantize (block amax / FP8_MAX, an
 * fp32 scale per 128 elements) or of mx8_quantize (an E8M0 scale per 32),
 * applied to the fp32 values: the norm is taken of the unrounded sum, and y
 * is rounded once.  A block holding an inf or NaN gets the codec's NaN scale
 * and codes 0x7F.  The sum of squares is held in fp32: a row where it passes
 * fp32's range (values of about 1e19) has rstd 0; with eps 0, a row where it
 * underflows to 0 (all values under 2^-75, about 2.6e-23, zeros included) has
 * rstd inf, y inf or NaN (0 * inf), and so NaN scales, and one where it is
 * subnormal (values under about 1e-19) an rstd of a subnormal's precision.
 * Any eps from 1e-30 up is far from all of that at the small end.
 * rows == 0 or hidden == 0 is a successful no-op.
 *   x_bf16, residual_bf16  [rows, hidden]; residual NULL: none
 *   weight                 [hidden] fp32 or bf16
 *   eps                    finite, >= 0
 *   h_out                  [rows, hidden] bf16, RNE(h), or NULL; only with a
 *                          residual.  May be x_bf16 or residual_bf16 itself
 *                          (the residual stream updated in place).
 *   y_out                  [rows, hidden] bf16, RNE(y), or NULL (a router
 *                          reads it)
 *   q_out, scales / e8m0   rows in 8 bits with their scales
 *   rstd_out               [rows] fp32, or NULL (a backward pass reads it)
 */
FP8Q_API fp8q_status fp8q_rms_norm_quantize(const void *x_bf16, const void *residual_bf16,
                                            const void *weight, fp8q_weight_dtype weight_dtype,
                                            float eps, size_t rows, size_t hidden,
                                            fp8q_format fmt, void *h_out, void *y_out,
                                            void *q_out, float *scales_out, float *rstd_out,
                                            void *stream);
FP8Q_API fp8q_status mx8_rms_norm_quantize(const void *x_bf16, const void *residual_bf16,
                                           const void *weight, fp8q_weight_dtype weight_dtype,
                                           float eps, size_t rows, size_t hidden, void *h_out,
                                           void *y_out, void *q_out, void *e8m0_out,
                                           float *rstd_out, void *stream);

/*
 * The norm's backward pass, straight through the 8-bit rounding: with dy the
 * gradient of y and dh that of the residual stream past this point (NULL:
 * none), per row
 *   g  = weight * dy,   c = sum(g * h) / hidden * rstd^2
 *   dx = (g - h * c) * rstd + dh        (x's and the residual's gradient)
 *   dweight = sum over the rows of dy * (h * rstd)
 * in fp32, dx rounded once to bf16, dweight fp32.  The rows are summed in a
 * fixed order: the same call gives the same bits.  rows == 0 writes zeros to
 * dweight.  hidden == 0 is a no-op.
 *   dy_bf16, h_bf16, dh_bf16, dx_out  [rows, hidden] bf16; dx_out may be
 *                                     dy_bf16 or dh_bf16 itself
 *   weight                            as in the forward pass
 *   rstd                              [rows] fp32, of the forward pass
 *   dweight_out                       [hidden] fp32
 *   workspace                         fp8q_rms_norm_backward_workspace bytes
 *                                     (NULL where that is 0), 16-byte aligned;
 *                                     its contents are not kept
 */
FP8Q_API size_t fp8q_rms_norm_backward_workspace(size_t rows, size_t hidden);
FP8Q_API fp8q_status fp8q_rms_norm_backward(const void *dy_bf16, const void *h_bf16,
                                            const void *weight, fp8q_weight_dtype weight_dtype,
                                            const float *rstd, const void *dh_bf16, size_t rows,
                                            size_t hidden, void *dx_out, float *dweight_out,
                                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * Tokens sorted by expert.  Pair p = t * topk + j is token t's j-th choice,
 * ids[p] its expert.  The pairs of expert 0 come first, then expert 1's, each
 * expert's in ascending p (a stable sort); a pair whose id is not in
 * [0, experts) (padding, or an expert that lives elsewhere) has no place.
 *   ids          [tokens, topk] int32 (id_bytes 4) or int64 (id_bytes 8)
 *   slots_out    [tokens, topk] int32: the pair's place, -1 if it has none
 *   pairs_out    [tokens * topk] int32: the pair at a place, -1 past the last
 *   offsets_out  [experts + 1] int32: each expert's first place; the last
 *                entry is the number of places
 *   workspace    fp8q_moe_sort_workspace bytes (NULL where that is 0),
 *                16-byte aligned; its contents are not kept
 * topk 1 .. FP8Q_MAX_TOPK, experts 1 .. FP8Q_MAX_EXPERTS, tokens * topk up to
 * FP8Q_MAX_PAIRS.  tokens == 0 writes zeros to offsets.
 */
FP8Q_API size_t fp8q_moe_sort_workspace(size_t tokens, int topk, int experts);
FP8Q_API fp8q_status fp8q_moe_sort(const void *ids, int id_bytes, size_t tokens, int topk,
                                   int experts, int *slots_out, int *pairs_out, int *offsets_out,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * The tokens' rows written to their places, scales alongside:
 *   dst[slots[t, j]] = src[t]      for every slot in [0, dst_rows)
 * Bytes are copied as they are, so rows may be of any type: row_bytes bytes
 * each, and scale_row_bytes bytes of scales (0 and NULL: none; each at most
 * 4 * FP8Q_MAX_HIDDEN).  Each source
 * row is read once, however many experts it goes to.  Rows of dst that no
 * slot names are not written; a slot outside [0, dst_rows) is skipped.
 *   src, src_scales  [tokens] rows of row_bytes / scale_row_bytes
 *   slots            [tokens, topk] int32 (fp8q_moe_sort), all different
 *   dst, dst_scales  [dst_rows] rows
 * The scale arrays may have any alignment.
 */
FP8Q_API fp8q_status fp8q_moe_permute(const void *src, size_t row_bytes, const void *src_scales,
                                      size_t scale_row_bytes, const int *slots, size_t tokens,
                                      int topk, size_t dst_rows, void *dst, void *dst_scales,
                                      void *stream);

/*
 * Each token's expert rows, weighted and summed:
 *   acc = 0;  acc = fma(weights[t, j], dec(rows[slots[t, j]]), acc)  for
 *   j = 0, 1, ... over the slots in [0, row_count);  out[t] = acc
 * in fp32, written as fp32 or rounded once to bf16.  dec is the value itself
 * (bf16) or code * scale, rounded to fp32, as the codec's dequantize gives it.
 * A token without a slot gets zeros, and no row that no slot names is read.
 * weights NULL: ones, which with bf16 rows is the gradient of
 * fp8q_moe_permute.
 *   rows, scales  [row_count] rows of `format`; scales NULL for bf16
 *   slots         [tokens, topk] int32
 *   weights       [tokens, topk] fp32, or NULL
 *   out           [tokens, hidden]
 */
FP8Q_API fp8q_status fp8q_moe_combine(const void *rows, fp8q_row_format format, const void *scales,
                                      const int *slots, const float *weights, size_t tokens,
                                      int topk, size_t row_count, size_t hidden, void *out,
                                      fp8q_out_dtype out_dtype, void *stream);

/*
 * The gradients of fp8q_moe_combine over bf16 rows: for every slot s = slots[t, j]
 * in [0, row_count) (rows in 8 bits are to be dequantized first)
 *   drows[s] = weights[t, j] * dy[t]                 (fp32, rounded once)
 *   dweights[t, j] = sum over hidden of dy[t] * rows[s]
 * and dweights[t, j] = 0 for every other slot.  Rows of drows that no slot
 * names are not written.
 *   dy_bf16           [tokens, hidden] bf16
 *   rows_bf16         [row_count, hidden] bf16, the forward pass's
 *   slots, weights    [tokens, topk]; slots all different
 *   drows_out         [row_count, hidden] bf16
 *   dweights_out      [tokens, topk] fp32
 */
FP8Q_API fp8q_status fp8q_moe_combine_backward(const void *dy_bf16, const void *rows_bf16,
                                               const int *slots, const float *weights,
                                               size_t tokens, int topk, size_t row_count,
                                               size_t hidden, void *drows_out,
                                               float *dweights_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_LAYER_H */
