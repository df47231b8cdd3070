/*
 * fp8q_model.h -- C ABI of the model's operators on both ends of the wire, on
 * MI355X (gfx950).  A receiver serves an MoE layer straight from weights in
 * the codec's formats: routing, and the whole layer for a few tokens.  A
 * trainer takes the routing's gradient, and the norm of its gradients and
 * their clipping between the reduce and the update.  The library is
 * libfp8q_model.so; formats, status codes and scale rules are those of fp8q.h
 * (libfp8q.so) and the limits of experts those of fp8q_layer.h
 * (libfp8q_layer.so), whose sort, permute and combine read what the routing
 * writes.
 *
 * Conventions: those of fp8q.h.  Data pointers are device pointers on the
 * current HIP device; calls enqueue on `stream` and return without
 * synchronising; the caller owns every buffer, workspaces included, and the
 * library allocates nothing and keeps no state; every argument is checked on
 * the host before any launch, and a rejected call writes nothing; every entry
 * point can be captured in a HIP graph (lists of structs are read during the
 * call only).  A workspace's contents are not kept, and two calls that may run
 * at once need one each.  No output may overlap an input or another output,
 * except where an entry point updates a buffer in place.
 */
#ifndef FP8Q_MODEL_H
#define FP8Q_MODEL_H

#include "fp8q_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8Q_EXPERTS_MAX_PAIRS 1024     /* tokens * topk of fp8q_moe_experts     */
#define FP8Q_EXPERTS_MAX_SIZE 65536     /* its longest row (hidden and inter)    */

typedef enum {
    FP8Q_LOGITS_F32 = 0,
    FP8Q_LOGITS_BF16 = 1
} fp8q_logits_dtype;

/*
 * Routing: each token's topk largest logits and their softmax weights.
 *   candidates  the experts whose logit is not -inf (NaN counts as one)
 *   ids[t, j]   the expert of the j-th largest logit: NaN before +inf before
 *               the rest, of equal ones (-0 and +0 are equal) the lowest index
 *               first; -1 where the token has no j-th candidate
 *   p[t, i]     exp(logits[t, i] - max) / sum over the candidates
 *   weights[t, j] = p[t, ids[t, j]], with `normalize` over the sum of the
 *               chosen ones' p; 0 where ids is -1
 * in fp32.  A row that holds a NaN or +inf gets NaN weights.  A row that is
 * -inf throughout (a padding token) gets ids of -1 and weights of 0, which
 * fp8q_moe_sort and fp8q_moe_experts take as tokens without experts.
 * tokens == 0 is a successful no-op.
 *   logits       [tokens, experts] fp32 or bf16, experts 1 .. FP8Q_MAX_EXPERTS,
 *                16-byte aligned
 *   weights_out  [tokens, topk] fp32, topk 1 .. FP8Q_MAX_TOPK and at most
 *                experts; tokens * topk up to FP8Q_MAX_PAIRS
 *   ids_out      [tokens, topk] int32
 */
FP8Q_API fp8q_status fp8q_moe_route(const void *logits, fp8q_logits_dtype dtype, size_t tokens,
                                    int experts, int topk, int normalize, float *weights_out,
                                    int *ids_out, void *stream);

/*
 * The routing's gradient: with c(t) the choices whose id is in [0, experts),
 *   normalize:  dlogits[t, i] = sum over j in c(t) with ids[t, j] == i of
 *                               weights[t, j] * (dweights[t, j] - s(t))
 *   otherwise:  the same sum of weights[t, j] * dweights[t, j], minus
 *               p[t, i] * s(t)
 *   s(t) = sum over c(t) of weights[t, j] * dweights[t, j]
 * in fp32, dlogits rounded once to the logits' type.  The choice itself has no
 * gradient.  A dweights entry outside c(t) is not used.  A row without a
 * candidate gets zeros.
 *   dweights, weights, ids  [tokens, topk], the forward pass's last two
 *   logits                  [tokens, experts]; not read (may be NULL) with
 *                           `normalize`
 *   dlogits_out             [tokens, experts] of `dtype`, 16-byte aligned; may
 *                           be `logits` itself
 */
FP8Q_API fp8q_status fp8q_moe_route_backward(const float *dweights, const void *logits,
                                             fp8q_logits_dtype dtype, const float *weights,
                                             const int *ids, size_t tokens, int experts, int topk,
                                             int normalize, void *dlogits_out, void *stream);

/*
 * One matrix of every expert: expert e's rows [r, width] are rows
 * [e * expert_rows, e * expert_rows + r) of one array of rows in a
 * fp8q_row_format: bf16, codes with ceil(width / 128) fp32 scales a row, or
 * MXFP8.  mx8_quantize leaves matrices so, and fp8q_quantize those whose width
 * is a multiple of 128 (its blocks run on from row to row; others are quantized
 * a row at a time).  expert_rows >= r: gate and up may be the two halves of one
 * [experts, 2 * inter, hidden] array.  Codes need no alignment, bf16 rows 2
 * bytes, fp32 scales 4.
 */
typedef struct {
    const void *rows;
    const void *scales;      /* NULL for bf16                                */
    size_t expert_rows;      /* rows from one expert's first to the next's   */
} fp8q_expert_matrix;

/*
 * A whole MoE layer for a few tokens.  Pair p = t * topk + j is token t's j-th
 * choice, e = ids[p]; for each with e in [0, experts)
 *   g = gate_e x_t,  u = up_e x_t,  h = g / (1 + exp(-g)) * u,  y_p = down_e h
 *   out_t = sum over j of weights[p] * y_p     (fused multiply-adds, j = 0, 1, ...)
 * and other pairs (padding, or an expert that lives elsewhere) are left out: a
 * token without any gets zeros.  The weights' values are exact (a code times
 * its scale is not rounded), products are summed in fp32, and g, u, h and y
 * are fp32 values; for bf16 output h is held to 15 bits or more, as two bf16
 * numbers.  Values under 2^-126 in magnitude (of x, weights and h) may be taken
 * as zero, and MXFP8 values past fp32's range are infinite, as mx8_dequantize
 * has them.  An infinite fp32 scale makes the g, u or y that it is part of
 * infinite or NaN: it multiplies the sum of 64 of its block's products, where
 * code * scale summed one by one would be NaN for codes of both signs.
 * The same expert may be chosen twice by one token.  The same call gives the
 * same bits.  tokens == 0 or hidden == 0 is a successful no-op; with inter == 0
 * out is zeros.
 *   x_bf16     [tokens, hidden], 16-byte aligned
 *   ids        [tokens, topk] int32 (id_bytes 4) or int64 (id_bytes 8)
 *   weights    [tokens, topk] fp32
 *   gate, up   rows [inter, hidden] an expert; down [hidden, inter]
 *              (all three of `format`; MXFP8: hidden and inter multiples of 32)
 *   out        [tokens, hidden] fp32 or bf16, 16-byte aligned
 *   workspace  fp8q_moe_experts_workspace bytes, 16-byte aligned
 * topk 1 .. FP8Q_MAX_TOPK, experts 1 .. FP8Q_MAX_EXPERTS, tokens * topk up to
 * FP8Q_EXPERTS_MAX_PAIRS, hidden and inter up to FP8Q_EXPERTS_MAX_SIZE.
 */
FP8Q_API size_t fp8q_moe_experts_workspace(size_t tokens, int topk, int experts, size_t hidden,
                                           size_t inter, fp8q_out_dtype out_dtype);
FP8Q_API fp8q_status fp8q_moe_experts(const void *x_bf16, const void *ids, int id_bytes,
                                      const float *weights, fp8q_row_format format,
                                      const fp8q_expert_matrix *gate, const fp8q_expert_matrix *up,
                                      const fp8q_expert_matrix *down, size_t tokens, int topk,
                                      int experts, size_t hidden, size_t inter, void *out,
                                      fp8q_out_dtype out_dtype, void *workspace,
                                      size_t workspace_bytes, void *stream);

typedef enum {
    FP8Q_GRAD_F32 = 0,
    FP8Q_GRAD_BF16 = 1,
    FP8Q_GRAD_E4M3 = 2,      /* codes with fp32 scales                       */
    FP8Q_GRAD_E5M2 = 3
} fp8q_grad_dtype;

/*
 * One gradient of a list: `count` values, aligned to their own size.  Codes
 * carry one fp32 scale per 128 of them (scale_count = ceil(count / 128), as
 * fp8q_quantize and fp8q_dequant_reduce_requantize write them) or one for all
 * (scale_count = 1, as fp8q_quantize_tensorwise does); otherwise scales is NULL
 * and scale_count 0.
 */
typedef struct {
    void *data;
    float *scales;
    size_t count;
    size_t scale_count;
    int dtype;               /* fp8q_grad_dtype                              */
} fp8q_grad;

/*
 * Sum of squares over all values of a list of gradients, in fp64: of the
 * values themselves, or of fl32(code * scale).  Neither overflows nor loses
 * small ones for any fp32 values; inf and NaN go into the sum.  Summed in an
 * order that the sizes fix: the same call gives the same bits.  Its square
 * root is the global norm; ranks that hold different gradients add their sums
 * up.  Gradients of no values, and an empty list (sum 0), are allowed.
 *   grads       n structs in host memory
 *   sumsq_out   [1] fp64
 *   workspace   fp8q_grad_sumsq_workspace bytes (NULL where that is 0), 16-byte
 *               aligned
 */
FP8Q_API size_t fp8q_grad_sumsq_workspace(const fp8q_grad *grads, size_t n);
FP8Q_API fp8q_status fp8q_grad_sumsq(const fp8q_grad *grads, size_t n, double *sumsq_out,
                                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * Clips gradients to a largest global norm, in place: with
 *   norm = sqrt(sumsq),   c = min(1, max_norm / (norm + eps))   (in fp64)
 * every value is multiplied by c, rounded to fp32, in fp32, and rounded once to
 * its type; of codes the scales are, and the codes stay.  With c == 1 nothing is
 * written.  A NaN norm makes all of them NaN (codes: their scales), as 0 / 0 does
 * (eps, max_norm and the norm all 0); an infinite one makes
 * finite values 0 and infinite ones NaN; unless max_norm is infinite: then
 * nothing is ever written.
 *   grads      n structs in host memory, none overlapping another
 *   sumsq      [1] fp64, of the whole gradient (all ranks)
 *   max_norm   >= 0;  eps  finite, >= 0
 *   norm_out   [1] fp32
 */
FP8Q_API fp8q_status fp8q_grad_clip(const fp8q_grad *grads, size_t n, const double *sumsq,
                                    double max_norm, double eps, float *norm_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_MODEL_H */
