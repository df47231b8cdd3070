// layer_api.hip -- the C ABI declared in include/fp8q_layer.h: host-side
// validation and dispatch to the gfx950 kernels.
//
// As in api.hip, every check runs before anything is enqueued (enums, counts
// and sizes, null pointers, alignment, overlap), and a failed check returns
// its status with no launch.
#include <stdint.h>

#include <initializer_list>

#include <hip/hip_runtime.h>

#include "fp8q_layer.h"
#include "layer_launch.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A byte range of a call.  A null pointer or a size of zero is no range.
struct Range {
  const void *p;
  uint64_t n;
};

bool overlaps(const Range &a, const Range &b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

bool overlaps_any(const Range &out, std::initializer_list<Range> others) {
  for (const Range &r : others)
    if (overlaps(out, r)) return true;
  return false;
}

// `out` overlaps `in` without being the very same range (an update in place).
bool overlaps_shifted(const Range &out, const Range &in) {
  return out.p != in.p && overlaps(out, in);
}

bool valid_weight(fp8q_weight_dtype d) { return d == FP8Q_WEIGHT_F32 || d == FP8Q_WEIGHT_BF16; }

// rows * hidden within the element limit (both above zero).
bool size_ok(uint64_t rows, uint64_t hidden) {
  return rows <= FP8Q_MAX_ELEMS && hidden <= FP8Q_MAX_ELEMS && rows <= FP8Q_MAX_ELEMS / hidden;
}

bool pairs_ok(size_t tokens, int topk) {
  return topk >= 1 && topk <= FP8Q_MAX_TOPK && tokens <= FP8Q_MAX_PAIRS / (size_t)topk;
}

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

fp8q_status from_hip(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_ERR_HIP; }

fp8q_status norm_quantize(int out, const void *x, const void *residual, const void *weight,
                          fp8q_weight_dtype weight_dtype, float eps, size_t rows, size_t hidden,
                          void *h_out, void *y_out, void *q_out, void *scales_out,
                          uint64_t scale_bytes, uintptr_t scale_align, float *rstd_out,
                          void *stream) {
  if (!valid_weight(weight_dtype) || !(eps >= 0.0f && eps <= 3.0e38f)) return FP8Q_ERR_ARG;
  if (h_out && !residual) return FP8Q_ERR_ARG;
  if (rows == 0 || hidden == 0) return FP8Q_OK;
  if (hidden > FP8Q_NORM_MAX_HIDDEN || !size_ok(rows, hidden)) return FP8Q_ERR_ARG;
  if (!x || !weight || !q_out || !scales_out) return FP8Q_ERR_NULL;
  for (const void *p : {x, residual, weight, (const void *)h_out, (const void *)y_out,
                        (const void *)q_out})
    if (!aligned(p, 16)) return FP8Q_ERR_ALIGN;
  if (!aligned(scales_out, scale_align) || !aligned(rstd_out, 4)) return FP8Q_ERR_ALIGN;
  const uint64_t n = (uint64_t)rows * hidden;
  const Range xr{x, 2 * n}, rr{residual, 2 * n},
      wr{weight, hidden * (weight_dtype == FP8Q_WEIGHT_F32 ? 4u : 2u)}, hr{h_out, 2 * n},
      yr{y_out, 2 * n}, qr{q_out, n}, sr{scales_out, scale_bytes}, tr{rstd_out, 4 * (uint64_t)rows};
  if (overlaps_shifted(hr, xr) || overlaps_shifted(hr, rr) || overlaps_any(hr, {wr, yr, qr, sr, tr}) ||
      overlaps_any(yr, {xr, rr, wr, qr, sr, tr}) || overlaps_any(qr, {xr, rr, wr, sr, tr}) ||
      overlaps_any(sr, {xr, rr, wr, tr}) || overlaps_any(tr, {xr, rr, wr}))
    return FP8Q_ERR_OVERLAP;
  const fp8q::NormForward a{x, residual, weight, weight_dtype == FP8Q_WEIGHT_BF16, eps,
                            (uint32_t)hidden, 1.0f / (float)hidden, rows, h_out, y_out, q_out,
                            scales_out, rstd_out};
  return from_hip(fp8q::launch_rms_norm(out, a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

fp8q_status fp8q_rms_norm_quantize(const void *x_bf16, const void *residual_bf16,
                                   const void *weight, fp8q_weight_dtype weight_dtype, float eps,
                                   size_t rows, size_t hidden, fp8q_format fmt, void *h_out,
                                   void *y_out, void *q_out, float *scales_out, float *rstd_out,
                                   void *stream) {
  if (fmt != FP8Q_E4M3 && fmt != FP8Q_E5M2) return FP8Q_ERR_ARG;
  const uint64_t scale_bytes = 4 * (uint64_t)rows * ceil_div(hidden, FP8Q_BLOCK);
  return norm_quantize(fmt == FP8Q_E4M3 ? 0 : 1, x_bf16, residual_bf16, weight, weight_dtype, eps,
                       rows, hidden, h_out, y_out, q_out, scales_out, scale_bytes, 4, rstd_out,
                       stream);
}

fp8q_status mx8_rms_norm_quantize(const void *x_bf16, const void *residual_bf16,
                                  const void *weight, fp8q_weight_dtype weight_dtype, float eps,
                                  size_t rows, size_t hidden, void *h_out, void *y_out,
                                  void *q_out, void *e8m0_out, float *rstd_out, void *stream) {
  if (hidden % FP8Q_MX_BLOCK != 0) return FP8Q_ERR_ARG;
  const uint64_t scale_bytes = (uint64_t)rows * (hidden / FP8Q_MX_BLOCK);
  return norm_quantize(2, x_bf16, residual_bf16, weight, weight_dtype, eps, rows, hidden, h_out,
                       y_out, q_out, e8m0_out, scale_bytes, 1, rstd_out, stream);
}

size_t fp8q_rms_norm_backward_workspace(size_t rows, size_t hidden) {
  if (rows == 0 || hidden == 0 || hidden > FP8Q_NORM_MAX_HIDDEN || !size_ok(rows, hidden)) return 0;
  return (size_t)fp8q::norm_backward_workspace(rows, (uint32_t)hidden);
}

fp8q_status fp8q_rms_norm_backward(const void *dy_bf16, const void *h_bf16, const void *weight,
                                   fp8q_weight_dtype weight_dtype, const float *rstd,
                                   const void *dh_bf16, size_t rows, size_t hidden, void *dx_out,
                                   float *dweight_out, void *workspace, size_t workspace_bytes,
                                   void *stream) {
  if (!valid_weight(weight_dtype)) return FP8Q_ERR_ARG;
  if (hidden == 0) return FP8Q_OK;
  if (hidden > FP8Q_NORM_MAX_HIDDEN || !size_ok(rows, hidden)) return FP8Q_ERR_ARG;
  const uint64_t need = fp8q_rms_norm_backward_workspace(rows, hidden);
  if (workspace_bytes < need) return FP8Q_ERR_ARG;
  if (!dweight_out) return FP8Q_ERR_NULL;
  if (rows && (!dy_bf16 || !h_bf16 || !weight || !rstd || !dx_out || (need && !workspace)))
    return FP8Q_ERR_NULL;
  for (const void *p : {dy_bf16, h_bf16, weight, dh_bf16, (const void *)dx_out,
                        (const void *)workspace})
    if (!aligned(p, 16)) return FP8Q_ERR_ALIGN;
  if (!aligned(rstd, 4) || !aligned(dweight_out, 4)) return FP8Q_ERR_ALIGN;
  const uint64_t n = (uint64_t)rows * hidden;
  const Range dyr{dy_bf16, 2 * n}, hr{h_bf16, 2 * n},
      wr{weight, hidden * (weight_dtype == FP8Q_WEIGHT_F32 ? 4u : 2u)},
      tr{rstd, 4 * (uint64_t)rows}, dhr{dh_bf16, 2 * n}, dxr{dx_out, 2 * n},
      dwr{dweight_out, 4 * (uint64_t)hidden}, sr{workspace, need};
  if (overlaps_shifted(dxr, dyr) || overlaps_shifted(dxr, dhr) ||
      overlaps_any(dxr, {hr, wr, tr, dwr, sr}) || overlaps_any(dwr, {dyr, hr, wr, tr, dhr, sr}) ||
      overlaps_any(sr, {dyr, hr, wr, tr, dhr}))
    return FP8Q_ERR_OVERLAP;
  const fp8q::NormBackward a{dy_bf16, h_bf16, weight, weight_dtype == FP8Q_WEIGHT_BF16, rstd,
                             dh_bf16, (uint32_t)hidden, 1.0f / (float)hidden, rows, dx_out,
                             dweight_out, static_cast<float *>(workspace)};
  return from_hip(fp8q::launch_rms_norm_backward(a, static_cast<hipStream_t>(stream)));
}

size_t fp8q_moe_sort_workspace(size_t tokens, int topk, int experts) {
  if (!pairs_ok(tokens, topk) || experts < 1 || experts > FP8Q_MAX_EXPERTS) return 0;
  return (size_t)fp8q::moe_sort_workspace((uint32_t)(tokens * topk), (uint32_t)experts);
}

fp8q_status fp8q_moe_sort(const void *ids, int id_bytes, size_t tokens, int topk, int experts,
                          int *slots_out, int *pairs_out, int *offsets_out, void *workspace,
                          size_t workspace_bytes, void *stream) {
  if (id_bytes != 4 && id_bytes != 8) return FP8Q_ERR_ARG;
  if (!pairs_ok(tokens, topk) || experts < 1 || experts > FP8Q_MAX_EXPERTS) return FP8Q_ERR_ARG;
  const uint64_t n = (uint64_t)tokens * topk;
  const uint64_t need = fp8q_moe_sort_workspace(tokens, topk, experts);
  if (workspace_bytes < need) return FP8Q_ERR_ARG;
  if (!offsets_out) return FP8Q_ERR_NULL;
  if (n && (!ids || !slots_out || !pairs_out || (need && !workspace))) return FP8Q_ERR_NULL;
  if (!aligned(ids, (uintptr_t)id_bytes) || !aligned(slots_out, 4) || !aligned(pairs_out, 4) ||
      !aligned(offsets_out, 4) || !aligned(workspace, 16))
    return FP8Q_ERR_ALIGN;
  const Range ir{ids, n * (uint64_t)id_bytes}, sr{slots_out, 4 * n}, pr{pairs_out, 4 * n},
      fr{offsets_out, 4 * ((uint64_t)experts + 1)}, wr{workspace, need};
  if (overlaps_any(sr, {ir, pr, fr, wr}) || overlaps_any(pr, {ir, fr, wr}) ||
      overlaps_any(fr, {ir, wr}) || overlaps(wr, ir))
    return FP8Q_ERR_OVERLAP;
  const fp8q::MoeSort a{ids, id_bytes == 8, (uint32_t)n, (uint32_t)experts, slots_out, pairs_out,
                        offsets_out, static_cast<uint32_t *>(workspace)};
  return from_hip(fp8q::launch_moe_sort(a, static_cast<hipStream_t>(stream)));
}

fp8q_status fp8q_moe_permute(const void *src, size_t row_bytes, const void *src_scales,
                             size_t scale_row_bytes, const int *slots, size_t tokens, int topk,
                             size_t dst_rows, void *dst, void *dst_scales, void *stream) {
  if (!pairs_ok(tokens, topk) || dst_rows > FP8Q_MAX_PAIRS) return FP8Q_ERR_ARG;
  if (row_bytes == 0 && scale_row_bytes != 0) return FP8Q_ERR_ARG;
  if (tokens == 0 || dst_rows == 0 || row_bytes == 0) return FP8Q_OK;
  for (const size_t bytes : {row_bytes, scale_row_bytes})
    if (bytes > 4 * FP8Q_MAX_HIDDEN || (bytes && (!size_ok(tokens, bytes) || !size_ok(dst_rows, bytes))))
      return FP8Q_ERR_ARG;
  if (!src || !slots || !dst) return FP8Q_ERR_NULL;
  if (scale_row_bytes && (!src_scales || !dst_scales)) return FP8Q_ERR_NULL;
  if (!aligned(src, 16) || !aligned(dst, 16) || !aligned(slots, 4)) return FP8Q_ERR_ALIGN;
  const Range xr{src, (uint64_t)tokens * row_bytes}, xs{src_scales, (uint64_t)tokens * scale_row_bytes},
      sl{slots, 4 * (uint64_t)tokens * topk}, dr{dst, (uint64_t)dst_rows * row_bytes},
      ds{dst_scales, (uint64_t)dst_rows * scale_row_bytes};
  if (overlaps_any(dr, {xr, xs, sl, ds}) || overlaps_any(ds, {xr, xs, sl}))
    return FP8Q_ERR_OVERLAP;
  const fp8q::MoePermute a{src, src_scales, row_bytes, scale_row_bytes, slots, (uint32_t)tokens,
                           (uint32_t)topk, dst_rows, dst, dst_scales};
  return from_hip(fp8q::launch_moe_permute(a, static_cast<hipStream_t>(stream)));
}

fp8q_status fp8q_moe_combine(const void *rows, fp8q_row_format format, const void *scales,
                             const int *slots, const float *weights, size_t tokens, int topk,
                             size_t row_count, size_t hidden, void *out, fp8q_out_dtype out_dtype,
                             void *stream) {
  if (format != FP8Q_ROWS_BF16 && format != FP8Q_ROWS_E4M3 && format != FP8Q_ROWS_E5M2 &&
      format != FP8Q_ROWS_MX8)
    return FP8Q_ERR_ARG;
  if (out_dtype != FP8Q_OUT_F32 && out_dtype != FP8Q_OUT_BF16) return FP8Q_ERR_ARG;
  if (!pairs_ok(tokens, topk) || row_count > FP8Q_MAX_PAIRS) return FP8Q_ERR_ARG;
  if (format == FP8Q_ROWS_MX8 && hidden % FP8Q_MX_BLOCK != 0) return FP8Q_ERR_ARG;
  if (tokens == 0 || hidden == 0) return FP8Q_OK;
  if (hidden > FP8Q_MAX_HIDDEN || !size_ok(tokens, hidden) || !size_ok(row_count, hidden)) return FP8Q_ERR_ARG;
  const bool coded = format != FP8Q_ROWS_BF16;
  if (!slots || !out || (row_count && (!rows || (coded && !scales)))) return FP8Q_ERR_NULL;
  if (!aligned(rows, 16) || !aligned(out, 16) || !aligned(slots, 4) || !aligned(weights, 4) ||
      (coded && !aligned(scales, format == FP8Q_ROWS_MX8 ? 1 : 4)))
    return FP8Q_ERR_ALIGN;
  const uint64_t rn = (uint64_t)row_count * hidden, pairs = (uint64_t)tokens * topk;
  const uint64_t sb = !coded ? 0
                      : format == FP8Q_ROWS_MX8
                          ? (uint64_t)row_count * (hidden / FP8Q_MX_BLOCK)
                          : 4 * (uint64_t)row_count * ceil_div(hidden, FP8Q_BLOCK);
  const Range outr{out, (uint64_t)tokens * hidden * (out_dtype == FP8Q_OUT_F32 ? 4 : 2)};
  if (overlaps_any(outr, {Range{rows, coded ? rn : 2 * rn}, Range{scales, sb},
                          Range{slots, 4 * pairs}, Range{weights, 4 * pairs}}))
    return FP8Q_ERR_OVERLAP;
  const fp8q::MoeCombine a{rows, coded ? scales : nullptr, slots, weights, (uint32_t)tokens,
                           (uint32_t)topk, row_count, hidden, out, out_dtype == FP8Q_OUT_BF16};
  return from_hip(fp8q::launch_moe_combine((int)format, a, static_cast<hipStream_t>(stream)));
}

fp8q_status fp8q_moe_combine_backward(const void *dy_bf16, const void *rows_bf16,
                                      const int *slots, const float *weights, size_t tokens,
                                      int topk, size_t row_count, size_t hidden, void *drows_out,
                                      float *dweights_out, void *stream) {
  if (!pairs_ok(tokens, topk) || row_count > FP8Q_MAX_PAIRS) return FP8Q_ERR_ARG;
  if (tokens == 0) return FP8Q_OK;
  if (hidden > FP8Q_MAX_HIDDEN) return FP8Q_ERR_ARG;
  if (hidden && (!size_ok(tokens, hidden) || !size_ok(row_count, hidden))) return FP8Q_ERR_ARG;
  if (!slots || !weights || !dweights_out) return FP8Q_ERR_NULL;
  if (hidden && (!dy_bf16 || (row_count && (!rows_bf16 || !drows_out)))) return FP8Q_ERR_NULL;
  if (!aligned(dy_bf16, 16) || !aligned(rows_bf16, 16) || !aligned(drows_out, 16) ||
      !aligned(slots, 4) || !aligned(weights, 4) || !aligned(dweights_out, 4))
    return FP8Q_ERR_ALIGN;
  const uint64_t pairs = (uint64_t)tokens * topk, rn = (uint64_t)row_count * hidden;
  const Range yr{dy_bf16, 2 * (uint64_t)tokens * hidden}, rr{rows_bf16, 2 * rn},
      sl{slots, 4 * pairs}, wr{weights, 4 * pairs}, dr{drows_out, 2 * rn},
      dw{dweights_out, 4 * pairs};
  if (overlaps_any(dr, {yr, rr, sl, wr, dw}) || overlaps_any(dw, {yr, rr, sl, wr}))
    return FP8Q_ERR_OVERLAP;
  const fp8q::MoeCombineBackward a{dy_bf16, rows_bf16, slots, weights, (uint32_t)tokens,
                                   (uint32_t)topk, row_count, hidden, drows_out, dweights_out};
  return from_hip(fp8q::launch_moe_combine_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
