// model_api.hip -- the C ABI declared in include/fp8q_model.h: host-side
// validation and dispatch to the gfx950 kernels.
//
// As in api.hip, every check runs before anything is enqueued (enums, counts
// and sizes, null pointers, alignment, overlap), and a failed check returns
// its status with no launch.
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <stdexcept>
#include <vector>

#include <hip/hip_runtime.h>

#include "fp8q_model.h"
#include "model_launch.h"

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

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

fp8q_status from_hip(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_ERR_HIP; }

bool route_sizes_ok(size_t tokens, int experts, int topk) {
  return experts >= 1 && experts <= FP8Q_MAX_EXPERTS && topk >= 1 && topk <= FP8Q_MAX_TOPK && topk <= experts &&
         tokens <= FP8Q_MAX_PAIRS / (size_t)topk;
}

bool valid_logits(fp8q_logits_dtype d) { return d == FP8Q_LOGITS_F32 || d == FP8Q_LOGITS_BF16; }

// The bytes of an expert matrix's rows and scales.
struct Extent {
  Range rows, scales;
};
Extent extent_of(const fp8q_expert_matrix &m, fp8q_row_format format, int experts, size_t rows, size_t width) {
  const uint64_t count = (uint64_t)(experts - 1) * m.expert_rows + rows;
  const uint64_t scales = format == FP8Q_ROWS_BF16  ? 0
                          : format == FP8Q_ROWS_MX8 ? count * (width / FP8Q_MX_BLOCK)
                                                    : 4 * count * ceil_div(width, FP8Q_BLOCK);
  return {{m.rows, count * width * (format == FP8Q_ROWS_BF16 ? 2 : 1)}, {m.scales, scales}};
}

bool experts_sizes_ok(size_t tokens, int topk, int experts, size_t hidden, size_t inter, fp8q_out_dtype out_dtype) {
  return experts >= 1 && experts <= FP8Q_MAX_EXPERTS && topk >= 1 && topk <= FP8Q_MAX_TOPK &&
         tokens <= FP8Q_EXPERTS_MAX_PAIRS / (size_t)topk &&
         hidden <= FP8Q_EXPERTS_MAX_SIZE && inter <= FP8Q_EXPERTS_MAX_SIZE &&
         (out_dtype == FP8Q_OUT_F32 || out_dtype == FP8Q_OUT_BF16);
}

// A gradient as the launchers take it, or the status of one that is not valid.
fp8q_status check_grad(const fp8q_grad &g, fp8q::Grad &out) {
  if (g.dtype < FP8Q_GRAD_F32 || g.dtype > FP8Q_GRAD_E5M2) return FP8Q_ERR_ARG;
  const bool coded = g.dtype == FP8Q_GRAD_E4M3 || g.dtype == FP8Q_GRAD_E5M2;
  if (g.count > FP8Q_MAX_ELEMS) return FP8Q_ERR_ARG;
  out = {g.data, nullptr, g.count, (int)g.dtype, false};
  if (g.count == 0) return FP8Q_OK;
  if (!coded && (g.scales || g.scale_count)) return FP8Q_ERR_ARG;
  if (coded && g.scale_count != 1 && g.scale_count != ceil_div(g.count, FP8Q_BLOCK)) return FP8Q_ERR_ARG;
  if (!g.data || (coded && !g.scales)) return FP8Q_ERR_NULL;
  if (!aligned(g.data, g.dtype == FP8Q_GRAD_F32 ? 4 : g.dtype == FP8Q_GRAD_BF16 ? 2 : 1) || !aligned(g.scales, 4))
    return FP8Q_ERR_ALIGN;
  out.scales = g.scales;
  out.one_scale = coded && g.scale_count == 1;
  return FP8Q_OK;
}

Range data_of(const fp8q::Grad &g) { return {g.data, g.count * (g.kind == 0 ? 4 : g.kind == 1 ? 2 : 1)}; }

// Every gradient checked.
fp8q_status check_grads(const fp8q_grad *grads, size_t n, std::vector<fp8q::Grad> &list) {
  if (n && !grads) return FP8Q_ERR_NULL;
  list.resize(n);
  for (size_t i = 0; i < n; ++i) {
    const fp8q_status st = check_grad(grads[i], list[i]);
    if (st != FP8Q_OK) return st;
  }
  return FP8Q_OK;
}

// One of the gradients, or its scales, overlaps one of the ranges.
bool any_overlaps(const fp8q_grad *grads, const std::vector<fp8q::Grad> &list, std::initializer_list<Range> ranges) {
  for (size_t i = 0; i < list.size(); ++i)
    if (overlaps_any(data_of(list[i]), ranges) ||
        overlaps_any({list[i].scales, 4 * (uint64_t)grads[i].scale_count}, ranges))
      return true;
  return false;
}

}  // namespace

extern "C" {

fp8q_status fp8q_moe_route(const void *logits, fp8q_logits_dtype dtype, size_t tokens, int experts, int topk,
                           int normalize, float *weights_out, int *ids_out, void *stream) {
  if (!valid_logits(dtype) || !route_sizes_ok(tokens, experts, topk)) return FP8Q_ERR_ARG;
  if (tokens == 0) return FP8Q_OK;
  if (!logits || !weights_out || !ids_out) return FP8Q_ERR_NULL;
  if (!aligned(logits, 16) || !aligned(weights_out, 4) || !aligned(ids_out, 4)) return FP8Q_ERR_ALIGN;
  const uint64_t pairs = (uint64_t)tokens * topk;
  const Range lr{logits, (uint64_t)tokens * experts * (dtype == FP8Q_LOGITS_F32 ? 4 : 2)}, wr{weights_out, 4 * pairs},
      ir{ids_out, 4 * pairs};
  if (overlaps_any(wr, {lr, ir}) || overlaps(ir, lr)) return FP8Q_ERR_OVERLAP;
  const fp8q::MoeRoute a{logits, dtype == FP8Q_LOGITS_BF16, tokens, (uint32_t)experts, (uint32_t)topk,
                         normalize != 0, weights_out, ids_out};
  return from_hip(fp8q::launch_moe_route(a, static_cast<hipStream_t>(stream)));
}

fp8q_status fp8q_moe_route_backward(const float *dweights, const void *logits, fp8q_logits_dtype dtype,
                                    const float *weights, const int *ids, size_t tokens, int experts, int topk,
                                    int normalize, void *dlogits_out, void *stream) {
  if (!valid_logits(dtype) || !route_sizes_ok(tokens, experts, topk)) return FP8Q_ERR_ARG;
  if (tokens == 0) return FP8Q_OK;
  if (!dweights || !weights || !ids || !dlogits_out || (!normalize && !logits)) return FP8Q_ERR_NULL;
  if (!aligned(logits, 16) || !aligned(dlogits_out, 16) || !aligned(dweights, 4) || !aligned(weights, 4) ||
      !aligned(ids, 4))
    return FP8Q_ERR_ALIGN;
  const uint64_t pairs = (uint64_t)tokens * topk;
  const Range out{dlogits_out, (uint64_t)tokens * experts * (dtype == FP8Q_LOGITS_F32 ? 4 : 2)};
  if ((logits != dlogits_out && overlaps(out, Range{logits, out.n})) ||
      overlaps_any(out, {Range{dweights, 4 * pairs}, Range{weights, 4 * pairs}, Range{ids, 4 * pairs}}))
    return FP8Q_ERR_OVERLAP;
  const fp8q::MoeRouteBackward a{dweights, logits, dtype == FP8Q_LOGITS_BF16, weights, ids, tokens,
                                 (uint32_t)experts, (uint32_t)topk, normalize != 0, dlogits_out};
  return from_hip(fp8q::launch_moe_route_backward(a, static_cast<hipStream_t>(stream)));
}

size_t fp8q_moe_experts_workspace(size_t tokens, int topk, int experts, size_t hidden, size_t inter,
                                  fp8q_out_dtype out_dtype) {
  if (!experts_sizes_ok(tokens, topk, experts, hidden, inter, out_dtype) || tokens == 0) return 0;
  return (size_t)fp8q::moe_experts_workspace((uint32_t)(tokens * topk), (uint32_t)experts, (uint32_t)hidden,
                                             (uint32_t)inter,
                                             out_dtype == FP8Q_OUT_BF16);
}

fp8q_status fp8q_moe_experts(const void *x_bf16, const void *ids, int id_bytes, const float *weights,
                             fp8q_row_format format, const fp8q_expert_matrix *gate, const fp8q_expert_matrix *up,
                             const fp8q_expert_matrix *down, size_t tokens, int topk, int experts, size_t hidden,
                             size_t inter, void *out, fp8q_out_dtype out_dtype, void *workspace,
                             size_t workspace_bytes, void *stream) {
  if (format != FP8Q_ROWS_BF16 && format != FP8Q_ROWS_E4M3 && format != FP8Q_ROWS_E5M2 && format != FP8Q_ROWS_MX8)
    return FP8Q_ERR_ARG;
  if (id_bytes != 4 && id_bytes != 8) return FP8Q_ERR_ARG;
  if (!experts_sizes_ok(tokens, topk, experts, hidden, inter, out_dtype)) return FP8Q_ERR_ARG;
  if (format == FP8Q_ROWS_MX8 && (hidden % FP8Q_MX_BLOCK || inter % FP8Q_MX_BLOCK)) return FP8Q_ERR_ARG;
  if (tokens == 0 || hidden == 0) return FP8Q_OK;
  const uint64_t need = fp8q_moe_experts_workspace(tokens, topk, experts, hidden, inter, out_dtype);
  if (workspace_bytes < need) return FP8Q_ERR_ARG;
  if (!gate || !up || !down || !x_bf16 || !ids || !weights || !out || (need && !workspace)) return FP8Q_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(ids, (uintptr_t)id_bytes) ||
      !aligned(weights, 4))
    return FP8Q_ERR_ALIGN;
  const uint64_t pairs = (uint64_t)tokens * topk;
  const Range xr{x_bf16, 2 * (uint64_t)tokens * hidden}, ir{ids, pairs * (uint64_t)id_bytes}, wr{weights, 4 * pairs},
      outr{out, (uint64_t)tokens * hidden * (out_dtype == FP8Q_OUT_F32 ? 4 : 2)}, sr{workspace, need};
  if (overlaps_any(outr, {xr, ir, wr, sr}) || overlaps_any(sr, {xr, ir, wr})) return FP8Q_ERR_OVERLAP;
  const fp8q_expert_matrix *all[3] = {gate, up, down};
  if (inter) {
    for (int i = 0; i < 3; ++i) {
      const fp8q_expert_matrix &m = *all[i];
      const size_t rows = i == 2 ? hidden : inter, width = i == 2 ? inter : hidden;
      if (m.expert_rows < rows || m.expert_rows > ((size_t)1 << 32)) return FP8Q_ERR_ARG;
      if ((format == FP8Q_ROWS_BF16) != !m.scales) return m.scales ? FP8Q_ERR_ARG : FP8Q_ERR_NULL;
      if (!m.rows) return FP8Q_ERR_NULL;
      if ((format == FP8Q_ROWS_BF16 && !aligned(m.rows, 2)) ||
          ((format == FP8Q_ROWS_E4M3 || format == FP8Q_ROWS_E5M2) && !aligned(m.scales, 4)))
        return FP8Q_ERR_ALIGN;
      const Extent x = extent_of(m, format, experts, rows, width);
      if (overlaps_any(outr, {x.rows, x.scales}) || overlaps_any(sr, {x.rows, x.scales})) return FP8Q_ERR_OVERLAP;
    }
  }
  const auto matrix = [](const fp8q_expert_matrix &m) {
    return fp8q::ExpertMatrix{static_cast<const uint8_t *>(m.rows), static_cast<const uint8_t *>(m.scales),
                              m.expert_rows};
  };
  const fp8q::MoeExperts a{static_cast<const uint16_t *>(x_bf16), ids, id_bytes == 8, weights, matrix(*gate),
                           matrix(*up), matrix(*down), (uint32_t)tokens, (uint32_t)topk, (uint32_t)experts,
                           (uint32_t)hidden, (uint32_t)inter, out, out_dtype == FP8Q_OUT_BF16,
                           static_cast<uint16_t *>(workspace)};
  return from_hip(fp8q::launch_moe_experts((int)format, a, static_cast<hipStream_t>(stream)));
}

// The lists below are copied into the launchers' form.  Where memory for that
// runs out nothing is enqueued, as for any other failed check.

size_t fp8q_grad_sumsq_workspace(const fp8q_grad *grads, size_t n) try {
  std::vector<fp8q::Grad> list;
  if (check_grads(grads, n, list) != FP8Q_OK) return 0;
  return (size_t)fp8q::grad_sumsq_workspace(list.data(), n);
} catch (const std::bad_alloc &) {
  return 0;
} catch (const std::length_error &) {
  return 0;
}

fp8q_status fp8q_grad_sumsq(const fp8q_grad *grads, size_t n, double *sumsq_out, void *workspace,
                            size_t workspace_bytes, void *stream) try {
  std::vector<fp8q::Grad> list;
  if (!sumsq_out) return FP8Q_ERR_NULL;
  if (!aligned(sumsq_out, 8) || !aligned(workspace, 16)) return FP8Q_ERR_ALIGN;
  fp8q_status st = check_grads(grads, n, list);
  if (st != FP8Q_OK) return st;
  const uint64_t need = fp8q::grad_sumsq_workspace(list.data(), n);
  if (workspace_bytes < need) return FP8Q_ERR_ARG;
  if (need && !workspace) return FP8Q_ERR_NULL;
  const Range out{sumsq_out, 8}, scratch{workspace, need};
  if (overlaps(out, scratch) || any_overlaps(grads, list, {out, scratch})) return FP8Q_ERR_OVERLAP;
  return from_hip(fp8q::launch_grad_sumsq(list.data(), n, sumsq_out, static_cast<double *>(workspace),
                                          static_cast<hipStream_t>(stream)));
} catch (const std::bad_alloc &) {
  return FP8Q_ERR_ARG;
} catch (const std::length_error &) {
  return FP8Q_ERR_ARG;
}

fp8q_status fp8q_grad_clip(const fp8q_grad *grads, size_t n, const double *sumsq, double max_norm, double eps,
                           float *norm_out, void *stream) try {
  std::vector<fp8q::Grad> list;
  if (!(max_norm >= 0.0) || !(eps >= 0.0 && eps <= 1.0e308)) return FP8Q_ERR_ARG;
  if (!sumsq || !norm_out) return FP8Q_ERR_NULL;
  if (!aligned(sumsq, 8) || !aligned(norm_out, 4)) return FP8Q_ERR_ALIGN;
  const Range in{sumsq, 8}, out{norm_out, 4};
  if (overlaps(in, out)) return FP8Q_ERR_OVERLAP;
  const fp8q_status st = check_grads(grads, n, list);
  if (st != FP8Q_OK) return st;
  if (any_overlaps(grads, list, {in, out})) return FP8Q_ERR_OVERLAP;
  // of codes, the scales are what is scaled
  for (size_t i = 0; i < n; ++i)
    if (list[i].kind >= FP8Q_GRAD_E4M3)
      list[i] = {grads[i].scales, nullptr, grads[i].count ? grads[i].scale_count : 0, FP8Q_GRAD_F32, false};
  // what is written once must not be written twice
  std::vector<Range> written;
  written.reserve(n);
  for (const fp8q::Grad &g : list)
    if (g.count) written.push_back(data_of(g));
  const auto before = [](const Range &a, const Range &b) { return a.p < b.p; };
  if (!std::is_sorted(written.begin(), written.end(), before)) std::sort(written.begin(), written.end(), before);
  for (size_t i = 1; i < written.size(); ++i)
    if (overlaps(written[i - 1], written[i])) return FP8Q_ERR_OVERLAP;
  return from_hip(fp8q::launch_grad_clip(list.data(), n, sumsq, max_norm, eps, norm_out,
                                         static_cast<hipStream_t>(stream)));
} catch (const std::bad_alloc &) {
  return FP8Q_ERR_ARG;
} catch (const std::length_error &) {
  return FP8Q_ERR_ARG;
}

}  // extern "C"
