// layer_stub_launchers.cpp -- host-only stand-ins for the layer operators'
// launchers, so that their C-ABI layer (csrc/layer_api.hip, compiled host-only
// with g++) can run under AddressSanitizer and UndefinedBehaviorSanitizer on a
// machine without a GPU.
//
// Each stub enqueues nothing.  It checks what the real launchers assume of a
// validated call (layer_launch.h) and records the call; a broken assumption
// returns hipErrorInvalidValue, which the ABI reports as FP8Q_ERR_HIP.
#include <stdint.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "fp8q_layer.h"
#include "layer_launch.h"

namespace {

struct Record {
  long calls;
  char last[32];
  uint64_t a, b;
};
Record g_rec = {0, {0}, 0, 0};

bool al(const void *p, uintptr_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
bool al0(const void *p, uintptr_t a) { return !p || al(p, a); }

bool apart(const void *a, uint64_t na, const void *b, uint64_t nb) {
  if (!a || !b || !na || !nb) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x + na <= y || y + nb <= x;
}

hipError_t record(const char *name, uint64_t a, uint64_t b) {
  ++g_rec.calls;
  strncpy(g_rec.last, name, sizeof(g_rec.last) - 1);
  g_rec.a = a;
  g_rec.b = b;
  return hipSuccess;
}

bool topk_ok(uint32_t topk) { return topk >= 1 && topk <= FP8Q_MAX_TOPK; }

}  // namespace

namespace fp8q {

hipError_t launch_rms_norm(int out, const NormForward &a, hipStream_t) {
  const uint64_t n = a.rows * a.hidden;
  const bool mx = out == 2;
  const uint64_t sb = mx ? n / 32 : 4 * a.rows * ((a.hidden + 127) / 128);
  const bool ok = out >= 0 && out <= 2 && a.rows && a.hidden && a.hidden <= FP8Q_NORM_MAX_HIDDEN &&
                  (!mx || a.hidden % 32 == 0) && a.inv_hidden == 1.0f / (float)a.hidden &&
                  a.eps >= 0.0f && al(a.x, 16) && al0(a.residual, 16) && al(a.weight, 16) &&
                  al0(a.h_out, 16) && al0(a.y_out, 16) && al(a.q_out, 16) &&
                  al(a.scales_out, mx ? 1 : 4) && al0(a.rstd_out, 4) && (a.residual || !a.h_out) &&
                  (a.h_out == a.x || apart(a.h_out, 2 * n, a.x, 2 * n)) &&
                  (a.h_out == a.residual || apart(a.h_out, 2 * n, a.residual, 2 * n)) &&
                  apart(a.q_out, n, a.x, 2 * n) && apart(a.scales_out, sb, a.q_out, n) &&
                  apart(a.y_out, 2 * n, a.h_out, 2 * n);
  return ok ? record(mx ? "mx8_rms_norm" : "fp8q_rms_norm", a.rows, a.hidden) : hipErrorInvalidValue;
}

uint64_t norm_backward_workspace(uint64_t rows, uint32_t hidden) { return rows > 1 ? 8ull * hidden : 0; }

hipError_t launch_rms_norm_backward(const NormBackward &a, hipStream_t) {
  const uint64_t n = a.rows * a.hidden;
  const bool inputs = a.rows == 0 || (al(a.dy, 16) && al(a.h, 16) && al(a.weight, 16) && al(a.rstd, 4) &&
                                      al(a.dx, 16) && apart(a.dx, 2 * n, a.h, 2 * n));
  const bool ok = inputs && a.hidden && a.hidden <= FP8Q_NORM_MAX_HIDDEN && al(a.dweight, 4) &&
                  al0(a.workspace, 16) && (norm_backward_workspace(a.rows, a.hidden) == 0 || a.workspace);
  return ok ? record("rms_norm_backward", a.rows, a.hidden) : hipErrorInvalidValue;
}

uint64_t moe_sort_workspace(uint32_t pairs, uint32_t experts) { return pairs > 100 ? 4ull * experts : 0; }

hipError_t launch_moe_sort(const MoeSort &a, hipStream_t) {
  const bool ok = a.experts >= 1 && a.experts <= FP8Q_MAX_EXPERTS && a.pairs <= FP8Q_MAX_PAIRS &&
                  al(a.offsets, 4) &&
                  (a.pairs == 0 || (al(a.ids, a.ids64 ? 8 : 4) && al(a.slots, 4) && al(a.pairs_out, 4))) &&
                  apart(a.slots, 4ull * a.pairs, a.pairs_out, 4ull * a.pairs) &&
                  (moe_sort_workspace(a.pairs, a.experts) == 0 || a.workspace);
  return ok ? record(a.ids64 ? "moe_sort64" : "moe_sort32", a.pairs, a.experts) : hipErrorInvalidValue;
}

hipError_t launch_moe_permute(const MoePermute &a, hipStream_t) {
  const bool ok = a.tokens && topk_ok(a.topk) && a.row_bytes && a.dst_rows && al(a.src, 16) && al(a.dst, 16) &&
                  al(a.slots, 4) && (a.scale_row_bytes == 0 || (a.src_scales && a.dst_scales)) &&
                  apart(a.dst, a.dst_rows * a.row_bytes, a.src, (uint64_t)a.tokens * a.row_bytes);
  return ok ? record("moe_permute", a.tokens, a.row_bytes) : hipErrorInvalidValue;
}

hipError_t launch_moe_combine(int format, const MoeCombine &a, hipStream_t) {
  const bool coded = format != FP8Q_ROWS_BF16;
  const bool ok = format >= 0 && format <= 3 && a.tokens && topk_ok(a.topk) && a.hidden &&
                  a.hidden <= FP8Q_MAX_HIDDEN && al(a.slots, 4) && al0(a.weights, 4) && al(a.out, 16) &&
                  (a.row_count == 0 || (al(a.rows, 16) && (!coded || a.scales))) && (coded || !a.scales);
  return ok ? record("moe_combine", a.tokens, a.hidden) : hipErrorInvalidValue;
}

hipError_t launch_moe_combine_backward(const MoeCombineBackward &a, hipStream_t) {
  const bool ok = a.tokens && topk_ok(a.topk) && a.hidden <= FP8Q_MAX_HIDDEN && al(a.slots, 4) &&
                  al(a.weights, 4) && al(a.dweights, 4) && al0(a.dy, 16) &&
                  (a.row_count == 0 || a.hidden == 0 || (al(a.rows, 16) && al(a.drows, 16)));
  return ok ? record("moe_combine_backward", a.tokens, a.hidden) : hipErrorInvalidValue;
}

}  // namespace fp8q

#define STUB extern "C" __attribute__((visibility("default")))
STUB long layer_stub_calls(void) { return g_rec.calls; }
STUB const char *layer_stub_last(void) { return g_rec.last; }
STUB unsigned long long layer_stub_a(void) { return g_rec.a; }
STUB unsigned long long layer_stub_b(void) { return g_rec.b; }
