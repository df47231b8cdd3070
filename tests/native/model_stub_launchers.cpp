// model_stub_launchers.cpp -- host-only stand-ins for the model operators'
// launchers, so that their C-ABI layer (csrc/model_api.hip, compiled host-only
// with g++) can run under AddressSanitizer and UndefinedBehaviorSanitizer on a
// machine without a GPU.
//
// Each stub enqueues nothing.  It checks what the real launchers assume of a
// validated call (model_launch.h) and records the call; a broken assumption
// returns hipErrorInvalidValue, which the ABI reports as FP8Q_ERR_HIP.
#include <stdint.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "fp8q_model.h"
#include "model_launch.h"

namespace {

struct Record {
  long calls;
  char last[32];
  uint64_t a, b;
};
Record g_rec = {0, {0}, 0, 0};

bool al(const void *p, uintptr_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

hipError_t record(const char *name, uint64_t a, uint64_t b) {
  ++g_rec.calls;
  strncpy(g_rec.last, name, sizeof(g_rec.last) - 1);
  g_rec.a = a;
  g_rec.b = b;
  return hipSuccess;
}

bool route_ok(uint64_t tokens, uint32_t experts, uint32_t topk) {
  return tokens && experts >= 1 && experts <= FP8Q_MAX_EXPERTS && topk >= 1 && topk <= FP8Q_MAX_TOPK &&
         topk <= experts && tokens * topk <= FP8Q_MAX_PAIRS;
}

bool grad_ok(const fp8q::Grad &g, bool clip) {
  if (g.kind < 0 || g.kind > (clip ? 1 : 3)) return false;
  if (!g.count) return true;
  return al(g.data, g.kind == 0 ? 4 : g.kind == 1 ? 2 : 1) && (g.kind < 2) == !g.scales && (g.kind >= 2 || !g.one_scale);
}

}  // namespace

namespace fp8q {

hipError_t launch_moe_route(const MoeRoute &a, hipStream_t) {
  const bool ok = route_ok(a.tokens, a.experts, a.topk) && al(a.logits, 16) && al(a.weights, 4) && al(a.ids, 4);
  return ok ? record("moe_route", a.tokens, a.experts) : hipErrorInvalidValue;
}

hipError_t launch_moe_route_backward(const MoeRouteBackward &a, hipStream_t) {
  const bool ok = route_ok(a.tokens, a.experts, a.topk) && (a.normalize || al(a.logits, 16)) && al(a.dweights, 4) &&
                  al(a.weights, 4) && al(a.ids, 4) && al(a.dlogits, 16);
  return ok ? record("moe_route_backward", a.tokens, a.experts) : hipErrorInvalidValue;
}

uint64_t moe_experts_workspace(uint32_t pairs, uint32_t, uint32_t, uint32_t inter, bool out_bf16) {
  return (out_bf16 ? 4ull : 6ull) * pairs * inter;
}

hipError_t launch_moe_experts(int format, const MoeExperts &a, hipStream_t) {
  bool ok = format >= 0 && format <= 3 && a.tokens && a.topk && a.tokens * a.topk <= FP8Q_EXPERTS_MAX_PAIRS &&
            a.experts >= 1 && a.experts <= FP8Q_MAX_EXPERTS && a.hidden && a.hidden <= FP8Q_EXPERTS_MAX_SIZE &&
            a.inter <= FP8Q_EXPERTS_MAX_SIZE && al(a.x, 16) && al(a.ids, a.ids64 ? 8 : 4) && al(a.weights, 4) &&
            al(a.out, 16) && (a.inter == 0 || al(a.workspace, 16));
  if (a.inter)
    for (const ExpertMatrix *m : {&a.gate, &a.up, &a.down})
      ok = ok && m->rows && (format == 0) == !m->scales && m->expert_rows >= (m == &a.down ? a.hidden : a.inter);
  return ok ? record("moe_experts", a.tokens, a.inter) : hipErrorInvalidValue;
}

uint64_t grad_sumsq_workspace(const Grad *grads, uint64_t n) {
  uint64_t all = 0;
  for (uint64_t i = 0; i < n; ++i) all += grads[i].count;
  return all > 1000 ? 64 : 0;
}

hipError_t launch_grad_sumsq(const Grad *grads, uint64_t n, double *sumsq, double *workspace, hipStream_t) {
  bool ok = al(sumsq, 8) && (!grad_sumsq_workspace(grads, n) || al(workspace, 16));
  for (uint64_t i = 0; i < n; ++i) ok = ok && grad_ok(grads[i], false);
  return ok ? record("grad_sumsq", n, n ? grads[0].count : 0) : hipErrorInvalidValue;
}

hipError_t launch_grad_clip(const Grad *grads, uint64_t n, const double *sumsq, double max_norm, double eps,
                            float *norm, hipStream_t) {
  bool ok = al(sumsq, 8) && al(norm, 4) && max_norm >= 0 && eps >= 0;
  for (uint64_t i = 0; i < n; ++i) ok = ok && grad_ok(grads[i], true);
  return ok ? record("grad_clip", n, n ? grads[0].count : 0) : hipErrorInvalidValue;
}

}  // namespace fp8q

#define STUB extern "C" __attribute__((visibility("default")))
STUB long model_stub_calls(void) { return g_rec.calls; }
STUB const char *model_stub_last(void) { return g_rec.last; }
STUB unsigned long long model_stub_a(void) { return g_rec.a; }
STUB unsigned long long model_stub_b(void) { return g_rec.b; }
