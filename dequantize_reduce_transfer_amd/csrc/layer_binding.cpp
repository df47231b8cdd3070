// layer_binding.cpp -- CPython module over libfp8q_layer.so: checks tensors,
// allocates the outputs that the caller does not give, and calls the C ABI.
//
// layer.py defines the public functions (signatures, defaults, documentation)
// and passes their arguments on in order.  The checks and allocations are here
// because they, not the kernels, set the time of a small call: through ctypes
// a norm of one row took 17.5 us of host time on MI355X, of which the launch
// is 3.5; through this module the whole call takes 6.5 us, 3.8 where the outputs
// are given.
//
// Every function returns (status, outputs...), with None for an output that is
// neither given nor asked for, and raises TypeError or ValueError for a tensor
// that does not fit.  The stream is the raw handle that layer.py passes, of the
// stream that is current during the call: torch's allocator takes memory from
// the current stream's own, so what is allocated here is the kernels' alone.
#include "binding.h"
#include "fp8q_layer.h"

namespace {

int weight_code(const at::Tensor &w, int64_t hidden) {
  if (w.numel() != hidden) refuse("weight must hold hidden = " + std::to_string(hidden) + " values");
  return w.scalar_type() == at::kFloat ? FP8Q_WEIGHT_F32 : FP8Q_WEIGHT_BF16;
}

int64_t hidden_of(const at::Tensor &t, const char *name) {
  if (t.dim() < 1) refuse(std::string(name) + " needs at least one dimension");
  return t.size(-1);
}

// mx, x, weight, eps, residual, fmt, want_h, want_y, want_rstd, h_out, y_out,
// q_out, scales_out, rstd_out, stream -> status, q, scales, h, y, rstd
PyObject *rms_norm_quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    const bool mx = n > 0 && args[0] == Py_True;
    Call c(mx ? "mx8_rms_norm_quantize" : "fp8q_rms_norm_quantize", args, n, 15);
    const bool want_h = c.truth(6, "want_h"), want_y = c.truth(7, "want_y"), want_rstd = c.truth(8, "want_rstd");
    const at::Tensor &x = c.tensor(1, "x", {at::kBFloat16});
    const int64_t hidden = hidden_of(x, "x"), rows = hidden ? x.numel() / hidden : 0;
    const at::Tensor &w = c.tensor(2, "weight", {at::kFloat, at::kBFloat16});
    const int wcode = weight_code(w, hidden);
    const float eps = (float)c.number(3, "eps");
    at::Tensor res;
    if (!c.absent(4)) {
      res = c.tensor(4, "residual", {at::kBFloat16});
      if (res.sizes() != x.sizes()) refuse("residual must have the shape of x");
    } else if (!c.absent(9)) {
      refuse("h_out needs a residual: without one h is x");
    }
    const fp8q_format fmt = mx ? FP8Q_E4M3 : format_code(c, 5);
    if (mx && hidden % FP8Q_MX_BLOCK) refuse("hidden must be a multiple of 32");
    at::Tensor h, y, rstd;
    if (res.defined() && (want_h || !c.absent(9))) h = c.output(9, "h_out", at::kBFloat16, x.sizes());
    if (want_y || !c.absent(10)) y = c.output(10, "y_out", at::kBFloat16, x.sizes());
    const at::Tensor q = c.output(11, "q_out", at::kByte, x.sizes());
    const at::Tensor s =
        mx ? c.output(12, "e8m0_out", at::kByte, {rows, hidden / FP8Q_MX_BLOCK})
           : c.output(12, "scales_out", at::kFloat, {rows, ceil_div(hidden, FP8Q_BLOCK)});
    if (want_rstd || !c.absent(13))
      rstd = c.output(13, "rstd_out", at::kFloat, x.sizes().slice(0, x.dim() - 1));
    const c10::DeviceGuard on(c.device());
    const fp8q_status st =
        mx ? mx8_rms_norm_quantize(ptr(x), ptr(res), ptr(w), (fp8q_weight_dtype)wcode, eps, rows, hidden,
                                   ptr(h), ptr(y), ptr(q), ptr(s), f32(rstd), c.stream(14))
           : fp8q_rms_norm_quantize(ptr(x), ptr(res), ptr(w), (fp8q_weight_dtype)wcode, eps, rows, hidden,
                                    fmt, ptr(h), ptr(y), ptr(q), f32(s), f32(rstd), c.stream(14));
    return result(st, {q, s, h, y, rstd});
  });
}

// dy, h, weight, rstd, dh, dx_out, dweight_out, workspace, stream
// -> status, dx, dweight
PyObject *rms_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_rms_norm_backward", args, n, 9);
    const at::Tensor &dy = c.tensor(0, "dy", {at::kBFloat16});
    const at::Tensor &h = c.tensor(1, "h", {at::kBFloat16});
    const int64_t hidden = hidden_of(h, "h"), rows = hidden ? h.numel() / hidden : 0;
    const at::Tensor &w = c.tensor(2, "weight", {at::kFloat, at::kBFloat16});
    const at::Tensor &rstd = c.tensor(3, "rstd", {at::kFloat});
    if (dy.sizes() != h.sizes() || rstd.numel() != rows)
      refuse("dy must have the shape of h, and rstd one value a row");
    at::Tensor dh;
    if (!c.absent(4)) {
      dh = c.tensor(4, "dh", {at::kBFloat16});
      if (dh.sizes() != h.sizes()) refuse("dh must have the shape of h");
    }
    const int wcode = weight_code(w, hidden);
    const at::Tensor dx = c.output(5, "dx_out", at::kBFloat16, h.sizes());
    const at::Tensor dw = c.output(6, "dweight_out", at::kFloat, {hidden});
    const at::Tensor ws = c.workspace(7, fp8q_rms_norm_backward_workspace(rows, hidden));
    const c10::DeviceGuard on(c.device());
    const fp8q_status st = fp8q_rms_norm_backward(
        ptr(dy), ptr(h), ptr(w), (fp8q_weight_dtype)wcode, f32(rstd), ptr(dh), rows, hidden, ptr(dx),
        f32(dw), ptr(ws), ws.defined() ? ws.numel() : 0, c.stream(8));
    return result(st, {dx, dw});
  });
}

// ids, experts, slots_out, pairs_out, offsets_out, workspace, stream
// -> status, slots, pairs, offsets
PyObject *moe_sort(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_moe_sort", args, n, 7);
    const at::Tensor &ids = c.tensor(0, "ids", {at::kInt, at::kLong});
    if (ids.dim() != 2 || ids.size(1) < 1 || ids.size(1) > FP8Q_MAX_TOPK)
      refuse("ids must be [tokens, topk], topk 1 .. " + std::to_string(FP8Q_MAX_TOPK));
    const long long experts = c.integer(1, "experts");
    if (experts < 1 || experts > FP8Q_MAX_EXPERTS)
      refuse("experts must be 1 .. " + std::to_string(FP8Q_MAX_EXPERTS));
    const int64_t tokens = ids.size(0);
    const int topk = (int)ids.size(1);
    const at::Tensor slots = c.output(2, "slots_out", at::kInt, ids.sizes());
    const at::Tensor pairs = c.output(3, "pairs_out", at::kInt, {tokens * topk});
    const at::Tensor offsets = c.output(4, "offsets_out", at::kInt, {experts + 1});
    const at::Tensor ws = c.workspace(5, fp8q_moe_sort_workspace(tokens, topk, (int)experts));
    const c10::DeviceGuard on(c.device());
    const fp8q_status st =
        fp8q_moe_sort(ptr(ids), (int)ids.element_size(), tokens, topk, (int)experts, i32(slots),
                      i32(pairs), i32(offsets), ptr(ws), ws.defined() ? ws.numel() : 0, c.stream(6));
    return result(st, {slots, pairs, offsets});
  });
}

// A slot table's tokens and topk; `tokens` -1: any number of them.
const at::Tensor &slot_table(Call &c, int i, int64_t tokens) {
  const at::Tensor &s = c.tensor(i, "slots", {at::kInt});
  if (s.dim() != 2) refuse("slots must be [tokens, topk]");
  if (tokens >= 0 && s.size(0) != tokens) refuse("slots must have one row a token");
  if (s.size(1) < 1 || s.size(1) > FP8Q_MAX_TOPK)
    refuse("topk must be 1 .. " + std::to_string(FP8Q_MAX_TOPK));
  return s;
}

// x, slots, scales, out, scales_out, stream -> status, rows, scales
PyObject *moe_permute(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_moe_permute", args, n, 6);
    const at::Tensor &x = c.tensor(0, "x", {});
    if (x.dim() != 2) refuse("x must be [tokens, hidden]");
    const at::Tensor &slots = slot_table(c, 1, x.size(0));
    int64_t rows = slots.numel();
    if (!c.absent(3)) {
      const at::Tensor &o = c.tensor(3, "out", {x.scalar_type()});
      rows = o.dim() ? o.size(0) : 0;
    }
    const at::Tensor out = c.output(3, "out", x.scalar_type(), {rows, x.size(1)});
    at::Tensor scales, scales_out;
    if (!c.absent(2)) {
      scales = c.tensor(2, "scales", {});
      if (scales.dim() != 2 || scales.size(0) != x.size(0)) refuse("scales must be [tokens, scales a row]");
      scales_out = c.output(4, "scales_out", scales.scalar_type(), {rows, scales.size(1)});
    } else if (!c.absent(4)) {
      refuse("scales_out needs scales");
    }
    const c10::DeviceGuard on(c.device());
    const fp8q_status st = fp8q_moe_permute(
        ptr(x), x.size(1) * x.element_size(), ptr(scales),
        scales.defined() ? scales.size(1) * scales.element_size() : 0, i32(slots), x.size(0),
        (int)slots.size(1), rows, ptr(out), ptr(scales_out), c.stream(5));
    return result(st, {out, scales_out});
  });
}

// rows, slots, weights, scales, fmt, out is bf16, out, stream -> status, out
PyObject *moe_combine(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_moe_combine", args, n, 8);
    const at::Tensor &rows = c.tensor(0, "rows", {at::kBFloat16, at::kByte});
    const at::Tensor &slots = slot_table(c, 1, -1);
    if (rows.dim() != 2) refuse("rows must be [n, hidden]");
    const int64_t count = rows.size(0), hidden = rows.size(1);
    at::Tensor weights, scales;
    if (!c.absent(2)) weights = c.shaped(2, "weights", at::kFloat, slots.sizes());
    fp8q_row_format format = FP8Q_ROWS_BF16;
    if (rows.scalar_type() == at::kBFloat16) {
      if (!c.absent(3)) refuse("bf16 rows have no scales");
    } else {
      if (c.absent(3)) refuse_type("codes need scales: a float32 tensor, or uint8 E8M0 codes");
      scales = c.tensor(3, "scales", {at::kFloat, at::kByte});
      int64_t each = ceil_div(hidden, FP8Q_BLOCK);
      if (scales.scalar_type() == at::kByte) {
        if (hidden % FP8Q_MX_BLOCK) refuse("hidden must be a multiple of 32");
        format = FP8Q_ROWS_MX8;
        each = hidden / FP8Q_MX_BLOCK;
      } else {
        format = format_code(c, 4) == FP8Q_E4M3 ? FP8Q_ROWS_E4M3 : FP8Q_ROWS_E5M2;
      }
      if (scales.numel() != count * each)
        refuse("scales must hold " + std::to_string(each) + " values a row");
    }
    const bool bf16 = c.truth(5, "out_dtype");
    const at::Tensor out =
        c.output(6, "out", bf16 ? at::kBFloat16 : at::kFloat, {slots.size(0), hidden});
    const c10::DeviceGuard on(c.device());
    const fp8q_status st = fp8q_moe_combine(
        ptr(rows), format, ptr(scales), i32(slots), f32(weights), slots.size(0), (int)slots.size(1),
        count, hidden, ptr(out), bf16 ? FP8Q_OUT_BF16 : FP8Q_OUT_F32, c.stream(7));
    return result(st, {out});
  });
}

// dy, rows, slots, weights, drows_out, dweights_out, stream
// -> status, drows, dweights
PyObject *moe_combine_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_moe_combine_backward", args, n, 7);
    const at::Tensor &dy = c.tensor(0, "dy", {at::kBFloat16});
    const at::Tensor &rows = c.tensor(1, "rows", {at::kBFloat16});
    if (dy.dim() != 2 || rows.dim() != 2 || dy.size(1) != rows.size(1))
      refuse("dy must be [tokens, hidden] and rows [n, hidden]");
    const at::Tensor &slots = slot_table(c, 2, dy.size(0));
    const at::Tensor &weights = c.shaped(3, "weights", at::kFloat, slots.sizes());
    const at::Tensor drows = c.output(4, "drows_out", at::kBFloat16, rows.sizes());
    const at::Tensor dweights = c.output(5, "dweights_out", at::kFloat, slots.sizes());
    const c10::DeviceGuard on(c.device());
    const fp8q_status st = fp8q_moe_combine_backward(
        ptr(dy), ptr(rows), i32(slots), f32(weights), dy.size(0), (int)slots.size(1), rows.size(0),
        dy.size(1), ptr(drows), f32(dweights), c.stream(6));
    return result(st, {drows, dweights});
  });
}

PyMethodDef methods[] = {FAST(rms_norm_quantize), FAST(rms_norm_backward), FAST(moe_sort),
                         FAST(moe_permute),       FAST(moe_combine),       FAST(moe_combine_backward),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", "Calls of libfp8q_layer.so on torch tensors.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer(void) { return PyModule_Create(&module); }
