// model_binding.cpp -- CPython module over libfp8q_model.so: checks tensors,
// allocates the outputs that the caller does not give, and calls the C ABI.
//
// model.py defines the public functions and passes their arguments on in
// order; what holds of layer_binding.cpp's functions (results, refusals, the
// stream) holds of these.
#include <vector>

#include "binding.h"
#include "fp8q_model.h"

namespace {

// Tells autograd that a call writes to a tensor of the caller's, as torch's own
// in-place functions do: a graph that has saved it refuses its backward pass.
void written(c10::TensorImpl *t) {
  if (!t->is_inference()) t->bump_version();
}

fp8q_logits_dtype logits_code(at::ScalarType t) { return t == at::kFloat ? FP8Q_LOGITS_F32 : FP8Q_LOGITS_BF16; }

void check_route(const at::Tensor &logits, long long topk) {
  if (logits.dim() != 2) refuse("logits must be [tokens, experts]");
  if (logits.size(1) < 1 || logits.size(1) > FP8Q_MAX_EXPERTS)
    refuse("experts must be 1 .. " + std::to_string(FP8Q_MAX_EXPERTS));
  if (topk < 1 || topk > FP8Q_MAX_TOPK || topk > logits.size(1))
    refuse("topk must be 1 .. " + std::to_string(FP8Q_MAX_TOPK) + " and at most experts");
}

// logits, topk, normalize, weights_out, ids_out, stream -> status, weights, ids
PyObject *moe_route(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_moe_route", args, n, 6);
    const at::Tensor &logits = c.tensor(0, "logits", {at::kFloat, at::kBFloat16});
    const long long topk = c.integer(1, "topk");
    const bool normalize = c.truth(2, "normalize");
    check_route(logits, topk);
    const at::Tensor weights = c.output(3, "weights_out", at::kFloat, {logits.size(0), topk});
    const at::Tensor ids = c.output(4, "ids_out", at::kInt, {logits.size(0), topk});
    const c10::DeviceGuard on(c.device());
    const fp8q_status st =
        fp8q_moe_route(ptr(logits), logits_code(logits.scalar_type()), logits.size(0), (int)logits.size(1), (int)topk,
                       normalize, f32(weights), i32(ids), c.stream(5));
    return result(st, {weights, ids});
  });
}

// dweights, logits, weights, ids, normalize, dlogits_out, stream
// -> status, dlogits
PyObject *moe_route_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_moe_route_backward", args, n, 7);
    const at::Tensor &dweights = c.tensor(0, "dweights", {at::kFloat});
    const at::Tensor &logits = c.tensor(1, "logits", {at::kFloat, at::kBFloat16});
    if (dweights.dim() != 2) refuse("dweights must be [tokens, topk]");
    check_route(logits, dweights.size(1));
    if (logits.size(0) != dweights.size(0)) refuse("logits must have one row a token");
    const at::Tensor &weights = c.shaped(2, "weights", at::kFloat, dweights.sizes());
    const at::Tensor &ids = c.shaped(3, "ids", at::kInt, dweights.sizes());
    const bool normalize = c.truth(4, "normalize");
    const at::Tensor dlogits = c.output(5, "dlogits_out", logits.scalar_type(), logits.sizes());
    const c10::DeviceGuard on(c.device());
    const fp8q_status st = fp8q_moe_route_backward(
        f32(dweights), ptr(logits), logits_code(logits.scalar_type()), f32(weights), i32(ids), logits.size(0),
        (int)logits.size(1), (int)dweights.size(1), normalize, ptr(dlogits), c.stream(6));
    if (st == FP8Q_OK && !c.absent(5)) written(dlogits.unsafeGetTensorImpl());
    return result(st, {dlogits});
  });
}

// An expert matrix's tensors: [experts, rows, width], each expert's rows one
// after the other, the experts any whole number of rows apart.
struct Matrix {
  fp8q_expert_matrix m;
  fp8q_row_format format;
};

Matrix matrix(Call &c, int i, int scales_at, const char *name, int64_t experts, int64_t rows, int64_t width,
              int fmt_at) {
  const at::Tensor &t = c.tensor(c.object(i), name, {at::kBFloat16, at::kByte}, false);
  const std::string what = name;
  if (t.dim() != 3 || t.size(0) != experts || t.size(1) != rows || t.size(2) != width)
    refuse(what + " must be of shape " + shape_name({experts, rows, width}) + ", got " + shape_name(t.sizes()));
  const auto rows_apart = [&](const at::Tensor &v, const std::string &label) -> int64_t {
    const int64_t r = v.size(1), w = v.size(2);
    if (v.numel() == 0 || v.is_contiguous()) return rows;
    if ((w > 1 && v.stride(2) != 1) || (r > 1 && v.stride(1) != w) || v.stride(0) % w || v.stride(0) < r * w)
      refuse(label + ": an expert's rows must be contiguous");
    return v.size(0) > 1 ? v.stride(0) / w : rows;
  };
  Matrix out{{ptr(t), nullptr, (size_t)rows_apart(t, what)}, FP8Q_ROWS_BF16};
  if (t.scalar_type() == at::kBFloat16) {
    if (!c.absent(scales_at)) refuse("bf16 matrices have no scales");
    return out;
  }
  if (c.absent(scales_at)) refuse_type(what + "'s codes need scales: a float32 tensor, or uint8 E8M0 codes");
  const std::string label = what + "_scales";
  const at::Tensor &s = c.tensor(c.object(scales_at), label.c_str(), {at::kFloat, at::kByte}, false);
  int64_t each = ceil_div(width, FP8Q_BLOCK);
  if (s.scalar_type() == at::kByte) {
    if (width % FP8Q_MX_BLOCK) refuse("hidden and inter must be multiples of 32");
    out.format = FP8Q_ROWS_MX8;
    each = width / FP8Q_MX_BLOCK;
  } else {
    out.format = format_code(c, fmt_at) == FP8Q_E4M3 ? FP8Q_ROWS_E4M3 : FP8Q_ROWS_E5M2;
  }
  if (s.numel() != experts * rows * each)
    refuse(label + " must hold " + std::to_string(each) + " values a row");
  if (!s.is_contiguous() && (s.dim() != 3 || s.size(0) != experts || s.size(1) != rows))
    refuse(label + " must be contiguous or [experts, rows, scales a row]");
  const int64_t apart = s.is_contiguous() ? rows : rows_apart(s, label);
  if (t.numel() && experts > 1 && apart != (int64_t)out.m.expert_rows)
    refuse(label + ": the experts must be as many rows apart as " + what + "'s");
  out.m.scales = ptr(s);
  return out;
}

// x, ids, weights, gate, up, down, gate_scales, up_scales, down_scales, fmt,
// out is bf16, out, workspace, stream -> status, out
PyObject *moe_experts(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_moe_experts", args, n, 14);
    const at::Tensor &x = c.tensor(0, "x", {at::kBFloat16});
    const at::Tensor &ids = c.tensor(1, "ids", {at::kInt, at::kLong});
    if (x.dim() != 2) refuse("x must be [tokens, hidden]");
    const int64_t tokens = x.size(0), hidden = x.size(1);
    if (ids.dim() != 2 || ids.size(0) != tokens || ids.size(1) < 1 || ids.size(1) > FP8Q_MAX_TOPK)
      refuse("ids must be [tokens, topk], topk 1 .. " + std::to_string(FP8Q_MAX_TOPK));
    if (ids.numel() > FP8Q_EXPERTS_MAX_PAIRS)
      refuse("tokens * topk must be at most " + std::to_string(FP8Q_EXPERTS_MAX_PAIRS) +
             ": more tokens are sorted, permuted and combined");
    const at::Tensor &weights = c.shaped(2, "weights", at::kFloat, ids.sizes());
    const at::Tensor &g = c.tensor(c.object(3), "gate", {at::kBFloat16, at::kByte}, false);
    if (g.dim() != 3) refuse("gate must be [experts, inter, hidden]");
    const int64_t experts = g.size(0), inter = g.size(1);
    if (experts < 1 || experts > FP8Q_MAX_EXPERTS)
      refuse("experts must be 1 .. " + std::to_string(FP8Q_MAX_EXPERTS));
    if (hidden > FP8Q_EXPERTS_MAX_SIZE || inter > FP8Q_EXPERTS_MAX_SIZE)
      refuse("hidden and inter must be at most " + std::to_string(FP8Q_EXPERTS_MAX_SIZE));
    const Matrix gate = matrix(c, 3, 6, "gate", experts, inter, hidden, 9);
    const Matrix up = matrix(c, 4, 7, "up", experts, inter, hidden, 9);
    const Matrix down = matrix(c, 5, 8, "down", experts, hidden, inter, 9);
    if (up.format != gate.format || down.format != gate.format) refuse("gate, up and down must be of one format");
    const bool bf16 = c.truth(10, "out_dtype");
    const fp8q_out_dtype dtype = bf16 ? FP8Q_OUT_BF16 : FP8Q_OUT_F32;
    const at::Tensor out = c.output(11, "out", bf16 ? at::kBFloat16 : at::kFloat, {tokens, hidden});
    const at::Tensor ws = c.workspace(12, fp8q_moe_experts_workspace(tokens, (int)ids.size(1), (int)experts, hidden, inter, dtype));
    const c10::DeviceGuard on(c.device());
    const fp8q_status st = fp8q_moe_experts(
        ptr(x), ptr(ids), (int)ids.element_size(), f32(weights), gate.format, &gate.m, &up.m, &down.m, tokens,
        (int)ids.size(1), (int)experts, hidden, inter, ptr(out), dtype, ptr(ws), ws.defined() ? ws.numel() : 0,
        c.stream(13));
    return result(st, {out});
  });
}

// A list or tuple, held.
class Items {
 public:
  Items(PyObject *o, const char *name) : list_(PyList_Check(o) || PyTuple_Check(o) ? Py_NewRef(o) : nullptr) {
    if (!list_) refuse_type(std::string(name) + " must be a list or tuple");
  }
  ~Items() { Py_DECREF(list_); }
  Items(const Items &) = delete;
  Items &operator=(const Items &) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(list_); }
  PyObject *operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(list_, i); }

 private:
  PyObject *list_;
};

// A list's gradients and, where `scales_at` holds any, their scales; and, where
// wanted, the tensors that clipping writes.  The caller's lists keep the tensors
// alive, so no Python code may run between this and the call (a number's
// __float__ could change the lists).
std::vector<fp8q_grad> gradients(Call &c, int grads_at, int scales_at, int fmt_at,
                                 std::vector<c10::TensorImpl *> *clipped = nullptr) {
  const Items grads(c.object(grads_at), "grads");
  const fp8q_format fmt = format_code(c, fmt_at);
  PyObject *none = Py_None;
  const bool any = !c.absent(scales_at);
  const Items *given = nullptr;
  std::vector<fp8q_grad> list;
  list.reserve((size_t)grads.size());
  if (clipped) clipped->reserve((size_t)grads.size());
  const auto fill = [&] {
    for (Py_ssize_t i = 0; i < grads.size(); ++i) {
      const at::Tensor &t = c.tensor(grads[i], "a gradient", {at::kFloat, at::kBFloat16, at::kByte}, true);
      PyObject *scale = given ? (*given)[i] : none;
      fp8q_grad g{ptr(t), nullptr, (size_t)t.numel(), 0,
                  t.scalar_type() == at::kFloat      ? FP8Q_GRAD_F32
                  : t.scalar_type() == at::kBFloat16 ? FP8Q_GRAD_BF16
                  : fmt == FP8Q_E4M3                 ? FP8Q_GRAD_E4M3
                                                     : FP8Q_GRAD_E5M2};
      if (t.scalar_type() != at::kByte) {
        if (scale != none) refuse("float32 and bfloat16 gradients have no scales");
      } else {
        if (scale == none) refuse_type("codes need scales: a float32 tensor");
        const at::Tensor &s = c.tensor(scale, "a gradient's scales", {at::kFloat}, true);
        if (s.numel() != 1 && s.numel() != ceil_div(t.numel(), FP8Q_BLOCK))
          refuse("a gradient's scales must be one per 128 codes, or one");
        g.scales = f32(s);
        g.scale_count = (size_t)s.numel();
        if (clipped) clipped->push_back(s.unsafeGetTensorImpl());
      }
      if (clipped && scale == none) clipped->push_back(t.unsafeGetTensorImpl());
      list.push_back(g);
    }
  };
  if (any) {
    const Items scales(c.object(scales_at), "scales");
    if (scales.size() != grads.size()) refuse("scales must have one entry a gradient (None for those without)");
    given = &scales;
    fill();
  } else {
    fill();
  }
  return list;
}

// grads, scales, fmt, out, workspace, stream -> status, sumsq
PyObject *grad_sumsq(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_grad_sumsq", args, n, 6);
    const std::vector<fp8q_grad> list = gradients(c, 0, 1, 2);
    if (list.empty() && c.absent(3)) refuse("an empty list needs out, whose device it is on");
    const at::Tensor out = c.output(3, "out", at::kDouble, {1});
    const at::Tensor ws = c.workspace(4, fp8q_grad_sumsq_workspace(list.data(), list.size()));
    const c10::DeviceGuard on(c.device());
    const fp8q_status st =
        fp8q_grad_sumsq(list.data(), list.size(), static_cast<double *>(ptr(out)), ptr(ws),
                        ws.defined() ? ws.numel() : 0, c.stream(5));
    return result(st, {out});
  });
}

// grads, sumsq, max_norm, scales, fmt, eps, norm_out, stream -> status, norm
PyObject *grad_clip(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return guarded([&] {
    Call c("fp8q_grad_clip", args, n, 8);
    const double max_norm = c.number(2, "max_norm"), eps = c.number(5, "eps");
    std::vector<c10::TensorImpl *> clipped;
    const std::vector<fp8q_grad> list = gradients(c, 0, 3, 4, &clipped);
    const at::Tensor &sumsq = c.shaped(1, "sumsq", at::kDouble, {1});
    const at::Tensor norm = c.output(6, "norm_out", at::kFloat, {1});
    const c10::DeviceGuard on(c.device());
    const fp8q_status st =
        fp8q_grad_clip(list.data(), list.size(), static_cast<const double *>(ptr(sumsq)), max_norm, eps,
                       f32(norm), c.stream(7));
    if (st == FP8Q_OK)
      for (c10::TensorImpl *t : clipped) written(t);
    return result(st, {norm});
  });
}

PyMethodDef methods[] = {FAST(moe_route),  FAST(moe_route_backward), FAST(moe_experts), FAST(grad_sumsq),
                         FAST(grad_clip), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_model", "Calls of libfp8q_model.so on torch tensors.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__model(void) { return PyModule_Create(&module); }
