// The usual calls of the operators in front of the projections from Python, in
// one native step each, like csrc/ffn/binding.cpp, whose module these functions
// are part of: a function answers None for a call that front.py has to take, an
// int, the status, where the C ABI (include/fp8q_front.h) refuses.  A small
// fp8_rmsnorm call takes 6 us, and 15 through ctypes.
#include "../../../include/fp8q_front.h"

#include "../binding_util.hpp"

namespace {

bool dtype_of(const at::Tensor* t, int* code) {
  if (!t || (t->scalar_type() != at::kBFloat16 && t->scalar_type() != at::kFloat)) return false;
  *code = t->scalar_type() == at::kBFloat16 ? FP8Q_BF16 : FP8Q_F32;
  return true;
}

bool ints(const at::Tensor* t, at::Device device, at::IntArrayRef shape) {
  return t && t->scalar_type() == at::kInt && t->device() == device && t->sizes() == shape && t->is_contiguous();
}

// None or a tensor: false for anything else.
bool optional(PyObject* o, const at::Tensor** t) {
  *t = o == Py_None ? nullptr : tensor(o);
  return *t || o == Py_None;
}

bool flag(PyObject* o, bool* v) {
  *v = o == Py_True;
  return *v || o == Py_False;
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(device));
}

void* at_or_null(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
const void* at_or_null(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// A tuple of those of the tensors that are defined.
PyObject* answer_all(int status, std::initializer_list<const at::Tensor*> all) {
  if (status != FP8Q_OK) return PyLong_FromLong(status);
  Py_ssize_t n = 0, i = 0;
  for (const at::Tensor* t : all) n += t->defined();
  PyObject* out = PyTuple_New(n);
  if (!out) return nullptr;
  for (const at::Tensor* t : all)
    if (t->defined()) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(*t));
  return out;
}

// What both norms take: x, weight, residual or None, eps.
struct Norm {
  const at::Tensor *x, *w, *r;
  int64_t ld_x, ld_r = 0, ld_h = 0, ld_y = 0, m, d;
  int x_code, w_code;
  double eps;
  at::Tensor h, rstd, y;

  bool take(PyObject* const* args) {
    x = tensor(args[0]);
    w = tensor(args[1]);
    if (!here(x) || !dtype_of(x, &x_code) || !dtype_of(w, &w_code) || !optional(args[2], &r) || !PyFloat_CheckExact(args[3]))
      return false;
    eps = PyFloat_AS_DOUBLE(args[3]);
    if (!matrix(x, x->device(), &ld_x)) return false;
    m = x->size(0);
    d = x->size(1);
    if (w->device() != x->device() || w->dim() != 1 || w->size(0) != d || !w->is_contiguous()) return false;
    return !r || (r->scalar_type() == x->scalar_type() && matrix(r, x->device(), &ld_r) && r->sizes() == x->sizes());
  }
  void outputs(bool keep_rstd, bool keep_y) {
    if (r) h = output(m, d, x_code, x->device(), &ld_h);
    if (keep_rstd) rstd = fresh({m}, at::kFloat, x->device());
    if (keep_y) y = output(m, d, x_code, x->device(), &ld_y);
  }
};

// fp8_rmsnorm(x, weight, residual or None, eps, mode, transposed, save_rstd, save_y)
PyObject* fp8_rmsnorm_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  Norm c;
  bool transposed, save_rstd, save_y;
  FP8Q_NONE_UNLESS(n == 8 && c.take(args) && flag(args[5], &transposed) && flag(args[6], &save_rstd) && flag(args[7], &save_y));
  const int mode = number(args[4]);
  FP8Q_NONE_UNLESS(mode >= 0 && c.d % 128 == 0);
  const at::Device dev = c.x->device();
  const int64_t mq = transposed ? round_up(c.m, 128) : c.m;
  at::Tensor q, s, qt, st, none;
  int status;
  {
    Unlocked others_run;
    c.outputs(save_rstd || transposed, save_y);
    q = fresh({mq, c.d}, at::kByte, dev);
    s = fresh({c.d / 128, mq}, at::kFloat, dev);
    if (transposed) {
      qt = fresh({c.d, mq}, at::kByte, dev);
      st = fresh({mq / 128, c.d}, at::kFloat, dev);
    }
    status = fp8_rmsnorm(c.x->data_ptr(), c.ld_x, at_or_null(c.r), c.ld_r, c.x_code, c.m, c.d, c.w->data_ptr(), c.w_code,
                         float(c.eps), mode, at_or_null(c.h), c.ld_h, static_cast<float*>(at_or_null(c.rstd)), at_or_null(c.y),
                         c.ld_y, static_cast<uint8_t*>(q.data_ptr()), c.d > 0 ? c.d : 16, static_cast<float*>(s.data_ptr()),
                         static_cast<uint8_t*>(at_or_null(qt)), mq > 0 ? mq : 16, static_cast<float*>(at_or_null(st)),
                         stream(dev));
  }
  return answer_all(status, {&q, &s, &qt, &st, &c.h, save_rstd ? &c.rstd : &none, &c.y});
  END_HANDLE_TH_ERRORS
}

// int8_rmsnorm(x, weight, residual or None, eps, save_rstd, save_y)
PyObject* int8_rmsnorm_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  Norm c;
  bool save_rstd, save_y;
  FP8Q_NONE_UNLESS(n == 6 && c.take(args) && flag(args[4], &save_rstd) && flag(args[5], &save_y));
  const at::Device dev = c.x->device();
  const int64_t ld_q = round_up(c.d > 0 ? c.d : 1, kChunk);
  at::Tensor q, s;
  int status;
  {
    Unlocked others_run;
    c.outputs(save_rstd, save_y);
    // the last row's bytes up to 16 exist too, as int8_gemm reads them
    q = fresh({c.m, ld_q}, at::kChar, dev);
    if (ld_q != c.d) q = q.as_strided({c.m, c.d}, {ld_q, 1});
    s = fresh({c.m}, at::kFloat, dev);
    status = int8_rmsnorm(c.x->data_ptr(), c.ld_x, at_or_null(c.r), c.ld_r, c.x_code, c.m, c.d, c.w->data_ptr(), c.w_code,
                          float(c.eps), at_or_null(c.h), c.ld_h, static_cast<float*>(at_or_null(c.rstd)), at_or_null(c.y),
                          c.ld_y, static_cast<int8_t*>(q.data_ptr()), ld_q, static_cast<float*>(s.data_ptr()), stream(dev));
  }
  return answer_all(status, {&q, &s, &c.h, &c.rstd, &c.y});
  END_HANDLE_TH_ERRORS
}

// rmsnorm_backward(dy, h, weight, rstd, dh or None)
PyObject* rmsnorm_backward_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  FP8Q_NONE_UNLESS(n == 5);
  const at::Tensor *dy = tensor(args[0]), *h = tensor(args[1]), *w = tensor(args[2]), *rstd = tensor(args[3]), *dh;
  int code, w_code;
  int64_t ld_dy, ld_h, ld_dh = 0, ld_dx;
  FP8Q_NONE_UNLESS(here(dy) && dtype_of(dy, &code) && h && dtype_of(w, &w_code) && optional(args[4], &dh));
  const at::Device dev = dy->device();
  FP8Q_NONE_UNLESS(matrix(dy, dev, &ld_dy) && matrix(h, dev, &ld_h) && h->scalar_type() == dy->scalar_type() &&
                   h->sizes() == dy->sizes());
  const int64_t m = dy->size(0), d = dy->size(1);
  FP8Q_NONE_UNLESS(w->device() == dev && w->dim() == 1 && w->size(0) == d && w->is_contiguous() && floats(rstd, dev, {m}));
  FP8Q_NONE_UNLESS(!dh || (dh->scalar_type() == dy->scalar_type() && matrix(dh, dev, &ld_dh) && dh->sizes() == dy->sizes()));
  const int64_t bytes = fp8q_rmsnorm_backward_workspace(m, d);
  at::Tensor dx, dw, work;
  int status;
  {
    Unlocked others_run;
    dx = output(m, d, code, dev, &ld_dx);
    dw = fresh({d}, at::kFloat, dev);
    if (bytes > 0) work = fresh({bytes}, at::kByte, dev);
    status = rmsnorm_backward(dy->data_ptr(), ld_dy, h->data_ptr(), ld_h, code, m, d, w->data_ptr(), w_code,
                              static_cast<const float*>(rstd->data_ptr()), at_or_null(dh), ld_dh, dx.data_ptr(), ld_dx,
                              static_cast<float*>(dw.data_ptr()), 0, at_or_null(work), stream(dev));
  }
  return answer_all(status, {&dx, &dw});
  END_HANDLE_TH_ERRORS
}

// moe_route(logits, k, valid or None, renormalize)
PyObject* moe_route_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  FP8Q_NONE_UNLESS(n == 4);
  const at::Tensor *z = tensor(args[0]), *valid;
  const int k = number(args[1]);
  bool renormalize;
  int code;
  int64_t ld;
  FP8Q_NONE_UNLESS(here(z) && dtype_of(z, &code) && k >= 0 && optional(args[2], &valid) && flag(args[3], &renormalize));
  const at::Device dev = z->device();
  FP8Q_NONE_UNLESS(matrix(z, dev, &ld));
  const int64_t t = z->size(0), e = z->size(1);
  FP8Q_NONE_UNLESS(!valid || ((valid->scalar_type() == at::kBool || valid->scalar_type() == at::kByte) &&
                              valid->device() == dev && valid->dim() == 1 && valid->size(0) == t && valid->is_contiguous()));
  // sizes are refused before memory is asked for: the C ABI looks at pointers behind them
  FP8Q_NONE_UNLESS(moe_route(nullptr, ld, code, t, e, k, nullptr, renormalize, nullptr, nullptr, nullptr, nullptr, nullptr,
                             nullptr, nullptr) == FP8Q_ERR_NULL);
  const int64_t bytes = fp8q_moe_route_workspace(t, e);
  at::Tensor w, ex, counts, loss, slope, work;
  int status;
  {
    Unlocked others_run;
    w = fresh({t, k}, at::kFloat, dev);
    ex = fresh({t, k}, at::kInt, dev);
    counts = fresh({e}, at::kInt, dev);
    loss = fresh({1}, at::kFloat, dev);
    slope = fresh({e}, at::kFloat, dev);
    if (bytes > 0) work = fresh({bytes}, at::kByte, dev);
    status = moe_route(z->data_ptr(), ld, code, t, e, k, static_cast<const uint8_t*>(at_or_null(valid)), renormalize,
                       static_cast<float*>(w.data_ptr()), static_cast<int32_t*>(ex.data_ptr()),
                       static_cast<int32_t*>(counts.data_ptr()), static_cast<float*>(loss.data_ptr()),
                       static_cast<float*>(slope.data_ptr()), at_or_null(work), stream(dev));
  }
  return answer_all(status, {&w, &ex, &counts, &loss, &slope});
  END_HANDLE_TH_ERRORS
}

// moe_route_backward(logits, experts, slope or None, dweights or None, dloss or None, renormalize)
PyObject* moe_route_backward_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  FP8Q_NONE_UNLESS(n == 6);
  const at::Tensor *z = tensor(args[0]), *ex = tensor(args[1]), *slope, *dw, *dl;
  bool renormalize;
  int code;
  int64_t ld, ld_dz;
  FP8Q_NONE_UNLESS(here(z) && dtype_of(z, &code) && ex && ex->dim() == 2 && optional(args[2], &slope) &&
                   optional(args[3], &dw) && optional(args[4], &dl) && flag(args[5], &renormalize) && (slope || !dl));
  const at::Device dev = z->device();
  FP8Q_NONE_UNLESS(matrix(z, dev, &ld));
  const int64_t t = z->size(0), e = z->size(1), k = ex->size(1);
  FP8Q_NONE_UNLESS(ints(ex, dev, {t, k}) && (!slope || floats(slope, dev, {e})) && (!dw || floats(dw, dev, {t, k})) &&
                   (!dl || floats(dl, dev, {1})));
  at::Tensor dz;
  int status;
  {
    Unlocked others_run;
    dz = output(t, e, code, dev, &ld_dz);
    status = moe_route_backward(z->data_ptr(), ld, code, t, e, k, static_cast<const int32_t*>(ex->data_ptr()),
                                static_cast<const float*>(at_or_null(slope)), static_cast<const float*>(at_or_null(dw)),
                                static_cast<const float*>(at_or_null(dl)), renormalize, dz.data_ptr(), ld_dz, stream(dev));
  }
  return answer(status, THPVariable_Wrap(dz));
  END_HANDLE_TH_ERRORS
}

// fp8_moe_dispatch(experts, q, scales, num_experts, a or None, a_scales or None): both given or neither
PyObject* moe_dispatch_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  FP8Q_NONE_UNLESS(n == 6 && PyLong_CheckExact(args[3]));
  const at::Tensor *ex = tensor(args[0]), *q = tensor(args[1]), *s = tensor(args[2]), *a, *sa;
  int overflow = 0;
  const long e = PyLong_AsLongAndOverflow(args[3], &overflow);
  int64_t ld_q, ld_a;
  FP8Q_NONE_UNLESS(!overflow && here(q) && codes(q) && ex && ex->dim() == 2 && optional(args[4], &a) && optional(args[5], &sa) &&
                   !a == !sa);
  const at::Device dev = q->device();
  FP8Q_NONE_UNLESS(matrix(q, dev, &ld_q) && (!a || (a->scalar_type() == at::kByte && matrix(a, dev, &ld_a))));
  const int64_t t = q->size(0), d = q->size(1), k = ex->size(1), groups = d / 128;
  const int64_t rows = a ? a->size(0) : fp8q_moe_max_rows(t, k, e), bytes = fp8q_moe_dispatch_workspace(t, k, e);
  FP8Q_NONE_UNLESS(d % 128 == 0 && rows >= 0 && rows % 128 == 0 && bytes >= 0 && ints(ex, dev, {t, k}) &&
                   floats(s, dev, {groups, t}) && (!a || (a->size(1) == d && floats(sa, dev, {groups, rows}))));
  at::Tensor new_a, new_sa, group, slots, tokens, work;
  int status;
  {
    Unlocked others_run;
    if (a) {
      new_a = *a;
      new_sa = *sa;
    } else {
      new_a = fresh({rows, d}, at::kByte, dev);
      new_sa = fresh({groups, rows}, at::kFloat, dev);
      ld_a = d > 0 ? d : 16;
    }
    group = fresh({rows / 128}, at::kInt, dev);
    slots = fresh({t, k}, at::kInt, dev);
    tokens = fresh({rows}, at::kInt, dev);
    if (bytes > 0) work = fresh({bytes}, at::kByte, dev);
    status = fp8_moe_dispatch(static_cast<const int32_t*>(ex->data_ptr()), t, k, e, static_cast<const uint8_t*>(q->data_ptr()),
                              ld_q, static_cast<const float*>(s->data_ptr()), d, rows, static_cast<uint8_t*>(new_a.data_ptr()),
                              ld_a, static_cast<float*>(new_sa.data_ptr()), static_cast<int32_t*>(group.data_ptr()),
                              static_cast<int32_t*>(slots.data_ptr()), static_cast<int32_t*>(tokens.data_ptr()),
                              at_or_null(work), stream(dev));
  }
  return answer_all(status, {&new_a, &new_sa, &group, &slots, &tokens});
  END_HANDLE_TH_ERRORS
}

}  // namespace

extern PyMethodDef fp8q_front_methods[];
PyMethodDef fp8q_front_methods[] = {FP8Q_METHOD("fp8_rmsnorm", fp8_rmsnorm_call),
                                    FP8Q_METHOD("int8_rmsnorm", int8_rmsnorm_call),
                                    FP8Q_METHOD("rmsnorm_backward", rmsnorm_backward_call),
                                    FP8Q_METHOD("moe_route", moe_route_call),
                                    FP8Q_METHOD("moe_route_backward", moe_route_backward_call),
                                    FP8Q_METHOD("fp8_moe_dispatch", moe_dispatch_call),
                                    {nullptr, nullptr, 0, nullptr}};
