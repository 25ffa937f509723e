// The usual call of a gated feed-forward operator from Python, in one native
// step: new outputs, the current stream of the current device.  Tensors are
// checked, outputs allocated and the C ABI (include/fp8q_ffn.h) called without
// an interpreted line in between, because a caller with few tokens waits for
// the host: a small int8_gemm call takes 4.5 us, of which the launch itself is
// 3, and 8.2 through ctypes.
//
// A function here answers None when anything is not as it expects; ffn.py then
// takes the call its own way, with the message that says what is wrong.  It
// answers an int, the status, when the C ABI refuses the call.
#include "../../../include/fp8q_ffn.h"

#include "../binding_util.hpp"

#include <torch/version.h>

// csrc/front/binding.cpp
extern PyMethodDef fp8q_front_methods[];

namespace {

// int8_gemm(a, a_scales, b, b_scales, bias or None, out code)
PyObject* int8_gemm_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  FP8Q_NONE_UNLESS(n == 6);
  const at::Tensor *a = tensor(args[0]), *sa = tensor(args[1]), *b = tensor(args[2]), *sb = tensor(args[3]);
  const at::Tensor* bias = args[4] == Py_None ? nullptr : tensor(args[4]);
  const int out = number(args[5]);
  FP8Q_NONE_UNLESS(here(a) && b && (args[4] == Py_None || bias) && (out == FP8Q_BF16 || out == FP8Q_F32));
  const at::Device dev = a->device();
  int64_t lda, ldb, ldc;
  FP8Q_NONE_UNLESS(a->scalar_type() == at::kChar && b->scalar_type() == at::kChar && matrix(a, dev, &lda) &&
                   matrix(b, dev, &ldb) && a->size(1) == b->size(1) && whole_chunks(*a, lda) && whole_chunks(*b, ldb));
  const int64_t m = a->size(0), rows = b->size(0), k = a->size(1);
  FP8Q_NONE_UNLESS(floats(sa, dev, {m}) && floats(sb, dev, {rows}) && (!bias || floats(bias, dev, {rows})));
  at::Tensor c;
  int st;
  {
    Unlocked others_run;
    c = output(m, rows, out, dev, &ldc);
    st = int8_gemm(m, rows, k, static_cast<const int8_t*>(a->data_ptr()), lda, static_cast<const float*>(sa->data_ptr()),
                   static_cast<const int8_t*>(b->data_ptr()), ldb, static_cast<const float*>(sb->data_ptr()),
                   bias ? static_cast<const float*>(bias->data_ptr()) : nullptr, c.data_ptr(), out, ldc, stream(dev));
  }
  return answer(st, THPVariable_Wrap(c));
  END_HANDLE_TH_ERRORS
}

// int8_gemm_gated(a, a_scales, b, b_scales, act, out code)
PyObject* int8_gated_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  FP8Q_NONE_UNLESS(n == 6);
  const at::Tensor *a = tensor(args[0]), *sa = tensor(args[1]), *b = tensor(args[2]), *sb = tensor(args[3]);
  const int act = number(args[4]), out = number(args[5]);
  FP8Q_NONE_UNLESS(here(a) && b && act >= 0 && (out == FP8Q_BF16 || out == FP8Q_F32));
  const at::Device dev = a->device();
  int64_t lda, ldb, ldh;
  FP8Q_NONE_UNLESS(a->scalar_type() == at::kChar && b->scalar_type() == at::kChar && matrix(a, dev, &lda) &&
                   matrix(b, dev, &ldb) && a->size(1) == b->size(1) && whole_chunks(*a, lda) && whole_chunks(*b, ldb));
  const int64_t m = a->size(0), rows = b->size(0), k = a->size(1);
  FP8Q_NONE_UNLESS(rows % 2 == 0 && floats(sa, dev, {m}) && floats(sb, dev, {rows}));
  at::Tensor h;
  int st;
  {
    Unlocked others_run;
    h = output(m, rows / 2, out, dev, &ldh);
    st = int8_gemm_gated(act, m, rows / 2, k, static_cast<const int8_t*>(a->data_ptr()), lda,
                         static_cast<const float*>(sa->data_ptr()), static_cast<const int8_t*>(b->data_ptr()), ldb,
                         static_cast<const float*>(sb->data_ptr()), h.data_ptr(), out, ldh, stream(dev));
  }
  return answer(st, THPVariable_Wrap(h));
  END_HANDLE_TH_ERRORS
}

// int8_quant_rows(x)
PyObject* int8_quant_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  FP8Q_NONE_UNLESS(n == 1);
  const at::Tensor* x = tensor(args[0]);
  FP8Q_NONE_UNLESS(here(x) && (x->scalar_type() == at::kBFloat16 || x->scalar_type() == at::kFloat));
  const at::Device dev = x->device();
  int64_t ldx;
  FP8Q_NONE_UNLESS(matrix(x, dev, &ldx));
  const int64_t rows = x->size(0), cols = x->size(1), ldq = round_up(cols > 0 ? cols : 1, kChunk);
  at::Tensor q, scales;
  int st;
  {
    Unlocked others_run;
    // the last row's bytes up to 16 exist too, as int8_gemm reads them
    q = at::empty({rows, ldq}, at::TensorOptions().dtype(at::kChar).device(dev));
    if (ldq != cols) q = q.as_strided({rows, cols}, {ldq, 1});
    scales = at::empty({rows}, at::TensorOptions().dtype(at::kFloat).device(dev));
    st = int8_quant_rows(x->data_ptr(), x->scalar_type() == at::kBFloat16 ? FP8Q_BF16 : FP8Q_F32, rows, cols, ldx,
                         static_cast<int8_t*>(q.data_ptr()), ldq, static_cast<float*>(scales.data_ptr()), stream(dev));
  }
  return answer(st, pair(q, scales));
  END_HANDLE_TH_ERRORS
}

// fp8_gemm_gated(a, a_scales, b, b_scales, act, out code, whether gate and up are kept)
PyObject* fp8_gated_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  FP8Q_NONE_UNLESS(n == 7);
  const at::Tensor *a = tensor(args[0]), *sa = tensor(args[1]), *b = tensor(args[2]), *sb = tensor(args[3]);
  const int act = number(args[4]), out = number(args[5]);
  const bool keep = args[6] == Py_True;
  FP8Q_NONE_UNLESS(here(a) && codes(a) && codes(b) && (keep || args[6] == Py_False) && act >= 0 &&
                   (out == FP8Q_BF16 || out == FP8Q_F32));
  const at::Device dev = a->device();
  int64_t lda, ldb, ldh, ldgu = 0;
  FP8Q_NONE_UNLESS(matrix(a, dev, &lda) && matrix(b, dev, &ldb) && a->size(1) == b->size(1));
  const int64_t m = a->size(0), rows = b->size(0), k = a->size(1), kg = (k + 127) / 128;
  FP8Q_NONE_UNLESS(rows % 2 == 0 && floats(sa, dev, {kg, m}) && floats(sb, dev, {(rows + 127) / 128, kg}));
  at::Tensor h, gu;
  int st;
  {
    Unlocked others_run;
    h = output(m, rows / 2, out, dev, &ldh);
    if (keep) gu = output(m, rows, out, dev, &ldgu);
    st = fp8_gemm_gated(act, m, rows / 2, k, static_cast<const uint8_t*>(a->data_ptr()), lda,
                        static_cast<const float*>(sa->data_ptr()), static_cast<const uint8_t*>(b->data_ptr()), ldb,
                        static_cast<const float*>(sb->data_ptr()), h.data_ptr(), out, ldh,
                        keep ? gu.data_ptr() : nullptr, ldgu, stream(dev));
  }
  return answer(st, keep ? pair(h, gu) : THPVariable_Wrap(h));
  END_HANDLE_TH_ERRORS
}

// fp8_gated_backward(dh, gu, act, mode)
PyObject* gated_backward_call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS                               // C++ exceptions become the interpreter's
  FP8Q_NONE_UNLESS(n == 4);
  const at::Tensor *dh = tensor(args[0]), *gu = tensor(args[1]);
  const int act = number(args[2]), mode = number(args[3]);
  FP8Q_NONE_UNLESS(here(dh) && gu && act >= 0 && mode >= 0 && gu->scalar_type() == dh->scalar_type() &&
                   (dh->scalar_type() == at::kBFloat16 || dh->scalar_type() == at::kFloat));
  const at::Device dev = dh->device();
  int64_t ld_dh, ld_gu;
  FP8Q_NONE_UNLESS(matrix(dh, dev, &ld_dh) && matrix(gu, dev, &ld_gu));
  const int64_t m = dh->size(0), f = dh->size(1), f2 = 2 * f, mp = round_up(m, 128);
  FP8Q_NONE_UNLESS(gu->size(0) == m && gu->size(1) == f2 && f % 128 == 0);
  const auto bytes = at::TensorOptions().dtype(at::kByte).device(dev);
  const auto reals = at::TensorOptions().dtype(at::kFloat).device(dev);
  at::Tensor q, s, qt, st;
  int status;
  {
    Unlocked others_run;
    q = at::empty({mp, f2}, bytes);
    s = at::empty({f2 / 128, mp}, reals);
    qt = at::empty({f2, mp}, bytes);
    st = at::empty({mp / 128, f2}, reals);
    status = fp8_gated_backward(
        act, m, f, dh->data_ptr(), ld_dh, gu->data_ptr(), ld_gu,
        dh->scalar_type() == at::kBFloat16 ? FP8Q_BF16 : FP8Q_F32, mode, static_cast<uint8_t*>(q.data_ptr()), f2,
        static_cast<float*>(s.data_ptr()), static_cast<uint8_t*>(qt.data_ptr()), mp > 0 ? mp : 16,
        static_cast<float*>(st.data_ptr()), nullptr, 0, stream(dev));
  }
  if (status != FP8Q_OK) return PyLong_FromLong(status);
  PyObject* t = PyTuple_New(4);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(q));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(s));
  PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(qt));
  PyTuple_SET_ITEM(t, 3, THPVariable_Wrap(st));
  return t;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {FP8Q_METHOD("int8_gemm", int8_gemm_call),
                         FP8Q_METHOD("int8_gemm_gated", int8_gated_call),
                         FP8Q_METHOD("int8_quant_rows", int8_quant_call),
                         FP8Q_METHOD("fp8_gemm_gated", fp8_gated_call),
                         FP8Q_METHOD("fp8_gated_backward", gated_backward_call),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ffn_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: what the tensors' layout was compiled for; ffn.py compares it.
PyMODINIT_FUNC PyInit__ffn_call(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && (PyModule_AddFunctions(m, fp8q_front_methods) < 0 ||
            PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0))
    Py_CLEAR(m);
  return m;
}
