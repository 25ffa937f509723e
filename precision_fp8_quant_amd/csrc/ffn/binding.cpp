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

#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

namespace {

constexpr int64_t kChunk = 16;   // bytes that rows are a multiple of apart

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// A 2-D row-major tensor on `device`; its leading dimension (a single row's is
// its width in whole 16-byte chunks).
bool matrix(const at::Tensor* t, at::Device device, int64_t* ld) {
  if (!t || t->dim() != 2 || t->device() != device || t->layout() != at::kStrided) return false;
  const int64_t rows = t->size(0), cols = t->size(1);
  if (cols > 1 && t->stride(1) != 1) return false;
  *ld = rows > 1 ? t->stride(0) : round_up(cols > 0 ? cols : 1, kChunk / int64_t(t->element_size()));
  return true;
}

bool floats(const at::Tensor* t, at::Device device, at::IntArrayRef shape) {
  return t && t->scalar_type() == at::kFloat && t->device() == device && t->sizes() == shape && t->is_contiguous();
}

bool codes(const at::Tensor* t) {
  return t && (t->scalar_type() == at::kByte || t->scalar_type() == at::kFloat8_e4m3fn);
}

// The library reads rows of 8-bit integers in whole 16-byte chunks.
bool whole_chunks(const at::Tensor& t, int64_t ld) {
  const int64_t rows = t.size(0), cols = t.size(1);
  if (cols % kChunk == 0 || rows == 0) return true;
  return ld % kChunk == 0 &&
         t.storage_offset() + (rows - 1) * ld + round_up(cols, kChunk) <= int64_t(t.storage().nbytes());
}

bool here(const at::Tensor* t) { return t && t->is_cuda() && t->device().index() == c10::hip::current_device(); }

void* stream(at::Device d) { return c10::hip::getCurrentHIPStream(d.index()).stream(); }

// out_code: FP8Q_BF16 or FP8Q_F32.  A new output whose rows are a multiple of
// 16 bytes apart.
at::Tensor output(int64_t rows, int64_t cols, int out_code, at::Device device, int64_t* ld) {
  const auto options = at::TensorOptions().dtype(out_code == FP8Q_BF16 ? at::kBFloat16 : at::kFloat).device(device);
  *ld = round_up(cols > 0 ? cols : 1, out_code == FP8Q_BF16 ? 8 : 4);
  if (*ld == cols) return at::empty({rows, cols}, options);
  return at::empty_strided({rows, cols}, {*ld, 1}, options);
}

// A small non-negative int; -1 for anything else.
int number(PyObject* o) {
  if (!PyLong_CheckExact(o)) return -1;
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  return overflow || v < 0 || v > 255 ? -1 : int(v);
}

PyObject* answer(int status, PyObject* result) {
  if (status == FP8Q_OK) return result;
  Py_XDECREF(result);
  return PyLong_FromLong(status);
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}

// Other threads run while a call allocates and launches: the allocator may wait
// for another thread that holds its lock and wants the interpreter's, and a
// launch for a full queue.  The caller's arguments stay referenced meanwhile.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

#define FP8Q_NONE_UNLESS(cond) \
  do {                         \
    if (!(cond)) Py_RETURN_NONE; \
  } while (0)

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

#define FP8Q_METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fn)), METH_FASTCALL, nullptr}
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
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
