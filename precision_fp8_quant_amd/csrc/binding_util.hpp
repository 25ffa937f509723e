// What the native call paths share: checks of the tensors that come from
// Python, new outputs, and the answer (csrc/ffn/binding.cpp says what a function
// of theirs answers).
#pragma once

#include "../../include/fp8q.h"

#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

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

#define FP8Q_METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fn)), METH_FASTCALL, nullptr}

}  // namespace
