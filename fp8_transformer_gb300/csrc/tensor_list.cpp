// Reads the tensors of a list of gradients into the C table of te_grad_norm and te_clip_grad_norm.  Built
// against the headers of the torch that is installed, into a library of its own, so that the kernels'
// library needs no torch.
//
// A tensor can change its address, size, type or strides between two calls (resize_, a new .data), some of
// them without the others, so each call reads them all: 4 us for 580 tensors, where four attributes of each
// take 110 us from Python.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "te_gb300.h"

namespace {

// A dense float32 or bfloat16 tensor; false for anything else.
bool read(PyObject* o, const at::TensorBase** t, int32_t* dtype) {
  if (!THPVariable_Check(o)) return false;
  const at::TensorBase& v = THPVariable_Unpack(o);
  if (!v.defined() || !(v.is_cuda() || v.is_cpu()) || v.layout() != at::kStrided || !v.has_storage() || !v.is_contiguous()) return false;
  if (v.scalar_type() == at::kFloat) *dtype = TE_F32;
  else if (v.scalar_type() == at::kBFloat16) *dtype = TE_BF16;
  else return false;
  *t = &v;
  return true;
}

}  // namespace

// grads: a list of n tensors; outs: another, or None.  Fills table (n entries) and *device (the first tensor's
// index, -1 on the CPU, left alone by an empty list) and returns -1, or the place of the first entry that is not a
// dense float32 / bfloat16 tensor on that device with an out of its shape and type, or n where these are no such lists.
extern "C" int64_t te_read_grads(PyObject* grads, PyObject* outs, int64_t n, te_grad* table, int64_t* device) {
  auto holds = [n](PyObject* o) { return PyList_Check(o) && PyList_GET_SIZE(o) == n; };
  int64_t i = 0;
  try {
    if (n == 0 && !(holds(grads) && (outs == Py_None || holds(outs)))) return n;
    for (; i < n; ++i) {
      if (!holds(grads) || !(outs == Py_None || holds(outs))) return n;  // (a type's own check may run Python)
      const at::TensorBase *g = nullptr, *o = nullptr;
      int32_t dtype = 0, out_dtype = 0;
      if (!read(PyList_GET_ITEM(grads, i), &g, &dtype)) return i;
      if (i == 0) *device = g->is_cuda() ? g->get_device() : -1;
      if ((g->is_cuda() ? g->get_device() : -1) != *device) return i;
      table[i].data = g->unsafeGetTensorImpl()->mutable_data();
      table[i].out = nullptr;
      table[i].numel = g->numel();
      table[i].dtype = dtype;
      if (outs == Py_None) continue;
      if (!read(PyList_GET_ITEM(outs, i), &o, &out_dtype) || out_dtype != dtype || o->device() != g->device() ||
          o->sizes() != g->sizes())
        return i;
      table[i].out = o->unsafeGetTensorImpl()->mutable_data();
    }
  } catch (...) {  // a tensor without memory of its own
    return i;
  }
  return -1;
}
