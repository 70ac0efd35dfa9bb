// What a list of torch tensors stands for at the moment: address, element
// count, type, device and whether its elements lie one behind the other.
//
// A handle made once of long-lived tensors (GradList) must not act on what they
// were: torch lets a tensor be given other memory, or another size, type or
// order in the same memory, without a trace in the object. Four attributes of
// each tensor, read from Python, cost 0.3 us (200 tensors: 60 us a list); read
// here 0.01 us. The only source that knows torch's C++ types, in a library of
// its own: libnvfp4moe.so needs none.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

constexpr int kWords = 3;                    // int64 of a tensor

// One tensor; false for what is none, or has no memory to point to.
bool look(PyObject* o, int64_t* out) {
  if (!THPVariable_Check(o)) return false;
  try {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined()) return false;
    out[0] = (int64_t)reinterpret_cast<uintptr_t>(t.const_data_ptr());
    out[1] = t.numel();
    out[2] = ((int64_t)t.scalar_type() << 32) | ((int64_t)t.is_contiguous() << 31) |
             ((int64_t)t.device().type() << 16) | (uint16_t)t.device().index();
    return true;
  } catch (...) {                            // no exception may leave a C call
    return false;
  }
}

}  // namespace

// Called with the interpreter's lock held.
extern "C" {

// The words of n tensors of a list into seen[3 n]; 0 if the list is not n tensors.
__attribute__((visibility("default"))) int nvfp4moe_tensors_look(PyObject* list, int64_t* seen,
                                                                 int64_t n) {
  if (!PyList_Check(list) || PyList_GET_SIZE(list) != n) return 0;
  for (int64_t i = 0; i < n; ++i)
    if (!look(PyList_GET_ITEM(list, i), seen + kWords * i)) return 0;
  return 1;
}

// 1 if the list's n tensors are what seen says.
__attribute__((visibility("default"))) int nvfp4moe_tensors_same(PyObject* list, const int64_t* seen,
                                                                 int64_t n) {
  if (!PyList_Check(list) || PyList_GET_SIZE(list) != n) return 0;
  for (int64_t i = 0; i < n; ++i) {
    int64_t w[kWords];
    if (!look(PyList_GET_ITEM(list, i), w)) return 0;
    for (int j = 0; j < kWords; ++j)
      if (w[j] != seen[kWords * i + j]) return 0;
  }
  return 1;
}

}  // extern "C"
