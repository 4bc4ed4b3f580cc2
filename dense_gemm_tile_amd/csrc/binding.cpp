// CPython calls of the layer operators' entry points (include/gemm_layer.h).
//
// A decoding step calls them for a few microseconds of GPU work each, so what
// the interpreter adds to a call counts: converting the arguments here takes
// about a third of the time that ctypes takes for them. Each function takes the
// entry point's arguments by position and returns its status code:
//   tensors   anything with data_ptr(), an integer address, or None for NULL
//   stream    anything with cuda_stream, an integer handle, or None for NULL
//   dtype     a code, or one of the names below (KeyError for another name);
//   act       the same, as is score
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <tuple>
#include <type_traits>
#include <utility>

#include "gemm_layer.h"

namespace {

struct Name {
  const char* name;
  int code;
};
constexpr Name kDtypes[] = {{"f16", GEMM_DTYPE_F16},       {"bf16", GEMM_DTYPE_BF16},
                            {"f32", GEMM_DTYPE_F32},       {"f32_f16", GEMM_DTYPE_F32_F16},
                            {"f32_bf16", GEMM_DTYPE_F32_BF16}, {"f8e4m3", GEMM_DTYPE_F8_E4M3},
                            {"f8e5m2", GEMM_DTYPE_F8_E5M2}};
constexpr Name kActs[] = {{"none", GEMM_ACT_NONE},
                          {"relu", GEMM_ACT_RELU},
                          {"gelu", GEMM_ACT_GELU},
                          {"gelu_erf", GEMM_ACT_GELU_ERF},
                          {"silu", GEMM_ACT_SILU}};
constexpr Name kScores[] = {{"softmax", GEMM_SCORE_SOFTMAX}, {"sigmoid", GEMM_SCORE_SIGMOID}};
// What a parameter holds, where its C type does not say.
struct Dtype {
  int code;
  operator int() const { return code; }
};
struct Act {
  int code;
  operator int() const { return code; }
};
struct Score {
  int code;
  operator int() const { return code; }
};
struct Stream {
  void* handle;
  operator void*() const { return handle; }
};

PyObject* g_data_ptr;     // interned attribute names
PyObject* g_cuda_stream;

bool convert(PyObject* o, int64_t& v) {
  v = PyLong_AsLongLong(o);
  return v != -1 || !PyErr_Occurred();
}
bool convert(PyObject* o, int& v) {
  int64_t w;
  if (!convert(o, w)) return false;
  if (w < INT32_MIN || w > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "value does not fit a C int");
    return false;
  }
  v = (int)w;
  return true;
}
template <size_t n>
bool convert_name(PyObject* o, const Name (&names)[n], int& v) {
  if (!PyUnicode_Check(o)) return convert(o, v);
  for (const Name& x : names)
    if (PyUnicode_CompareWithASCIIString(o, x.name) == 0) {
      v = x.code;
      return true;
    }
  PyErr_SetObject(PyExc_KeyError, o);
  return false;
}
bool convert(PyObject* o, Dtype& v) { return convert_name(o, kDtypes, v.code); }
bool convert(PyObject* o, Act& v) { return convert_name(o, kActs, v.code); }
bool convert(PyObject* o, Score& v) { return convert_name(o, kScores, v.code); }
bool convert(PyObject* o, float& v) {
  const double d = PyFloat_AsDouble(o);
  v = (float)d;
  return d != -1.0 || !PyErr_Occurred();
}
bool convert_address(PyObject* o, void*& v) {
  v = PyLong_AsVoidPtr(o);
  return v || !PyErr_Occurred();
}
bool convert_owned(PyObject* o, void*& v) {  // takes over a reference; null: an error is set
  if (!o) return false;
  const bool ok = convert_address(o, v);
  Py_DECREF(o);
  return ok;
}
bool convert(PyObject* o, Stream& v) {
  v.handle = nullptr;
  if (o == Py_None) return true;
  if (PyLong_Check(o)) return convert_address(o, v.handle);
  return convert_owned(PyObject_GetAttr(o, g_cuda_stream), v.handle);
}
template <class T>
bool convert(PyObject* o, T*& v) {
  void* p = nullptr;
  if (o != Py_None) {
    if (!(PyLong_Check(o) ? convert_address(o, p)
                          : convert_owned(PyObject_CallMethodNoArgs(o, g_data_ptr), p)))
      return false;
  }
  v = static_cast<T*>(p);
  return true;
}

// F called with arguments converted to P..., which the entry point's own
// parameter types accept.
template <auto F, class... P>
struct Call {
  template <size_t... i>
  static PyObject* call(PyObject* const* args, std::index_sequence<i...>) {
    std::tuple<P...> v;
    if (!(convert(args[i], std::get<i>(v)) && ...)) return nullptr;
    int64_t r;
    Py_BEGIN_ALLOW_THREADS
    r = (int64_t)F(std::get<i>(v)...);
    Py_END_ALLOW_THREADS
    return PyLong_FromLongLong(r);
  }
  static PyObject* run(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != (Py_ssize_t)sizeof...(P))
      return PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd",
                          (Py_ssize_t)sizeof...(P), n);
    return call(args, std::index_sequence_for<P...>{});
  }
};

using I = int64_t;
using In = const void*;
using Out = void*;
template <class C>
PyMethodDef entry(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(C::run)), METH_FASTCALL,
          nullptr};
}

PyMethodDef g_methods[] = {
    entry<Call<gemm_linear, I, I, I, Dtype, int, int, In, I, In, I, In, Act, In, I, Out, I, Dtype,
               Out, I, Stream>>("gemm_linear"),
    entry<Call<gemm_grouped, I, I, I, I, Dtype, int, const int32_t*, In, I, In, I, I, In, Act, In,
               I, Out, I, Dtype, Out, I, Stream>>("gemm_grouped"),
    entry<Call<gemm_grouped_grad_weight, I, I, I, I, Dtype, const int32_t*, In, I, In, I, Out, I, I,
               Dtype, int, Stream>>("gemm_grouped_grad_weight"),
    entry<Call<gemm_act_grad, I, I, I, Dtype, Act, const int32_t*, In, I, In, I, Out, I, float*,
               Out, I, Stream>>("gemm_act_grad"),
    entry<Call<gemm_act_grad_workspace, I, I, I>>("gemm_act_grad_workspace"),
    entry<Call<gemm_route, I, I, I, const int32_t*, int32_t*, int32_t*, int32_t*, Out, I, Stream>>(
        "gemm_route"),
    entry<Call<gemm_route_workspace, I, I, I>>("gemm_route_workspace"),
    entry<Call<gemm_dispatch, I, I, I, Dtype, In, I, const int32_t*, Out, I, Stream>>(
        "gemm_dispatch"),
    entry<Call<gemm_combine, I, I, I, Dtype, In, I, const int32_t*, const float*, In, I, Out, I,
               Stream>>("gemm_combine"),
    entry<Call<gemm_combine_grad, I, I, I, Dtype, In, I, In, I, const int32_t*, const float*, Out,
               I, float*, Stream>>("gemm_combine_grad"),
    entry<Call<gemm_norm, I, I, Dtype, In, I, In, In, float, Out, I, float*, float*, Stream>>("gemm_norm"),
    entry<Call<gemm_norm_grad, I, I, Dtype, In, I, In, I, In, const float*, const float*, In, I, Out, I, float*,
               float*, Out, I, Stream>>("gemm_norm_grad"),
    entry<Call<gemm_norm_grad_workspace, I, I>>("gemm_norm_grad_workspace"),
    entry<Call<gemm_gate, I, I, I, Dtype, In, I, Score, const float*, I, I, I, int, float, int32_t*, float*,
               Stream>>("gemm_gate"),
    entry<Call<gemm_gate_grad, I, I, I, Dtype, In, I, Score, int, float, const int32_t*, const float*, Out, I,
               Stream>>("gemm_gate_grad"),
    entry<Call<gemm_linear_w4, I, I, I, Dtype, In, I, In, I, In, In, I, I, In, Act, In, I, Out, I, Dtype,
               Stream>>("gemm_linear_w4"),
    entry<Call<gemm_grouped_w4, I, I, I, I, Dtype, const int32_t*, In, I, In, I, I, In, In, I, I, I, In, Act, In, I,
               Out, I, Dtype, Stream>>("gemm_grouped_w4"),
    entry<Call<gemm_loss, I, I, I, Dtype, In, I, In, I, const int32_t*, float*, float*, Out, I, Stream>>("gemm_loss"),
    entry<Call<gemm_loss_workspace, I, I, I>>("gemm_loss_workspace"),
    entry<Call<gemm_loss_grad, I, I, I, Dtype, In, I, In, I, const int32_t*, const float*, const float*, Out, I, Out,
               I, Dtype, int, Out, I, Stream>>("gemm_loss_grad"),
    entry<Call<gemm_loss_grad_workspace, I, I, I>>("gemm_loss_grad_workspace"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding",
                        "Calls of the layer operators' entry points.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  g_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!g_data_ptr || !g_cuda_stream) return nullptr;
  return PyModule_Create(&g_module);
}
