// torch_calls.cpp -- the calls of fp32_gemm_amd/grouped.py: checks tensors,
// turns them into pointers and leading dimensions and calls the C ABI of
// include/grouped_gemm.h on a stream.  In Python the same takes longer than the
// small products themselves (a grouped product: 8.9 us a call, so 3.8, of
// which the launch takes 3.6).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/grouped_gemm.h"

namespace {

constexpr int kI8 = 3;
enum Allowed { kFloats, kInt8 };

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

int code_of(const at::Tensor& t, const char* name, Allowed allowed) {
  const auto type = t.scalar_type();
  if (allowed == kInt8) {
    if (type == at::kChar) return kI8;
    refuse(PyExc_TypeError, std::string(name) + " must be torch.int8, got " + c10::toString(type));
  }
  if (type == at::kFloat) return GEMM_F32;
  if (type == at::kBFloat16) return GEMM_BF16;
  if (type == at::kHalf) return GEMM_F16;
  refuse(PyExc_TypeError, std::string(name) + " must be torch.float32, torch.bfloat16 or torch.float16, got " +
                              c10::toString(type));
}

// On GPU `dev`, which the first operand (dev < 0) sets.
void on_device(const at::Tensor& t, const char* name, int& dev) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be on a GPU device");
  if (dev < 0) dev = t.get_device();
  else if (t.get_device() != dev) refuse(PyExc_ValueError, std::string(name) + " is on another device");
}

struct Operand {
  int code = 0;
  char* data = nullptr;
  int64_t groups = 1, rows = 0, cols = 0, ld = 1, stride = 0;
};

// A matrix with unit column stride, or a stack of them.
Operand operand(PyObject* o, const char* name, Allowed allowed, bool stack, int& dev) {
  const at::Tensor& t = tensor(o, name);
  Operand r;
  r.code = code_of(t, name, allowed);
  if (t.dim() != (stack ? 3 : 2))
    refuse(PyExc_ValueError, std::string(name) + (stack ? " must be 3-D (experts, rows, columns) when offsets are given"
                                                        : " must be 2-D"));
  on_device(t, name, dev);
  const auto size = t.sizes(), step = t.strides();
  const int at = stack ? 1 : 0;
  r.rows = size[at];
  r.cols = size[at + 1];
  if (stack) {
    r.groups = size[0];
    if (r.groups == 0) refuse(PyExc_ValueError, std::string(name) + " holds no expert");
    r.stride = r.groups > 1 ? step[0] : 0;
  }
  if (r.cols > 1 && step[at + 1] != 1)
    refuse(PyExc_ValueError, std::string(name) + " must have unit column stride (row-major)");
  r.ld = r.cols > 1 ? r.cols : 1;
  if (r.rows > 1) {
    if (step[at] < r.cols)
      refuse(PyExc_ValueError, std::string(name) + ": rows overlap (row stride " + std::to_string(step[at]) + " < " +
                                   std::to_string(r.cols) + " columns)");
    r.ld = step[at] > 1 ? step[at] : 1;
  }
  r.data = static_cast<char*>(t.data_ptr());
  return r;
}

const int32_t* group_offsets(PyObject* o, int64_t groups, int dev) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).scalar_type() != at::kInt)
    refuse(PyExc_TypeError, "offsets must be an int32 torch.Tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != 1 || t.size(0) != groups + 1 || t.stride(0) != 1)
    refuse(PyExc_ValueError, "offsets must be " + std::to_string(groups + 1) + " consecutive row numbers for " +
                                 std::to_string(groups) + " experts");
  if (!t.is_cuda() || t.get_device() != dev) refuse(PyExc_ValueError, "offsets must be on the operands' device");
  return static_cast<const int32_t*>(t.data_ptr());
}

// Contiguous floats: n of them, or groups x n.
float* scales(PyObject* o, const char* name, bool grouped, int64_t groups, int64_t n, int dev) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).scalar_type() != at::kFloat)
    refuse(PyExc_TypeError, std::string(name) + " must be a float32 torch.Tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  const bool fits = grouped ? t.dim() == 2 && t.size(0) == groups && t.size(1) == n : t.dim() == 1 && t.size(0) == n;
  if (!fits || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be contiguous with shape (" +
                                 (grouped ? std::to_string(groups) + ", " : "") + std::to_string(n) +
                                 (grouped ? ")" : ",)"));
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(PyExc_ValueError, std::string(name) + " must be on the operands' device");
  return static_cast<float*>(t.data_ptr());
}

std::string shape(const char* name, const Operand& o, bool stack) {
  return std::string(name) + " (" + (stack ? std::to_string(o.groups) + ", " : "") + std::to_string(o.rows) + ", " +
         std::to_string(o.cols) + ")";
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return static_cast<float>(v);
}

// torch's current stream, a torch stream, or a handle.
void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(dev)).stream();
  PyObject* held = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : nullptr;
  void* handle = PyLong_AsVoidPtr(held ? held : o);
  Py_XDECREF(held);
  if (handle == nullptr && PyErr_Occurred()) throw Refused{};
  return handle;
}

// Makes `dev` the current device for the call.
struct On {
  c10::DeviceIndex was;
  bool changed;
  explicit On(int dev) : was(c10::hip::current_device()), changed(was != dev) {
    if (changed) c10::hip::set_device(static_cast<c10::DeviceIndex>(dev));
  }
  ~On() {
    if (changed) c10::hip::set_device(was);
  }
};

// Runs a call's body; its status comes back as an integer.
template <class F>
PyObject* status(Py_ssize_t given, Py_ssize_t wanted, F body) {
  try {
    if (given != wanted) refuse(PyExc_TypeError, "wrong number of arguments");
    return PyLong_FromLong(body());
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

void out_type(const Operand& in, const Operand& out, const char* name) {
  if (out.code != in.code && out.code != GEMM_F32)
    refuse(PyExc_TypeError, std::string(name) + " must have the operands' type or be float32");
}

// X, W, offsets, Y, alpha, beta, transpose_w, stream
PyObject* call_grouped(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return status(n, 8, [&] {
    int dev = -1;
    const bool grouped = v[2] != Py_None;
    const Operand x = operand(v[0], "X", kFloats, false, dev), w = operand(v[1], "W", kFloats, grouped, dev),
                  y = operand(v[3], "Y", kFloats, false, dev);
    const int trans = PyObject_IsTrue(v[6]);
    if (trans < 0) throw Refused{};
    if (w.code != x.code) refuse(PyExc_TypeError, "X and W must have the same type");
    out_type(x, y, "Y");
    const int64_t depth = trans ? w.cols : w.rows, width = trans ? w.rows : w.cols;
    if (depth != x.cols || y.rows != x.rows || y.cols != width)
      refuse(PyExc_ValueError, "shape mismatch: " + shape("X", x, false) + ", " + shape("W", w, grouped) + ", " +
                                   shape("Y", y, false));
    const int32_t* offsets = group_offsets(v[2], w.groups, dev);
    const float alpha = number(v[4]), beta = number(v[5]);
    void* const stream = stream_of(v[7], dev);
    On on(dev);
    return gemm_grouped(x.code, y.code, trans, static_cast<int32_t>(w.groups), offsets, x.rows, width, depth, alpha,
                        x.data, x.ld, w.data, w.ld, w.stride, beta, y.data, y.ld, stream);
  });
}

// X, dY, offsets, dW, alpha, beta, stream
PyObject* call_wgrad(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return status(n, 7, [&] {
    int dev = -1;
    const bool grouped = v[2] != Py_None;
    const Operand x = operand(v[0], "X", kFloats, false, dev), dy = operand(v[1], "dY", kFloats, false, dev),
                  dw = operand(v[3], "dW", kFloats, grouped, dev);
    if (dy.code != x.code) refuse(PyExc_TypeError, "X and dY must have the same type");
    out_type(x, dw, "dW");
    if (dy.rows != x.rows || dw.rows != x.cols || dw.cols != dy.cols)
      refuse(PyExc_ValueError, "shape mismatch: " + shape("X", x, false) + ", " + shape("dY", dy, false) + ", " +
                                   shape("dW", dw, grouped));
    const int32_t* offsets = group_offsets(v[2], dw.groups, dev);
    const float alpha = number(v[4]), beta = number(v[5]);
    void* const stream = stream_of(v[6], dev);
    On on(dev);
    return gemm_grouped_wgrad(x.code, dw.code, static_cast<int32_t>(dw.groups), offsets, x.rows, dy.cols, x.cols,
                              alpha, x.data, x.ld, dy.data, dy.ld, beta, dw.data, dw.ld, dw.stride, stream);
  });
}

// X, Q, scale, stream
PyObject* call_quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return status(n, 4, [&] {
    int dev = -1;
    const Operand x = operand(v[0], "X", kFloats, false, dev), q = operand(v[1], "Q", kInt8, false, dev);
    if (q.rows != x.rows || q.cols != x.cols)
      refuse(PyExc_ValueError, "shape mismatch: " + shape("X", x, false) + ", " + shape("Q", q, false));
    float* const scale = scales(v[2], "scale", false, 1, x.rows, dev);
    void* const stream = stream_of(v[3], dev);
    On on(dev);
    return quantize_rows(x.code, x.rows, x.cols, x.data, x.ld, reinterpret_cast<int8_t*>(q.data), q.ld, scale,
                         stream);
  });
}

// A, scale_a, B, scale_b, C, bias, offsets, stream
PyObject* call_igemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return status(n, 8, [&] {
    int dev = -1;
    const bool grouped = v[6] != Py_None;
    const Operand a = operand(v[0], "A", kInt8, false, dev), b = operand(v[2], "B", kInt8, grouped, dev),
                  c = operand(v[4], "C", kFloats, false, dev);
    if (b.cols != a.cols || c.rows != a.rows || c.cols != b.rows)
      refuse(PyExc_ValueError, "shape mismatch: " + shape("A", a, false) + ", " + shape("B", b, grouped) + ", " +
                                   shape("C", c, false));
    const int32_t* offsets = group_offsets(v[6], b.groups, dev);
    const float* scale_a = scales(v[1], "scale_a", false, 1, a.rows, dev);
    const float* scale_b = scales(v[3], "scale_b", grouped, b.groups, b.rows, dev);
    const float* bias = v[5] == Py_None ? nullptr : scales(v[5], "bias", grouped, b.groups, b.rows, dev);
    void* const stream = stream_of(v[7], dev);
    On on(dev);
    return igemm(c.code, static_cast<int32_t>(b.groups), offsets, a.rows, b.rows, a.cols,
                 reinterpret_cast<const int8_t*>(a.data), a.ld, scale_a, reinterpret_cast<const int8_t*>(b.data), b.ld,
                 b.stride, scale_b, bias, c.data, c.ld, stream);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef kMethods[] = {
    {"gemm_grouped", fast<call_grouped>(), METH_FASTCALL, nullptr},
    {"gemm_grouped_wgrad", fast<call_wgrad>(), METH_FASTCALL, nullptr},
    {"quantize_rows", fast<call_quantize>(), METH_FASTCALL, nullptr},
    {"igemm", fast<call_igemm>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch's C++ interface differs between versions: only the one this was
// compiled against may load it.
PyMODINIT_FUNC PyInit__torch_calls() {
  PyObject* const torch = PyImport_ImportModule("torch");
  PyObject* const held = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  PyObject* const version = held ? PyObject_Str(held) : nullptr;
  const char* const text = version ? PyUnicode_AsUTF8(version) : nullptr;
  const bool same = text && std::string(text) == BUILT_FOR_TORCH;
  if (text && !same)
    PyErr_Format(PyExc_ImportError, "built for torch " BUILT_FOR_TORCH ", this is torch %s", text);
  Py_XDECREF(version);
  Py_XDECREF(held);
  Py_XDECREF(torch);
  return same ? PyModule_Create(&kModule) : nullptr;
}
