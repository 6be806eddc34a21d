// The torch side of the mixture-of-experts operators: argument checks, output
// tensors and the current stream, then the C calls of dg.h.  dg.py's functions of
// the same names call these; in Python the same checks and allocations take as
// long again as the kernel launch (combine: 7.6 us a call, here 3.8).
#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "dg.h"

namespace {

using at::Tensor;
using c10::ScalarType;

struct Library {
  decltype(&dg_moe_rows) moe_rows;
  decltype(&dg_moe_sort_workspace) moe_sort_workspace;
  decltype(&dg_moe_sort) moe_sort;
  decltype(&dg_moe_permute) moe_permute;
  decltype(&dg_moe_permute_fp8) moe_permute_fp8;
  decltype(&dg_moe_combine) moe_combine;
  decltype(&dg_moe_combine_bwd) moe_combine_bwd;
  decltype(&dg_swiglu_fp8) swiglu_fp8;
  decltype(&dg_swiglu_fp8_bwd) swiglu_fp8_bwd;
  decltype(&dg_grouped_wgrad_fp8) grouped_wgrad_fp8;
} lib;
PyObject* dg_error = nullptr;      // dg.DGError

// ---- arguments ------------------------------------------------------------------

std::string name_of(ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    case at::kByte: return "uint8";
    case at::kFloat8_e4m3fn: return "float8_e4m3fn";
    default: return c10::toString(t);
  }
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// The Python error is set here and passed on by END_HANDLE_TH_ERRORS.
[[noreturn]] void raise(PyObject* type, const std::string& message) {
  PyErr_SetString(type, message.c_str());
  throw python_error();
}
[[noreturn]] void type_error(const std::string& m) { raise(PyExc_TypeError, m); }
[[noreturn]] void value_error(const std::string& m) { raise(PyExc_ValueError, m); }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// `t` is a contiguous tensor on the current device, of one of `dtypes`.
void check(const Tensor& t, const char* name, std::initializer_list<ScalarType> dtypes) {
  bool known = false;
  for (ScalarType d : dtypes) known |= t.scalar_type() == d;
  if (!known) {
    std::string m = std::string(name) + " must be ";
    const char* sep = "";
    for (ScalarType d : dtypes) {
      m += sep + name_of(d);
      sep = " or ";
    }
    type_error(m + ", got " + name_of(t.scalar_type()));
  }
  if (!t.is_cuda() || !t.is_contiguous()) value_error(std::string(name) + " must be a contiguous device tensor");
  if (t.get_device() != c10::hip::current_device())
    value_error(std::string(name) + " is on " + t.device().str() + ", the current device is cuda:" +
                std::to_string(c10::hip::current_device()));
}

void check(const Tensor& t, const char* name, std::initializer_list<ScalarType> dtypes, at::IntArrayRef shape) {
  check(t, name, dtypes);
  if (t.sizes() != shape)
    value_error(std::string(name) + " has shape " + shape_of(t.sizes()) + ", expected " + shape_of(shape));
}

// A matrix of activations; its dg_in_dtype.
int check_values(const Tensor& t, const char* name) {
  if (t.dim() != 2) value_error(std::string(name) + " must be a 2-D tensor");
  check(t, name, {at::kBFloat16, at::kFloat});
  return t.scalar_type() == at::kBFloat16 ? DG_IN_BF16 : DG_IN_F32;
}

// top_k of a plan's map of T tokens.
int check_slots(const Tensor& slot_row, int64_t T) {
  if (slot_row.dim() != 2 || slot_row.size(0) != T || slot_row.size(1) < 1)
    value_error("slot_row has shape " + shape_of(slot_row.sizes()) + ", expected (" + std::to_string(T) + ", top_k)");
  check(slot_row, "slot_row", {at::kInt});
  return int(std::min<int64_t>(slot_row.size(1), INT32_MAX));
}

int64_t check_rows(const Tensor& row_slot) {
  if (row_slot.dim() != 1) value_error("row_slot must be a 1-D tensor");
  check(row_slot, "row_slot", {at::kInt});
  return row_slot.size(0);
}

// A new tensor on `like`'s device (at::empty without its dispatch, 0.3 us).
Tensor create(at::IntArrayRef shape, ScalarType dtype, const Tensor& like) {
  return at::detail::empty_cuda(shape, dtype, like.device(), c10::nullopt);
}

// The output `o`, checked, or a new tensor.  What is written counts as written:
// autograd then sees a saved tensor that has changed.
Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, ScalarType dtype, const Tensor& like) {
  if (o == nullptr || o == Py_None) return create(shape, dtype, like);
  const Tensor& t = tensor(o, name);
  check(t, name, {dtype}, shape);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return t;
}

// Elements from the `at`-th on of `whole`, as a tensor of their own.
Tensor part(const Tensor& whole, int64_t at, at::IntArrayRef sizes) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), whole.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  return t;
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be an integer");
  }
  return v;
}

int small(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
  return int(v);
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

hipStream_t stream() { return c10::hip::getCurrentHIPStream().stream(); }

template <typename T>
T* data(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// ---- results --------------------------------------------------------------------

PyObject* failure(int64_t status, const char* call) {
  PyObject* e = PyObject_CallFunction(dg_error, "Ls", (long long)status, call);
  if (e) {
    PyErr_SetObject(dg_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

template <typename... Ts>
PyObject* tuple(const Ts&... ts) {
  PyObject* r = PyTuple_New(sizeof...(ts));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, wrap(ts)), ...);
  return r;
}

// ---- the operators ----------------------------------------------------------------

// moe_sort(ids, num_groups, align, rows or None)
PyObject* moe_sort(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Tensor& ids = tensor(a[0], "ids");
  if (ids.dim() != 2) value_error("ids must be [T][top_k]");
  check(ids, "ids", {at::kInt, at::kLong});
  const int64_t T = ids.size(0), k = ids.size(1);
  const int G = small(a[1], "num_groups"), align = small(a[2], "align");
  // what the sort would refuse is refused before anything is allocated for it
  int64_t M = k > INT32_MAX ? int64_t(DG_ERR_INVALID_ARG) : lib.moe_rows(T, int(k), G, align);
  if (M < 0) return failure(M, "dg_moe_sort");
  const int64_t ws = lib.moe_sort_workspace(T, int(k), G);
  if (a[3] != Py_None) {
    const int64_t rows = integer(a[3], "rows");
    if (rows < M || rows % align != 0) return failure(DG_ERR_INVALID_ARG, "dg_moe_sort");
    M = rows;
  }
  if (M > INT32_MAX) return failure(DG_ERR_INVALID_ARG, "dg_moe_sort");
  // one allocation for the plan: four cost 2 us more
  const Tensor all = create({2 * int64_t(G) + 1 + M + T * k}, at::kInt, ids);
  const Tensor offs = part(all, 0, {G + 1}), counts = part(all, G + 1, {G});
  const Tensor row_slot = part(all, 2 * int64_t(G) + 1, {M});
  const Tensor slot_row = part(all, 2 * int64_t(G) + 1 + M, {T, k});
  // (the workspace is free for the stream's later work when the call returns)
  const Tensor work = ws ? create({ws}, at::kByte, ids) : Tensor();
  const int st = lib.moe_sort(ids.data_ptr(), ids.scalar_type() == at::kLong ? DG_IDX_I64 : DG_IDX_I32, T, int(k), G,
                              align, M, data<int32_t>(offs), data<int32_t>(counts), data<int32_t>(row_slot),
                              data<int32_t>(slot_row), ws ? work.data_ptr() : nullptr, stream());
  if (st != DG_OK) return failure(st, "dg_moe_sort");
  return tuple(offs, counts, row_slot, slot_row);
  END_HANDLE_TH_ERRORS
}

// moe_permute(X, slot_row, row_slot, Y)
PyObject* moe_permute(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Tensor &X = tensor(a[0], "X"), &slot_row = tensor(a[1], "slot_row"), &row_slot = tensor(a[2], "row_slot");
  const int code = check_values(X, "X");
  const int64_t T = X.size(0), H = X.size(1);
  const int k = check_slots(slot_row, T);
  const int64_t M = check_rows(row_slot);
  const Tensor Y = output(a[3], "Y", {M, H}, X.scalar_type(), X);
  const int st = lib.moe_permute(X.data_ptr(), code, Y.data_ptr(), data<int32_t>(slot_row), data<int32_t>(row_slot), T,
                                 k, M, H, stream());
  if (st != DG_OK) return failure(st, "dg_moe_permute");
  return wrap(Y);
  END_HANDLE_TH_ERRORS
}

// moe_permute_fp8(X, slot_row, row_slot, scale mode, Q, S)
PyObject* moe_permute_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 6);
  const Tensor &X = tensor(a[0], "X"), &slot_row = tensor(a[1], "slot_row"), &row_slot = tensor(a[2], "row_slot");
  const int code = check_values(X, "X"), mode = small(a[3], "scale");
  const int64_t T = X.size(0), H = X.size(1);
  const int k = check_slots(slot_row, T);
  const int64_t M = check_rows(row_slot);
  const Tensor Q = output(a[4], "Q", {M, H}, at::kByte, X);
  const Tensor S = output(a[5], "S", {M, (H + 127) / 128}, at::kFloat, X);
  const int st = lib.moe_permute_fp8(X.data_ptr(), code, Q.data_ptr(), data<float>(S), mode, data<int32_t>(slot_row),
                                     data<int32_t>(row_slot), T, k, M, H, stream());
  if (st != DG_OK) return failure(st, "dg_moe_permute_fp8");
  return tuple(Q, S);
  END_HANDLE_TH_ERRORS
}

// moe_combine(Y, slot_row, weights, out)
PyObject* moe_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Tensor &Y = tensor(a[0], "Y"), &slot_row = tensor(a[1], "slot_row");
  const int code = check_values(Y, "Y");
  const int64_t M = Y.size(0), H = Y.size(1), T = slot_row.dim() > 0 ? slot_row.size(0) : 0;
  const int k = check_slots(slot_row, T);
  const float* w = nullptr;
  if (a[2] != Py_None) {
    const Tensor& weights = tensor(a[2], "weights");
    check(weights, "weights", {at::kFloat}, {T, k});
    w = data<float>(weights);
  }
  const Tensor out = output(a[3], "out", {T, H}, Y.scalar_type(), Y);
  const int st = lib.moe_combine(Y.data_ptr(), code, w, data<int32_t>(slot_row), out.data_ptr(), T, k, M, H, stream());
  if (st != DG_OK) return failure(st, "dg_moe_combine");
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// moe_combine_bwd(dOut, Y, slot_row, row_slot, weights, dY, dweights)
PyObject* moe_combine_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const Tensor &dOut = tensor(a[0], "dOut"), &Y = tensor(a[1], "Y"), &slot_row = tensor(a[2], "slot_row"),
               &row_slot = tensor(a[3], "row_slot"), &weights = tensor(a[4], "weights");
  const int code = check_values(dOut, "dOut");
  const int64_t T = dOut.size(0), H = dOut.size(1);
  const int k = check_slots(slot_row, T);
  const int64_t M = check_rows(row_slot);
  check(Y, "Y", {dOut.scalar_type()}, {M, H});
  check(weights, "weights", {at::kFloat}, {T, k});
  const Tensor dY = output(a[5], "dY", {M, H}, dOut.scalar_type(), dOut);
  const Tensor dw = output(a[6], "dweights", {T, k}, at::kFloat, dOut);
  const int st = lib.moe_combine_bwd(dOut.data_ptr(), Y.data_ptr(), code, data<float>(weights), data<int32_t>(slot_row),
                                     data<int32_t>(row_slot), dY.data_ptr(), data<float>(dw), T, k, M, H, stream());
  if (st != DG_OK) return failure(st, "dg_moe_combine_bwd");
  return tuple(dY, dw);
  END_HANDLE_TH_ERRORS
}

// swiglu_fp8(H, checkpoint)
PyObject* swiglu_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 2);
  const Tensor& H = tensor(a[0], "H");
  const int code = check_values(H, "H");
  const int checkpoint = PyObject_IsTrue(a[1]);
  if (checkpoint < 0) return nullptr;
  if (H.size(1) % 2) value_error("H must have an even number of columns");
  const int64_t M = H.size(0), I = H.size(1) / 2, Ib = (I + 127) / 128;
  const Tensor A = create({M, I}, at::kByte, H);
  Tensor sA, Hq, sH;
  if (checkpoint) {
    // the scales, 1/32 of the codes' bytes, in one allocation (256 rows of 2 x 2048:
    // 6.4 us a call, with two 6.8); codes are of another type, which could not be
    // saved to a file together with scales in the same memory
    const Tensor scales = create({3 * M * Ib}, at::kFloat, H);
    sA = part(scales, 0, {M, Ib});
    sH = part(scales, M * Ib, {M, 2, Ib});
    Hq = create({M, 2 * I}, at::kByte, H);
  } else {
    sA = create({M, Ib}, at::kFloat, H);
  }
  // an empty checkpoint's addresses are null, which would ask for none: no work either way
  const int st = lib.swiglu_fp8(H.data_ptr(), code, A.data_ptr(), data<float>(sA), checkpoint ? Hq.data_ptr() : nullptr,
                                checkpoint ? data<float>(sH) : nullptr, M, I, stream());
  if (st != DG_OK) return failure(st, "dg_swiglu_fp8");
  return tuple(A, sA, Hq, sH);
  END_HANDLE_TH_ERRORS
}

// swiglu_fp8_bwd(dA, Hq, sH, dH)
PyObject* swiglu_fp8_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Tensor &dA = tensor(a[0], "dA"), &Hq = tensor(a[1], "Hq"), &sH = tensor(a[2], "sH");
  const int code = check_values(dA, "dA");
  const int64_t M = dA.size(0), I = dA.size(1);
  check(Hq, "Hq", {at::kByte, at::kFloat8_e4m3fn}, {M, 2 * I});
  check(sH, "sH", {at::kFloat}, {M, 2, (I + 127) / 128});
  const Tensor dH = output(a[3], "dH", {M, 2 * I}, dA.scalar_type(), dA);
  const int st = lib.swiglu_fp8_bwd(dA.data_ptr(), code, Hq.data_ptr(), data<float>(sH), dH.data_ptr(), M, I, stream());
  if (st != DG_OK) return failure(st, "dg_swiglu_fp8_bwd");
  return wrap(dH);
  END_HANDLE_TH_ERRORS
}

// grouped_wgrad_fp8(dY, X, sX, group_offsets, group_counts, out dtype, dW, accumulate)
PyObject* grouped_wgrad_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  const Tensor &dY = tensor(a[0], "dY"), &X = tensor(a[1], "X"), &sX = tensor(a[2], "sX"),
               &offs = tensor(a[3], "group_offsets");
  if (dY.dim() != 2 || X.dim() != 2 || offs.dim() != 1) value_error("dY and X must be 2-D, group_offsets 1-D");
  const int64_t M = dY.size(0), N = dY.size(1), K = X.size(1), G = offs.size(0) - 1;
  check(dY, "dY", {at::kBFloat16});
  check(X, "X", {at::kByte, at::kFloat8_e4m3fn}, {M, K});
  check(sX, "sX", {at::kFloat}, {M, (K + 127) / 128});
  check(offs, "group_offsets", {at::kInt});
  const int32_t* counts = nullptr;
  if (a[4] != Py_None) {
    const Tensor& t = tensor(a[4], "group_counts");
    check(t, "group_counts", {at::kInt}, {G});
    counts = data<int32_t>(t);
  }
  const int out = small(a[5], "out_dtype"), accumulate = PyObject_IsTrue(a[7]);
  if (accumulate < 0) return nullptr;
  if (accumulate && a[6] == Py_None) value_error("accumulate needs dW");
  if (G < 1 || G > INT32_MAX) value_error("group_offsets must have at least two entries");
  const Tensor dW = output(a[6], "dW", {G, N, K}, out == DG_OUT_F32 ? at::kFloat : at::kBFloat16, dY);
  const int st = lib.grouped_wgrad_fp8(dY.data_ptr(), X.data_ptr(), data<float>(sX), data<int32_t>(offs), counts,
                                       int(G), M, N, K, dW.data_ptr(), out, accumulate, stream());
  if (st != DG_OK) return failure(st, "dg_grouped_wgrad_fp8");
  return wrap(dW);
  END_HANDLE_TH_ERRORS
}

// load(path of libdg.so, DGError)
PyObject* load(PyObject*, PyObject* args) {
  const char* path;
  PyObject* error;
  if (!PyArg_ParseTuple(args, "sO", &path, &error)) return nullptr;
  void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  bool all = true;
  auto find = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
    all = all && f;
  };
  find(lib.moe_rows, "dg_moe_rows");
  find(lib.moe_sort_workspace, "dg_moe_sort_workspace");
  find(lib.moe_sort, "dg_moe_sort");
  find(lib.moe_permute, "dg_moe_permute");
  find(lib.moe_permute_fp8, "dg_moe_permute_fp8");
  find(lib.moe_combine, "dg_moe_combine");
  find(lib.moe_combine_bwd, "dg_moe_combine_bwd");
  find(lib.swiglu_fp8, "dg_swiglu_fp8");
  find(lib.swiglu_fp8_bwd, "dg_swiglu_fp8_bwd");
  find(lib.grouped_wgrad_fp8, "dg_grouped_wgrad_fp8");
  if (!all) {
    PyErr_Format(PyExc_RuntimeError, "%s lacks functions of dg.h: build it again", path);
    return nullptr;
  }
  Py_INCREF(error);
  Py_XDECREF(dg_error);
  dg_error = error;
  Py_RETURN_NONE;
}

#define DG_FAST(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"load", load, METH_VARARGS, nullptr},
                         DG_FAST(moe_sort),
                         DG_FAST(moe_permute),
                         DG_FAST(moe_permute_fp8),
                         DG_FAST(moe_combine),
                         DG_FAST(moe_combine_bwd),
                         DG_FAST(swiglu_fp8),
                         DG_FAST(swiglu_fp8_bwd),
                         DG_FAST(grouped_wgrad_fp8),
                         {nullptr, nullptr, 0, nullptr}};
#undef DG_FAST

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dg_torch() { return PyModule_Create(&module); }
