// The plain case of the routing, dispatch, combine and 4-bit calls without the
// interpreter: tensors on the current device, contiguous and of the right types and
// sizes, outputs and workspace allocated here.  Anything else (other arguments, a
// non-zero status) returns None, and the Python function of the same name checks,
// converts, calls and reports.  A decoded token's kernels run for a few microseconds,
// so the host's share of a call counts: a small combine's call takes it 4.9 us, of them
// 2.9 the launch, and 8.9 through the interpreter; one token's routing 9.0 and 14.1.
//
// The library's entry points are handed over as addresses (bind), so this file links
// against no particular copy of it.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include "../../include/fp8_moe_grouped.h"

namespace {

using at::Tensor;

#define CALLS(X)                                                                                                 \
  X(moe_route) X(moe_route_bwd) X(moe_permute) X(moe_permute_fp8) X(moe_combine) X(moe_combine_bwd)               \
  X(quantize_mxfp4_weights) X(dequantize_mxfp4) X(gmm_mxfp4_fwd) X(gmm_silu_mxfp4) X(fp8gmm_workspace_bytes)

struct Library {
#define X(name) decltype(&::name) name = nullptr;
  CALLS(X)
#undef X
} lib;

// bind(address, ...) in the order of CALLS
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Py_ssize_t i = 0;
#define X(name)                                                                          \
  {                                                                                      \
    void* p = i < n ? PyLong_AsVoidPtr(args[i]) : nullptr;                               \
    if (PyErr_Occurred()) return nullptr;                                                \
    lib.name = reinterpret_cast<decltype(&::name)>(p);                                   \
    ++i;                                                                                 \
  }
  CALLS(X)
#undef X
  Py_RETURN_NONE;
}

PyObject* names(PyObject*, PyObject*) {
  return Py_BuildValue("["
#define X(name) "s"
                       CALLS(X)
#undef X
                       "]"
#define X(name) , #name
                       CALLS(X)
#undef X
  );
}

constexpr auto kF32 = at::kFloat, kBf16 = at::kBFloat16, kI32 = at::kInt, kU8 = at::kByte;

// The arguments' tensors so far: all on one device, the current one.
struct Args {
  int dev = -1;
  bool ok = true;

  const Tensor* any(PyObject* o, int64_t dims) {
    if (!ok || !THPVariable_Check(o)) return fail();
    const Tensor* t = &THPVariable_Unpack(o);
    if (!t->is_cuda() || t->dim() != dims || !t->is_contiguous()) return fail();
    if (dev < 0) {
      dev = t->get_device();
      if (c10::hip::current_device() != dev) return fail();
    } else if (t->get_device() != dev) {
      return fail();
    }
    return t;
  }
  const Tensor* get(PyObject* o, at::ScalarType type, int64_t dims) {
    const Tensor* t = any(o, dims);
    return t && t->scalar_type() == type ? t : fail();
  }
  const Tensor* fail() {
    ok = false;
    return nullptr;
  }
  Tensor make(at::IntArrayRef size, at::ScalarType type) const {
    return at::empty(size, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
  }
  void* stream() const { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }
};

template <typename T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
bool is(const Tensor& t, int64_t a, int64_t b) { return t.size(0) == a && t.size(1) == b; }

// an integer argument; -1 (which no call takes) for one past 64 bits
int64_t integer(PyObject* o) {
  int past;
  return PyLong_AsLongLongAndOverflow(o, &past);
}

PyObject* pack(std::initializer_list<Tensor> ts) {
  if (ts.size() == 1) return THPVariable_Wrap(*ts.begin());
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// A call takes exactly `count` arguments from its Python function.
#define BEGIN(count)                                    \
  HANDLE_TH_ERRORS                                      \
  if (n != (count)) {                                   \
    PyErr_SetString(PyExc_TypeError, "argument count"); \
    return nullptr;                                     \
  }                                                     \
  Args in;
#define PLAIN(condition) \
  if (!(condition)) Py_RETURN_NONE;
#define END END_HANDLE_TH_ERRORS

// (logits, k, renormalize)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(3)
  const Tensor* x = in.any(a[0], 2);
  const int64_t k = integer(a[1]);
  const int renormalize = PyObject_IsTrue(a[2]);
  if (PyErr_Occurred()) return nullptr;
  PLAIN(in.ok && (x->scalar_type() == kF32 || x->scalar_type() == kBf16))
  const int64_t T = x->size(0), E = x->size(1);
  PLAIN(k >= 1 && k <= E && E < (1 << 30))
  const Tensor ids = in.make({T, k}, kI32), w = in.make({T, k}, kF32), sizes = in.make({E}, kI32);
  const Tensor rows = in.make({T, k}, kI32), slots = in.make({T * k}, kI32);
  const size_t need = lib.fp8gmm_workspace_bytes(FP8GMM_OP_ROUTE, T, E, k, 1, 0);
  Tensor ws;
  if (need) ws = in.make({(int64_t)need}, kU8);
  PLAIN(lib.moe_route(x->data_ptr(), x->scalar_type() == kBf16 ? FP8GMM_BF16 : FP8GMM_F32, T, (int32_t)E, (int32_t)k,
                      renormalize, ptr<int32_t>(ids), ptr<float>(w), ptr<int32_t>(sizes),
                      ptr<int32_t>(rows), ptr<int32_t>(slots), need ? ws.data_ptr() : nullptr, need,
                      in.stream()) == FP8GMM_OK)
  return pack({ids, w, sizes, rows, slots});
  END
}

// (dweights, logits, ids, weights, renormalize)
PyObject* route_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(5)
  const Tensor* x = in.any(a[1], 2);
  const Tensor *dw = in.get(a[0], kF32, 2), *ids = in.get(a[2], kI32, 2), *w = in.get(a[3], kF32, 2);
  const int renormalize = PyObject_IsTrue(a[4]);
  if (renormalize < 0) return nullptr;
  PLAIN(in.ok && (x->scalar_type() == kF32 || x->scalar_type() == kBf16))
  const int64_t T = x->size(0), E = x->size(1), k = ids->size(1);
  PLAIN(is(*ids, T, k) && is(*w, T, k) && is(*dw, T, k) && E < (1 << 30) && k < (1 << 30))
  const Tensor out = in.make({T, E}, x->scalar_type());
  PLAIN(lib.moe_route_bwd(ptr<float>(*dw), x->data_ptr(), x->scalar_type() == kBf16 ? FP8GMM_BF16 : FP8GMM_F32,
                          ptr<int32_t>(*ids), ptr<float>(*w), T, (int32_t)E, (int32_t)k, renormalize,
                          out.data_ptr(), in.stream()) == FP8GMM_OK)
  return pack({out});
  END
}

// (x, row_of_slot)
PyObject* permute(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(2)
  const Tensor *x = in.get(a[0], kBf16, 2), *rows = in.get(a[1], kI32, 2);
  PLAIN(in.ok && x->size(0) == rows->size(0))
  const int64_t T = x->size(0), H = x->size(1), k = rows->size(1);
  const Tensor out = in.make({T * k, H}, kBf16);
  PLAIN(k < (1 << 30) && lib.moe_permute(x->data_ptr(), ptr<int32_t>(*rows), T, (int32_t)k, T * k, H, out.data_ptr(),
                                         in.stream()) == FP8GMM_OK)
  return pack({out});
  END
}

// (x, row_of_slot)
PyObject* permute_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(2)
  const Tensor *x = in.get(a[0], kBf16, 2), *rows = in.get(a[1], kI32, 2);
  PLAIN(in.ok && x->size(0) == rows->size(0))
  const int64_t T = x->size(0), H = x->size(1), k = rows->size(1);
  const Tensor codes = in.make({T * k, H}, kU8), scales = in.make({T * k}, kF32);
  PLAIN(k < (1 << 30) && lib.moe_permute_fp8(x->data_ptr(), ptr<int32_t>(*rows), T, (int32_t)k, T * k, H,
                                             ptr<uint8_t>(codes), ptr<float>(scales), in.stream()) == FP8GMM_OK)
  return pack({codes, scales});
  END
}

// (y, row_of_slot, weights or None)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(3)
  const Tensor *y = in.get(a[0], kBf16, 2), *rows = in.get(a[1], kI32, 2);
  const Tensor* w = a[2] == Py_None ? nullptr : in.get(a[2], kF32, 2);
  PLAIN(in.ok)
  const int64_t R = y->size(0), H = y->size(1), T = rows->size(0), k = rows->size(1);
  PLAIN((!w || is(*w, T, k)) && k < (1 << 30))
  const Tensor out = in.make({T, H}, kBf16);
  PLAIN(lib.moe_combine(y->data_ptr(), ptr<int32_t>(*rows), w ? ptr<float>(*w) : nullptr, T, (int32_t)k, R, H,
                        out.data_ptr(), in.stream()) == FP8GMM_OK)
  return pack({out});
  END
}

// (dout, y, row_of_slot, weights)
PyObject* combine_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(4)
  const Tensor *d = in.get(a[0], kBf16, 2), *y = in.get(a[1], kBf16, 2), *rows = in.get(a[2], kI32, 2),
               *w = in.get(a[3], kF32, 2);
  PLAIN(in.ok)
  const int64_t R = y->size(0), H = y->size(1), T = rows->size(0), k = rows->size(1);
  PLAIN(is(*d, T, H) && is(*w, T, k) && k < (1 << 30))
  const Tensor dy = in.make({R, H}, kBf16), dw = in.make({T, k}, kF32);
  PLAIN(lib.moe_combine_bwd(d->data_ptr(), y->data_ptr(), ptr<int32_t>(*rows), ptr<float>(*w), T, (int32_t)k, R, H,
                            dy.data_ptr(), ptr<float>(dw), in.stream()) == FP8GMM_OK)
  return pack({dy, dw});
  END
}

// (w)
PyObject* quantize_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(1)
  const Tensor* w = in.get(a[0], kBf16, 3);
  PLAIN(in.ok)
  const int64_t G = w->size(0), K = w->size(1), N = w->size(2);
  PLAIN(G < (1 << 30))
  const Tensor codes = in.make({G, N, K / 2}, kU8), scales = in.make({G, K / 128, N, 4}, kU8);
  PLAIN(lib.quantize_mxfp4_weights(w->data_ptr(), K, N, (int32_t)G, ptr<uint8_t>(codes), ptr<uint8_t>(scales),
                                   in.stream()) == FP8GMM_OK)
  return pack({codes, scales});
  END
}

// codes [G, N, K/2] with their scales
bool four_bit(const Tensor& codes, const Tensor& scales) {
  return codes.size(0) < (1 << 30) && scales.size(0) == codes.size(0) && scales.size(1) == 2 * codes.size(2) / 128 &&
         scales.size(2) == codes.size(1) && scales.size(3) == 4;
}

// (codes, scales)
PyObject* values(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(2)
  const Tensor *codes = in.get(a[0], kU8, 3), *scales = in.get(a[1], kU8, 4);
  PLAIN(in.ok && four_bit(*codes, *scales))
  const int64_t G = codes->size(0), N = codes->size(1), K = 2 * codes->size(2);
  const Tensor out = in.make({G, N, K}, kBf16);
  PLAIN(lib.dequantize_mxfp4(ptr<uint8_t>(*codes), ptr<uint8_t>(*scales), K, N, (int32_t)G, out.data_ptr(),
                             in.stream()) == FP8GMM_OK)
  return pack({out});
  END
}

// (x, codes, scales, group_sizes, slot_of_row or None, topk, swiglu)
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(7)
  const Tensor *x = in.get(a[0], kBf16, 2), *codes = in.get(a[1], kU8, 3), *scales = in.get(a[2], kU8, 4),
               *sizes = in.get(a[3], kI32, 1);
  const Tensor* slots = a[4] == Py_None ? nullptr : in.get(a[4], kI32, 1);
  const int64_t topk = integer(a[5]);
  if (PyErr_Occurred()) return nullptr;
  PLAIN(in.ok && four_bit(*codes, *scales) && topk > 0 && topk < (1 << 30))
  const int64_t T = x->size(0), G = codes->size(0), N = codes->size(1), K = 2 * codes->size(2);
  const int64_t M = slots ? slots->size(0) : T;
  const bool swiglu = PyObject_IsTrue(a[6]) == 1;
  PLAIN(x->size(1) == K && sizes->size(0) == G)
  const Tensor out = in.make({M, swiglu ? N / 2 : N}, kBf16);
  const size_t need = lib.fp8gmm_workspace_bytes(FP8GMM_OP_MXFP4, T, K, N, (int32_t)G, 0);
  Tensor ws;
  if (need) ws = in.make({(int64_t)need}, kU8);
  PLAIN((swiglu ? lib.gmm_silu_mxfp4 : lib.gmm_mxfp4_fwd)(
            x->data_ptr(), ptr<uint8_t>(*codes), ptr<uint8_t>(*scales), ptr<int32_t>(*sizes),
            slots ? ptr<int32_t>(*slots) : nullptr, (int32_t)topk, T, M, K, N, (int32_t)G, out.data_ptr(),
            need ? ws.data_ptr() : nullptr, need, nullptr, in.stream()) == FP8GMM_OK)
  return pack({out});
  END
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),     {"names", names, METH_NOARGS, nullptr},
                         METHOD(route),    METHOD(route_bwd),
                         METHOD(permute),  METHOD(permute_fp8),
                         METHOD(combine),  METHOD(combine_bwd),
                         METHOD(quantize_weights), METHOD(values),
                         METHOD(product),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
