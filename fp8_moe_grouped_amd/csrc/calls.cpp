// The plain case of the routing, dispatch, combine, 4-bit, balance, AdamW and weight quantizer
// calls without the interpreter: tensors on the current device, contiguous and of the right types and
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

#include <cmath>
#include <vector>

#include "../../include/fp8_moe_grouped.h"

namespace {

using at::Tensor;

#define CALLS(X)                                                                                                 \
  X(moe_route) X(moe_route_bwd) X(moe_permute) X(moe_permute_fp8) X(moe_combine) X(moe_combine_bwd)               \
  X(quantize_mxfp4_weights) X(dequantize_mxfp4) X(gmm_mxfp4_fwd) X(gmm_silu_mxfp4) X(fp8gmm_workspace_bytes)     \
  X(moe_balance_loss) X(moe_balance_loss_bwd) X(quantize_fp8_weights) X(adamw_step) X(adamw_step_8bit)

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

// n numbers of 4 bytes of a storage, from the at-th, as a tensor with a made one's keys
Tensor piece(const Tensor& made, const c10::Storage& of, at::ScalarType type, int64_t at, int64_t n) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(of), made.key_set(), c10::scalarTypeToTypeMeta(type));
  impl->set_storage_offset(at);
  impl->set_sizes_contiguous({n});
  return Tensor(std::move(impl));
}

bool logits_type(const Tensor& t) { return t.scalar_type() == kF32 || t.scalar_type() == kBf16; }
int32_t type_of(const Tensor& t) { return t.scalar_type() == kBf16 ? FP8GMM_BF16 : FP8GMM_F32; }

// (logits, ids or None, counts or None)
PyObject* balance(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(3)
  const Tensor* x = in.any(a[0], 2);
  const Tensor* ids = a[1] == Py_None ? nullptr : in.get(a[1], kI32, 2);
  const Tensor* given = a[2] == Py_None ? nullptr : in.get(a[2], kI32, 1);
  PLAIN(in.ok && logits_type(*x) && !ids != !given)
  const int64_t T = x->size(0), E = x->size(1), k = ids ? ids->size(1) : 1;
  PLAIN(T > 0 && E < (1 << 30) && k < (1 << 30) && (!ids || ids->size(0) == T) && (!given || given->size(0) == E))
  // A storage for the small outputs of each type: a tensor in it costs the host a fifth of one by itself.  Not one for
  // both types: tensors of two types over one storage cannot be saved together.
  const int64_t row = (E + 3) / 4 * 4, numbers = given ? 1 : row + 1;
  const Tensor made = in.make({4 + E}, kF32);
  const c10::Storage& floats = made.storage();
  c10::Allocator* const from = floats.allocator();
  const c10::Storage integers(c10::Storage::use_byte_size_t(), 4 * (size_t)numbers, from->allocate(4 * (size_t)numbers),
                              from, true);
  const Tensor losses = piece(made, floats, kF32, 0, 2), probs = piece(made, floats, kF32, 4, E);
  const Tensor counts = given ? *given : piece(made, integers, kI32, 0, E);
  const Tensor tokens = piece(made, integers, kI32, given ? 0 : row, 1);
  const size_t need = lib.fp8gmm_workspace_bytes(FP8GMM_OP_BALANCE, T, E, k, 1, 0);
  const c10::DataPtr ws = need ? from->allocate(need) : c10::DataPtr();
  PLAIN(lib.moe_balance_loss(x->data_ptr(), type_of(*x), ids ? ptr<int32_t>(*ids) : nullptr, T, (int32_t)E,
                             (int32_t)k, ptr<float>(losses), ptr<int32_t>(counts), ptr<float>(probs),
                             ptr<int32_t>(tokens), ws.get(), need, in.stream()) == FP8GMM_OK)
  return pack({losses, counts, probs, tokens});
  END
}

// (dlosses, logits, counts, tokens, add or None)
PyObject* balance_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(5)
  const Tensor* x = in.any(a[1], 2);
  const Tensor *d = in.get(a[0], kF32, 1), *counts = in.get(a[2], kI32, 1), *tokens = in.get(a[3], kI32, 1);
  PLAIN(in.ok && logits_type(*x))
  const Tensor* add = a[4] == Py_None ? nullptr : in.get(a[4], x->scalar_type(), 2);
  const int64_t T = x->size(0), E = x->size(1);
  PLAIN(in.ok && d->size(0) == 2 && counts->size(0) == E && tokens->size(0) == 1 && (!add || is(*add, T, E)) &&
        E < (1 << 30))
  const Tensor out = in.make({T, E}, x->scalar_type());
  PLAIN(lib.moe_balance_loss_bwd(ptr<float>(*d), x->data_ptr(), type_of(*x), ptr<int32_t>(*counts),
                                 ptr<int32_t>(*tokens), T, (int32_t)E, add ? add->data_ptr() : nullptr,
                                 out.data_ptr(), in.stream()) == FP8GMM_OK)
  return pack({out});
  END
}

// (w)
PyObject* quantize_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN(1)
  const Tensor* w = in.any(a[0], 3);
  PLAIN(in.ok && logits_type(*w))
  const int64_t G = w->size(0), K = w->size(1), N = w->size(2);
  PLAIN(G < (1 << 30))
  const Tensor codes = in.make({G, K, N}, kU8), scales = in.make({G, N}, kF32);
  const size_t need = lib.fp8gmm_workspace_bytes(FP8GMM_OP_QUANT_WEIGHTS, 0, K, N, (int32_t)G, type_of(*w));
  Tensor ws;
  if (need) ws = in.make({(int64_t)need}, kU8);
  PLAIN(lib.quantize_fp8_weights(w->data_ptr(), type_of(*w), K, N, (int32_t)G, ptr<uint8_t>(codes), ptr<float>(scales),
                                 need ? ws.data_ptr() : nullptr, need, in.stream()) == FP8GMM_OK)
  return pack({codes, scales});
  END
}

// A list of tensors with as many members as the call's other lists.
struct List {
  PyObject* fast = nullptr;
  Py_ssize_t n = 0;
  explicit List(PyObject* o) {
    if (!PyList_Check(o) && !PyTuple_Check(o)) return;
    fast = PySequence_Fast(o, "");
    if (fast) n = PySequence_Fast_GET_SIZE(fast);
  }
  ~List() { Py_XDECREF(fast); }
  List(const List&) = delete;
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// A number, or a tensor of one element of this type on the device.
bool number(Args& in, PyObject* o, at::ScalarType type, double* value, const void** device) {
  if (THPVariable_Check(o)) {
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != type || t.numel() != 1 || (in.dev >= 0 && t.get_device() != in.dev))
      return false;
    *device = t.data_ptr();
    return true;
  }
  if (!value || !PyFloat_Check(o)) return false;
  *value = PyFloat_AS_DOUBLE(o);
  return true;
}

// Tensors of any shape, contiguous, on one device, the current one.
const Tensor* member(Args& in, PyObject* o) {
  if (!THPVariable_Check(o)) return in.fail();
  return in.any(o, THPVariable_Unpack(o).dim());
}

// (params, grads, m, second state, lr, step, beta1, beta2, eps, weight_decay, grad_scale or None[, seed]): with a
// seed the states are pairs of codes and scales.  Answers the status.
PyObject* adamw_call(PyObject* const* a, bool held) {
  HANDLE_TH_ERRORS
  Args in;
  const List p(a[0]), g(a[1]), m(a[2]), v(a[3]);
  PLAIN(p.fast && g.fast && m.fast && v.fast && p.n == g.n && p.n == m.n && p.n == v.n && p.n > 0 && p.n < (1 << 24))
  std::vector<int64_t> sizes((size_t)p.n);
  std::vector<void*> at((size_t)p.n * 6);
  void** const cols = at.data();                    // params, grads, then the states' buffers
  at::ScalarType types[2] = {kF32, kF32};
  for (Py_ssize_t i = 0; i < p.n; ++i) {
    const Tensor *pt = member(in, p[i]), *gt = member(in, g[i]);
    PLAIN(in.ok && logits_type(*pt) && logits_type(*gt))
    if (i == 0) {
      types[0] = pt->scalar_type();
      types[1] = gt->scalar_type();
    }
    const int64_t size = pt->numel();
    PLAIN(pt->scalar_type() == types[0] && gt->scalar_type() == types[1] && gt->sizes() == pt->sizes())
    sizes[(size_t)i] = size;
    cols[i] = pt->data_ptr();
    cols[p.n + i] = gt->data_ptr();
    PyObject* const states[2] = {m[i], v[i]};
    for (int s = 0; s < 2; ++s) {
      if (held) {
        PLAIN(PyTuple_Check(states[s]) && PyTuple_GET_SIZE(states[s]) == 2)
        const Tensor* codes = member(in, PyTuple_GET_ITEM(states[s], 0));
        const Tensor* scales = in.get(PyTuple_GET_ITEM(states[s], 1), kF32, 1);
        PLAIN(in.ok && codes->scalar_type() == kU8 && codes->sizes() == pt->sizes() &&
              scales->numel() == (size + 255) / 256)
        cols[(2 + 2 * s) * p.n + i] = codes->data_ptr();
        cols[(3 + 2 * s) * p.n + i] = scales->data_ptr();
      } else {
        const Tensor* t = member(in, states[s]);
        PLAIN(in.ok && t->scalar_type() == kF32 && t->sizes() == pt->sizes())
        cols[(2 + s) * p.n + i] = t->data_ptr();
      }
    }
  }
  fp8gmm_adamw how = {};
  const void *lr = nullptr, *step = nullptr, *scale = nullptr;
  PLAIN(number(in, a[4], kF32, &how.lr, &lr))
  if (PyLong_Check(a[5])) how.step = integer(a[5]);
  else PLAIN(number(in, a[5], at::kLong, nullptr, &step))
  double* const rates[4] = {&how.beta1, &how.beta2, &how.eps, &how.weight_decay};
  for (int i = 0; i < 4; ++i) {
    PLAIN(PyFloat_Check(a[6 + i]))
    *rates[i] = PyFloat_AS_DOUBLE(a[6 + i]);
  }
  PLAIN(a[10] == Py_None || number(in, a[10], kF32, nullptr, &scale))
  how.lr_dev = static_cast<const float*>(lr);
  how.step_dev = static_cast<const int64_t*>(step);
  how.grad_scale = static_cast<const float*>(scale);
  const int32_t n = (int32_t)p.n, pd = types[0] == kBf16, gd = types[1] == kBf16;
  const void* const* const grads = cols + p.n;
  int st;
  if (held) {
    const unsigned long long seed = PyLong_Check(a[11]) ? PyLong_AsUnsignedLongLong(a[11]) : 0;
    if (PyErr_Occurred() || !PyLong_Check(a[11])) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    st = lib.adamw_step_8bit(n, sizes.data(), cols, pd, grads, gd, reinterpret_cast<uint8_t**>(cols + 2 * p.n),
                             reinterpret_cast<float**>(cols + 3 * p.n), reinterpret_cast<uint8_t**>(cols + 4 * p.n),
                             reinterpret_cast<float**>(cols + 5 * p.n), seed, &how, in.stream());
  } else {
    st = lib.adamw_step(n, sizes.data(), cols, pd, grads, gd, reinterpret_cast<float**>(cols + 2 * p.n),
                        reinterpret_cast<float**>(cols + 3 * p.n), &how, in.stream());
  }
  // not left to Python after a launch, which has changed some tensors already
  PLAIN(st == FP8GMM_OK || st == FP8GMM_ERR_HIP)
  for (Py_ssize_t i = 0; i < p.n; ++i) {            // a graph that has saved a parameter notices that it changed
    at::TensorImpl* const impl = THPVariable_Unpack(p[i]).unsafeGetTensorImpl();
    if (!impl->is_inference()) impl->bump_version();
  }
  return PyLong_FromLong(st);
  END
}
PyObject* adamw(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n == 11) return adamw_call(a, false);
  PyErr_SetString(PyExc_TypeError, "argument count");
  return nullptr;
}
PyObject* adamw8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n == 12) return adamw_call(a, true);
  PyErr_SetString(PyExc_TypeError, "argument count");
  return nullptr;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),     {"names", names, METH_NOARGS, nullptr},
                         METHOD(route),    METHOD(route_bwd),
                         METHOD(permute),  METHOD(permute_fp8),
                         METHOD(combine),  METHOD(combine_bwd),
                         METHOD(quantize_weights), METHOD(values),
                         METHOD(product),  METHOD(balance), METHOD(balance_bwd),
                         METHOD(quantize_fp8), METHOD(adamw), METHOD(adamw8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
