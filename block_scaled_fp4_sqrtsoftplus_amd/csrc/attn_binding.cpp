// Native half of the Python binding of include/moe_attn.h and include/moe_serving.h: takes torch tensors
// apart, checks them, makes the outputs and calls the C ABI.  A decode step's
// calls are short (the launch itself takes the host about 4 us), and the same
// checks in Python and ctypes took 6 to 9 us more.  Keyword handling and the
// handles stay in attention.py and serving.py.
//
// Host code only, built by the C++ compiler against torch's headers; the
// kernels are in libmoe_fp4.so.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "moe_serving.h"

namespace {

PyObject* g_error = nullptr;   // MoeError, called with the status

// Thrown for an argument that the binding refuses.
struct Refused {
  std::string why;
};

[[noreturn]] void refuse(const char* name, const std::string& why) {
  throw Refused{std::string(name) + " " + why};
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, "must be a tensor");
  return THPVariable_Unpack(o);
}

void same_device(const at::Tensor& t, int index, const char* name) {
  if (!t.is_cuda()) throw Refused{"tensors passed to the HIP library must be on the GPU"};
  if (t.get_device() != index)
    refuse(name, "is on " + t.device().str() + ", the call's other tensors are on cuda:" +
                     std::to_string(index));
}

// A [tokens, heads, dim] bf16 tensor; tokens or heads -1: whatever it has.
moe_rows rows(const at::Tensor& t, int64_t tokens, int64_t heads, int64_t dim, int index,
              const char* name) {
  if (t.scalar_type() != at::kBFloat16) refuse(name, "must be torch.bfloat16");
  const auto s = t.sizes();
  if (s.size() != 3) refuse(name, "must be [tokens, heads, head_dim]");
  if ((tokens >= 0 && s[0] != tokens) || (heads >= 0 && s[1] != heads) || s[2] != dim)
    refuse(name, "has shape " + shape_text(s) + ", expected " +
                     shape_text({tokens >= 0 ? tokens : s[0], heads >= 0 ? heads : s[1], dim}));
  same_device(t, index, name);
  if (s[2] > 1 && t.stride(2) != 1) refuse(name, "must be contiguous in its last index");
  if (t.requires_grad() && c10::GradMode::is_enabled())
    refuse(name, "requires a gradient, which these operators do not pass on: detach it or call "
                 "under torch.no_grad()");
  // strides over indices of one value are free
  return moe_rows{static_cast<uint16_t*>(t.data_ptr()), s[0] > 1 ? t.stride(0) : 0,
                  s[1] > 1 ? t.stride(1) : 0};
}

// A contiguous tensor of integers.
void* ints(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, int index,
           const char* name) {
  if (t.scalar_type() != type)
    refuse(name, type == at::kLong ? "must be torch.int64" : "must be torch.int32");
  if (t.sizes() != shape)
    refuse(name, "has shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
  same_device(t, index, name);
  if (!t.is_contiguous()) refuse(name, "must be contiguous");
  if (t.numel()) return t.data_ptr();
  // an empty view still points into its storage (NULL only if that is empty too)
  char* base = static_cast<char*>(const_cast<void*>(t.storage().data()));
  return base ? base + t.storage_offset() * t.element_size() : nullptr;
}

// The tensors' GPU is the current one for a call.
struct OnDevice {
  c10::DeviceGuard guard;
  explicit OnDevice(int index) : guard(at::Device(at::kCUDA, (c10::DeviceIndex)index)) {}
};

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int index) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, index)));
}

int64_t number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r != 0;
}
template <class T>
T* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return static_cast<T*>(p);
}

PyObject* failed(moe_status s) {
  PyObject* v = PyLong_FromLong(s);
  if (v) PyErr_SetObject(g_error, v);
  Py_XDECREF(v);
  return nullptr;
}

// out, or (out, lse)
PyObject* results(const at::Tensor& out, const at::Tensor& lse) {
  PyObject* a = THPVariable_Wrap(out);
  if (!a || !lse.defined()) return a;
  PyObject* b = THPVariable_Wrap(lse);
  PyObject* t = b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_DECREF(a);
  Py_XDECREF(b);
  return t;
}

#define BINDING_TRY HANDLE_TH_ERRORS try {
#define BINDING_END                                   \
  }                                                   \
  catch (const Refused& r) {                          \
    PyErr_SetString(PyExc_ValueError, r.why.c_str()); \
    return nullptr;                                   \
  }                                                   \
  END_HANDLE_TH_ERRORS

bool expects(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// kv_append(cache, rope or 0, device, stream, k, v, slots, positions, q, q_out, k_out)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BINDING_TRY
  if (!expects(n, 11)) return nullptr;
  const auto* cache = address<const moe_kv_cache>(a[0]);
  const auto* rope = address<const moe_rope>(a[1]);
  const int index = (int)number(a[2]);
  void* stream = address<void>(a[3]);
  const OnDevice on(index);
  const int64_t heads = cache->heads, dim = cache->head_dim;
  const at::Tensor& kt = tensor(a[4], "k");
  const moe_rows k = rows(kt, -1, heads, dim, index, "k");
  const int64_t tokens = kt.size(0);
  const bool has_v = a[5] != Py_None, has_pos = a[7] != Py_None, has_q = a[8] != Py_None,
             has_ko = a[10] != Py_None;
  moe_rows v{}, q{}, qo{}, ko{};
  if (has_v) v = rows(tensor(a[5], "v"), tokens, heads, dim, index, "v");
  const auto* slots = static_cast<const int64_t*>(
      ints(tensor(a[6], "slots"), at::kLong, {tokens}, index, "slots"));
  const int32_t* positions = nullptr;
  if (has_pos)
    positions = static_cast<const int32_t*>(
        ints(tensor(a[7], "positions"), at::kInt, {tokens}, index, "positions"));
  int64_t hq = 0;
  at::Tensor out;
  if (has_q) {
    const at::Tensor& qt = tensor(a[8], "q");
    q = rows(qt, tokens, -1, dim, index, "q");
    hq = qt.size(1);
    if (hq > INT32_MAX) return failed(MOE_ERR_BAD_SHAPE);
    out = a[9] == Py_None ? fresh({tokens, hq, dim}, at::kBFloat16, index) : tensor(a[9], "q_out");
    qo = rows(out, tokens, hq, dim, index, "q_out");
  } else if (a[9] != Py_None) {
    throw Refused{"q_out without q"};
  }
  if (has_ko) ko = rows(tensor(a[10], "k_out"), tokens, heads, dim, index, "k_out");
  const moe_status s =
      moe_kv_append(cache, rope, tokens, slots, positions, &k, has_v ? &v : nullptr,
                    (int32_t)hq, has_q ? &q : nullptr, has_q ? &qo : nullptr,
                    has_ko ? &ko : nullptr, stream);
  if (s != MOE_OK) return failed(s);
  if (!has_q) Py_RETURN_NONE;
  if (a[9] != Py_None) {
    Py_INCREF(a[9]);
    return a[9];
  }
  return THPVariable_Wrap(out);
  BINDING_END
}

// attn_decode(config, cache, device, stream, ws, ws_bytes, q, block_table, seq_lens, out, want_lse, sinks)
// and with masks behind them attn_tree
PyObject* decode(PyObject* const* a, bool tree) {
  BINDING_TRY
  const auto* cfg = address<const moe_attn_config>(a[0]);
  const auto* cache = address<const moe_kv_cache>(a[1]);
  const int index = (int)number(a[2]);
  void* stream = address<void>(a[3]);
  const OnDevice on(index);
  const int64_t tokens = cfg->tokens, hq = cfg->heads_q, dim = cfg->head_dim, batch = cfg->batch;
  const moe_rows q = rows(tensor(a[6], "q"), tokens, hq, dim, index, "q");
  const at::Tensor& tt = tensor(a[7], "block_table");
  if (tt.dim() != 2) throw Refused{"block_table must be [batch, width]"};
  const int64_t width = tt.size(1);
  const auto* table = static_cast<const int32_t*>(
      ints(tt, at::kInt, {batch, width}, index, "block_table"));
  const auto* lens = static_cast<const int32_t*>(
      ints(tensor(a[8], "seq_lens"), at::kInt, {batch}, index, "seq_lens"));
  const at::Tensor out =
      a[9] == Py_None ? fresh({tokens, hq, dim}, at::kBFloat16, index) : tensor(a[9], "out");
  const moe_rows o = rows(out, tokens, hq, dim, index, "out");
  at::Tensor lse;
  if (truth(a[10])) lse = fresh({tokens, hq}, at::kFloat, index);
  if (width > INT32_MAX) return failed(MOE_ERR_BAD_SHAPE);
  const int32_t sinks = (int32_t)number(a[11]);   // the handle has checked that it fits
  float* l = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
  moe_status s;
  if (tree) {
    const auto* masks = static_cast<const uint64_t*>(
        ints(tensor(a[12], "masks"), at::kLong, {batch, cfg->q_len}, index, "masks"));
    s = moe_attn_tree(cfg, sinks, &q, cache, table, (int32_t)width, lens, masks, &o, l,
                      address<void>(a[4]), (size_t)number(a[5]), stream);
  } else {
    s = moe_attn_decode_sinks(cfg, sinks, &q, cache, table, (int32_t)width, lens, &o, l,
                              address<void>(a[4]), (size_t)number(a[5]), stream);
  }
  return s == MOE_OK ? results(out, lse) : failed(s);
  BINDING_END
}
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return expects(n, 12) ? decode(a, false) : nullptr;
}
PyObject* attn_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return expects(n, 13) ? decode(a, true) : nullptr;
}

// tree_masks(device, stream, parents) -> masks, depths
PyObject* tree_masks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BINDING_TRY
  if (!expects(n, 3)) return nullptr;
  const int index = (int)number(a[0]);
  const OnDevice on(index);
  const at::Tensor& pt = tensor(a[2], "parents");
  if (pt.dim() != 2) throw Refused{"parents must be [batch, nodes]"};
  const int64_t batch = pt.size(0), nodes = pt.size(1);
  const auto* parents = static_cast<const int32_t*>(
      ints(pt, at::kInt, {batch, nodes}, index, "parents"));
  if (batch > INT32_MAX || nodes > INT32_MAX) return failed(MOE_ERR_BAD_SHAPE);
  const at::Tensor masks = fresh({batch, nodes}, at::kLong, index);
  const at::Tensor depths = fresh({batch, nodes}, at::kInt, index);
  const moe_status s = moe_tree_masks((int32_t)batch, (int32_t)nodes, parents,
                                      static_cast<uint64_t*>(masks.data_ptr()),
                                      static_cast<int32_t*>(depths.data_ptr()),
                                      address<void>(a[1]));
  return s == MOE_OK ? results(masks, depths) : failed(s);
  BINDING_END
}

// kv_compact(cache, device, stream, block_table, context_lens, path, counts)
PyObject* kv_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BINDING_TRY
  if (!expects(n, 7)) return nullptr;
  const auto* cache = address<const moe_kv_cache>(a[0]);
  const int index = (int)number(a[1]);
  const OnDevice on(index);
  const at::Tensor &tt = tensor(a[3], "block_table"), &pt = tensor(a[5], "path");
  if (tt.dim() != 2) throw Refused{"block_table must be [batch, width]"};
  const int64_t batch = tt.size(0), width = tt.size(1);
  if (pt.dim() != 2) throw Refused{"path must be [batch, nodes]"};
  const int64_t nodes = pt.size(1);
  const auto* table =
      static_cast<const int32_t*>(ints(tt, at::kInt, {batch, width}, index, "block_table"));
  const auto* lens = static_cast<const int32_t*>(
      ints(tensor(a[4], "context_lens"), at::kInt, {batch}, index, "context_lens"));
  const auto* path =
      static_cast<const int32_t*>(ints(pt, at::kInt, {batch, nodes}, index, "path"));
  const auto* counts = static_cast<const int32_t*>(
      ints(tensor(a[6], "counts"), at::kInt, {batch}, index, "counts"));
  if (batch > INT32_MAX || width > INT32_MAX || nodes > INT32_MAX) return failed(MOE_ERR_BAD_SHAPE);
  const moe_status s = moe_kv_compact(cache, (int32_t)batch, (int32_t)nodes, table, (int32_t)width,
                                      lens, path, counts, address<void>(a[2]));
  if (s != MOE_OK) return failed(s);
  Py_RETURN_NONE;
  BINDING_END
}

// kv_copy_pages(cache, device, stream, src, dst)
PyObject* kv_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BINDING_TRY
  if (!expects(n, 5)) return nullptr;
  const auto* cache = address<const moe_kv_cache>(a[0]);
  const int index = (int)number(a[1]);
  const OnDevice on(index);
  const at::Tensor& st = tensor(a[3], "src");
  if (st.dim() != 1) throw Refused{"src must be [pairs]"};
  const int64_t pairs = st.size(0);
  const auto* src = static_cast<const int32_t*>(ints(st, at::kInt, {pairs}, index, "src"));
  const auto* dst =
      static_cast<const int32_t*>(ints(tensor(a[4], "dst"), at::kInt, {pairs}, index, "dst"));
  const moe_status s = moe_kv_copy_pages(cache, pairs, src, dst, address<void>(a[2]));
  if (s != MOE_OK) return failed(s);
  Py_RETURN_NONE;
  BINDING_END
}

// pool_grow(pool, device, stream, ws, ws_bytes, cu, tokens, missing) -> slots, positions, src, dst
PyObject* pool_grow(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BINDING_TRY
  if (!expects(n, 8)) return nullptr;
  const auto* pool = address<const moe_page_pool>(a[0]);
  const int index = (int)number(a[1]);
  const OnDevice on(index);
  const int64_t batch = pool->batch, tokens = number(a[6]);
  if (tokens < 0 || tokens > INT32_MAX) return failed(MOE_ERR_BAD_SHAPE);
  const auto* cu = static_cast<const int32_t*>(
      ints(tensor(a[5], "cu"), at::kInt, {batch + 1}, index, "cu"));
  const at::Tensor slots = fresh({tokens}, at::kLong, index);
  const at::Tensor positions = fresh({tokens}, at::kInt, index);
  const at::Tensor src = fresh({batch}, at::kInt, index), dst = fresh({batch}, at::kInt, index);
  const moe_status s =
      moe_pool_grow(pool, tokens, cu, static_cast<int64_t*>(slots.data_ptr()),
                    static_cast<int32_t*>(positions.data_ptr()),
                    static_cast<int32_t*>(src.data_ptr()), static_cast<int32_t*>(dst.data_ptr()),
                    address<int32_t>(a[7]), address<void>(a[3]), (size_t)number(a[4]),
                    address<void>(a[2]));
  if (s != MOE_OK) return failed(s);
  PyObject* t = PyTuple_New(4);
  if (!t) return nullptr;
  const at::Tensor* all[] = {&slots, &positions, &src, &dst};
  for (int i = 0; i < 4; ++i) {
    PyObject* x = THPVariable_Wrap(*all[i]);
    if (!x) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i, x);
  }
  return t;
  BINDING_END
}

// pool_fork(pool, device, stream, parents)
PyObject* pool_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BINDING_TRY
  if (!expects(n, 4)) return nullptr;
  const auto* pool = address<const moe_page_pool>(a[0]);
  const int index = (int)number(a[1]);
  const OnDevice on(index);
  const auto* parents = static_cast<const int32_t*>(
      ints(tensor(a[3], "parents"), at::kInt, {pool->batch}, index, "parents"));
  const moe_status s = moe_pool_fork(pool, parents, address<void>(a[2]));
  if (s != MOE_OK) return failed(s);
  Py_RETURN_NONE;
  BINDING_END
}

// pool_trim(pool, device, stream, lens or None, window, sinks)
PyObject* pool_trim(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BINDING_TRY
  if (!expects(n, 6)) return nullptr;
  const auto* pool = address<const moe_page_pool>(a[0]);
  const int index = (int)number(a[1]);
  const OnDevice on(index);
  const int32_t* lens = nullptr;
  if (a[3] != Py_None)
    lens = static_cast<const int32_t*>(
        ints(tensor(a[3], "lens"), at::kInt, {pool->batch}, index, "lens"));
  const int64_t window = number(a[4]), sinks = number(a[5]);
  if (window < INT32_MIN || window > INT32_MAX || sinks < INT32_MIN || sinks > INT32_MAX)
    return failed(MOE_ERR_BAD_SHAPE);
  const moe_status s =
      moe_pool_trim(pool, lens, (int32_t)window, (int32_t)sinks, address<void>(a[2]));
  if (s != MOE_OK) return failed(s);
  Py_RETURN_NONE;
  BINDING_END
}

// attn_prefill(device, stream, q, k, v, cu_q, cu_k, causal, window, scale or None, out, want_lse, sinks)
PyObject* attn_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BINDING_TRY
  if (!expects(n, 13)) return nullptr;
  const int index = (int)number(a[0]);
  void* stream = address<void>(a[1]);
  const OnDevice on(index);
  const at::Tensor &qt = tensor(a[2], "q"), &kt = tensor(a[3], "k"), &vt = tensor(a[4], "v");
  const at::Tensor& cu = tensor(a[5], "cu_q");
  if (qt.dim() != 3 || kt.dim() != 3 || cu.dim() != 1)
    throw Refused{"q, k and v must be [tokens, heads, head_dim], cu_q [sequences + 1]"};
  if (cu.size(0) < 1) throw Refused{"cu_q has sequences + 1 entries"};
  const int64_t tokens = qt.size(0), hq = qt.size(1), dim = qt.size(2);
  const int64_t keys = kt.size(0), hkv = kt.size(1), batch = cu.size(0) - 1;
  const bool has_cu_k = a[6] != Py_None;
  if (!has_cu_k && keys != tokens) throw Refused{"without cu_k, k has as many rows as q"};
  const moe_rows q = rows(qt, tokens, hq, dim, index, "q");
  const moe_rows k = rows(kt, keys, hkv, dim, index, "k");
  const moe_rows v = a[4] == a[3] ? k : rows(vt, keys, hkv, dim, index, "v");
  const auto* cu_q =
      static_cast<const int32_t*>(ints(cu, at::kInt, {batch + 1}, index, "cu_q"));
  const int32_t* cu_k = nullptr;
  if (has_cu_k)
    cu_k = static_cast<const int32_t*>(
        ints(tensor(a[6], "cu_k"), at::kInt, {batch + 1}, index, "cu_k"));
  const int64_t window = number(a[8]), sinks = number(a[12]);
  double scale = 0.0;
  if (a[9] == Py_None) {
    scale = 1.0 / std::sqrt((double)dim);
  } else {
    scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  if (batch > INT32_MAX || hq > INT32_MAX || hkv > INT32_MAX || dim > INT32_MAX ||
      window < INT32_MIN || window > INT32_MAX || sinks < INT32_MIN || sinks > INT32_MAX)
    return failed(MOE_ERR_BAD_SHAPE);
  const at::Tensor out =
      a[10] == Py_None ? fresh({tokens, hq, dim}, at::kBFloat16, index) : tensor(a[10], "out");
  const moe_rows o = rows(out, tokens, hq, dim, index, "out");
  at::Tensor lse;
  if (truth(a[11])) lse = fresh({tokens, hq}, at::kFloat, index);
  const moe_attn_config cfg{tokens,       keys,         (int32_t)batch, 1,
                            (int32_t)hq,  (int32_t)hkv, (int32_t)dim,   truth(a[7]),
                            (int32_t)window, (float)scale};
  const moe_status s =
      moe_attn_prefill_sinks(&cfg, (int32_t)sinks, &q, &k, &v, cu_q, cu_k, &o,
                             lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, stream);
  return s == MOE_OK ? results(out, lse) : failed(s);
  BINDING_END
}

PyObject* set_error(PyObject*, PyObject* o) {
  Py_INCREF(o);
  Py_XDECREF(g_error);
  g_error = o;
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"kv_append", fast(kv_append), METH_FASTCALL, nullptr},
    {"attn_decode", fast(attn_decode), METH_FASTCALL, nullptr},
    {"attn_prefill", fast(attn_prefill), METH_FASTCALL, nullptr},
    {"attn_tree", fast(attn_tree), METH_FASTCALL, nullptr},
    {"tree_masks", fast(tree_masks), METH_FASTCALL, nullptr},
    {"kv_compact", fast(kv_compact), METH_FASTCALL, nullptr},
    {"kv_copy_pages", fast(kv_copy_pages), METH_FASTCALL, nullptr},
    {"pool_grow", fast(pool_grow), METH_FASTCALL, nullptr},
    {"pool_fork", fast(pool_fork), METH_FASTCALL, nullptr},
    {"pool_trim", fast(pool_trim), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn_binding", nullptr, -1, g_methods,
                        nullptr,               nullptr,         nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding() { return PyModule_Create(&g_module); }
