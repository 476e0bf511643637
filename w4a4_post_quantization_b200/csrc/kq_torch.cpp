// The part of the Python binding that runs per call of the block operators
// (product with epilogue, K/V cache, attention): checks of the tensors, outputs
// and workspaces that the caller does not bring, the device and the stream, and
// the C ABI's entry points.  Argument marshalling only, as in _lib.py, where the
// calls are documented; in Python the checks of one call took 9 us on the host,
// more than most single-token kernels take on the GPU.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <string>
#include <utility>
#include <vector>

#include "kq.h"

namespace {

// Addresses of the library that _lib.py has loaded, and what raises its errors.
struct Entry {
  decltype(&kq_gemm_mxfp4_epilogue) epilogue = nullptr;
  decltype(&kq_scales_tiled_bytes) scales_tiled_bytes = nullptr;
  decltype(&kq_cache_write) cache_write = nullptr;
  decltype(&kq_cache_read) cache_read = nullptr;
  decltype(&kq_attention_mxfp4) attention = nullptr;
  decltype(&kq_attention_workspace_bytes) attention_workspace_bytes = nullptr;
  PyObject* raise = nullptr;
} g;

// A refusal: ValueError with this text.
struct Refused {
  std::string text;
};
[[noreturn]] void refuse(const std::string& text) { throw Refused{text}; }

const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  return &THPVariable_Unpack(o);
}

// A CUDA tensor of this type on device `dev` (-1: any).
void check(const at::Tensor& t, at::ScalarType type, int64_t dev, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (dev >= 0 && t.get_device() != dev) refuse(std::string(name) + " must be on the operands' device");
}
void check_dense(const at::Tensor& t, at::ScalarType type, int64_t dev, const char* name) {
  check(t, type, dev, name);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  return v;
}

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// Calls `f(stream)` with device `dev` current; raises what it returns.
template <typename F>
bool call(const char* name, int64_t dev, F&& f) {
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
  const int status = f(static_cast<void*>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream()));
  if (status == KQ_OK) return true;
  PyObject* r = PyObject_CallFunction(g.raise, "si", name, status);
  Py_XDECREF(r);
  return false;
}

// [batch, rows, heads, head_dim] rows of unit channel stride that start on
// 16-byte boundaries: their strides (0 for a dimension of size 1, whose stride
// has no meaning).
std::array<int64_t, 3> head_rows(const at::Tensor& x, at::ScalarType type, int64_t dev, const char* name) {
  check(x, type, dev, name);
  if (x.dim() != 4) refuse(std::string(name) + " must be [batch, rows, heads, head_dim]");
  if (x.stride(3) != 1 && x.size(3) > 1) refuse(std::string(name) + " must have unit stride along head_dim");
  const int64_t unit = 16 / static_cast<int64_t>(x.element_size());
  std::array<int64_t, 3> s{};
  bool ok = x.numel() == 0 || reinterpret_cast<uintptr_t>(x.data_ptr()) % 16 == 0;
  for (int i = 0; i < 3; ++i) {
    s[i] = x.size(i) > 1 ? x.stride(i) : 0;
    ok = ok && s[i] % unit == 0;
  }
  if (!ok) refuse("every row of " + std::string(name) + " must start on a 16-byte boundary");
  return s;
}

using Dims = std::vector<std::pair<int64_t, int64_t>>;     // (stride, size), sizes above 1
Dims dims_of(const at::Tensor& x) {
  Dims d;
  for (int64_t i = 0; i < x.dim(); ++i)
    if (x.size(i) > 1) d.emplace_back(x.stride(i), x.size(i));
  std::sort(d.begin(), d.end());
  return d;
}
// The last element's offset, and whether every stride steps over all that the smaller
// ones reach (then no two elements coincide).
int64_t reach_of(const Dims& d, bool* nested) {
  int64_t reach = 0;
  *nested = true;
  for (const auto& [s, n] : d) {
    *nested = *nested && s > reach;
    reach += s * (n - 1);
  }
  return reach;
}

// Whether two elements of tensors with these nested dimensions, their starts `d` apart,
// coincide: d is a sum of steps, fewer than the size along each.  What the smaller
// dimensions can make up for is less than a step, so two counts of steps are possible.
bool meet(const Dims& dims, size_t n, int64_t d) {
  if (n == 0) return d == 0;
  const auto [s, size] = dims[n - 1];
  const int64_t q = d / s - (d % s < 0);
  for (int64_t steps : {q, q + 1})
    if (std::abs(steps) < size && meet(dims, n - 1, d - steps * s)) return true;
  return false;
}

// Whether two tensors share memory.  Exact where they are laid out alike, as slices of
// one buffer are; tensors of different layouts count as sharing where their extents meet.
bool share(const at::Tensor& a, const at::Tensor& b) {
  if (a.numel() == 0 || b.numel() == 0) return false;
  const intptr_t d = static_cast<char*>(b.data_ptr()) - static_cast<char*>(a.data_ptr());
  if (a.is_contiguous() && b.is_contiguous())
    return d < static_cast<intptr_t>(a.nbytes()) && d > -static_cast<intptr_t>(b.nbytes());
  const Dims da = dims_of(a), db = dims_of(b);
  bool nested, other;
  const int64_t ea = static_cast<int64_t>(a.element_size()), eb = static_cast<int64_t>(b.element_size());
  const int64_t ra = (reach_of(da, &nested) + 1) * ea, rb = (reach_of(db, &other) + 1) * eb;
  if (d >= ra || d <= -rb) return false;
  return !nested || da != db || ea != eb || d % ea != 0 || meet(da, da.size(), d / ea);
}

// An output's elements must not overlap one another.
void disjoint(const at::Tensor& x, const char* name) {
  bool nested = true;
  if (!x.is_contiguous()) reach_of(dims_of(x), &nested);
  if (!nested) refuse("the rows of " + std::string(name) + " overlap");
}

struct CacheRef {
  const kq_cache* c;
  int64_t dev;
};
// The cache's description, and its four tensors: what the description points to must
// still be theirs.
CacheRef cache_ref(PyObject* address, PyObject* device, PyObject* tensors) {
  const kq_cache* c = reinterpret_cast<const kq_cache*>(integer(address, "cache"));
  const void* at[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
  const size_t rows = static_cast<size_t>(c->pages * c->heads * c->page_size), nb = (c->head_dim + 31) / 32;
  for (int i = 0; i < 4; ++i) {
    const at::Tensor& t = *tensor(PyTuple_GET_ITEM(tensors, i), "the cache's arrays");
    if (t.data_ptr() != at[i] || t.storage().nbytes() < t.storage_offset() + rows * nb * (i & 1 ? 1 : 16))
      refuse("the cache's tensors have been resized or given other memory: make a new KVCache");
  }
  return {c, integer(device, "device")};
}

const at::Tensor& check_table(PyObject* o, const CacheRef& c, int64_t batch) {
  const at::Tensor& t = *tensor(o, "block_table");
  check_dense(t, at::kInt, c.dev, "block_table");
  if (t.dim() != 2 || (batch >= 0 && t.size(0) != batch) || t.size(1) < 1)
    refuse("block_table must be int32 [batch, pages of a sequence]");
  return t;
}
const at::Tensor* check_per_seq(PyObject* o, const CacheRef& c, int64_t batch, const char* name, bool optional) {
  const at::Tensor* t = tensor(o, name, optional);
  if (!t) return nullptr;
  check_dense(*t, at::kInt, c.dev, name);
  if (t->dim() != 1 || t->size(0) != batch) refuse(std::string(name) + " must be int32 [batch]");
  return t;
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  HANDLE_TH_ERRORS
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (qa, sa_tiled, qb, sb_tiled, bias, act, gate, tokens, residual, out, f32)
PyObject* epilogue(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &qa = *tensor(a[0], "qa"), &sa = *tensor(a[1], "sa_tiled"), &qb = *tensor(a[2], "qb"),
                     &sb = *tensor(a[3], "sb_tiled");
    check_dense(qa, at::kByte, -1, "qa");
    const int64_t dev = qa.get_device();
    check_dense(sa, at::kByte, dev, "sa_tiled");
    check_dense(qb, at::kByte, dev, "qb");
    check_dense(sb, at::kByte, dev, "sb_tiled");
    if (qa.dim() != 2 || qb.dim() != 2 || qa.size(1) == 0 || qa.size(1) % 16 != 0 || qb.size(1) != qa.size(1))
      refuse("qa must be [M, K/2] and qb [N, K/2], K a multiple of 32");
    const int64_t M = qa.size(0), N = qb.size(0), K = 2 * qa.size(1);
    if (sa.numel() < static_cast<int64_t>(g.scales_tiled_bytes(M, K)) ||
        sb.numel() < static_cast<int64_t>(g.scales_tiled_bytes(N, K)))
      refuse("tiled scale arrays are too small");
    const at::ScalarType type = a[10] == Py_True ? at::kFloat : at::kBFloat16;
    const at::Tensor* bias = tensor(a[4], "bias", true);
    if (bias) {
      check_dense(*bias, at::kBFloat16, dev, "bias");
      if (bias->dim() != 1 || bias->size(0) != N) refuse("bias must be bf16 [N]");
    }
    const at::Tensor* gate = tensor(a[6], "gate", true);
    int64_t tokens = 0;
    if (gate) {
      check_dense(*gate, at::kBFloat16, dev, "gate");
      tokens = a[7] == Py_None ? 0 : integer(a[7], "tokens_per_sample");
      if (tokens < 1) refuse("a gate needs tokens_per_sample >= 1");
      if (gate->dim() != 2 || gate->size(1) != N || gate->size(0) < (M == 0 ? 0 : (M - 1) / tokens + 1))
        refuse("gate must be bf16 [B, N] with B >= ceil(M / tokens_per_sample)");
    }
    const at::Tensor* residual = tensor(a[8], "residual", true);
    const at::Tensor* given = tensor(a[9], "out", true);
    for (const auto& [t, name] : {std::make_pair(residual, "residual"), std::make_pair(given, "out")})
      if (t) {
        check_dense(*t, type, dev, name);
        if (t->dim() != 2 || t->size(0) != M || t->size(1) != N) refuse(std::string(name) + " must be [M, N]");
      }
    if (residual && given && residual->data_ptr() != given->data_ptr() && M * N > 0) {
      const intptr_t d = reinterpret_cast<intptr_t>(residual->data_ptr()) - reinterpret_cast<intptr_t>(given->data_ptr());
      if (std::abs(d) < static_cast<intptr_t>(given->nbytes())) refuse("residual must be out itself or not overlap it");
    }
    at::Tensor out = given ? *given : at::empty({M, N}, qa.options().dtype(type));
    if (!call("kq_gemm_mxfp4_epilogue", dev, [&](void* st) {
          return g.epilogue(static_cast<uint8_t*>(qa.data_ptr()), static_cast<uint8_t*>(sa.data_ptr()),
                            static_cast<uint8_t*>(qb.data_ptr()), static_cast<uint8_t*>(sb.data_ptr()), M, N, K,
                            static_cast<uint16_t*>(ptr(bias)), static_cast<int>(integer(a[5], "activation")),
                            static_cast<uint16_t*>(ptr(gate)), tokens, ptr(residual), out.data_ptr(),
                            type == at::kFloat ? KQ_OUT_F32 : KQ_OUT_BF16, st);
        }))
      return nullptr;
    if (given) {
      Py_INCREF(a[9]);
      return a[9];
    }
    return wrap(out);
  });
}

// (cache, device, tensors, block_table, k, v, start, lens)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const CacheRef c = cache_ref(a[0], a[1], a[2]);
    const at::Tensor &k = *tensor(a[4], "k"), &v = *tensor(a[5], "v");
    const auto ks = head_rows(k, at::kBFloat16, c.dev, "k"), vs = head_rows(v, at::kBFloat16, c.dev, "v");
    if (v.sizes() != k.sizes()) refuse("k and v must have the same shape");
    const int64_t B = k.size(0);
    if (k.size(2) != c.c->heads || k.size(3) != c.c->head_dim) refuse("k and v must have the cache's heads and head_dim");
    const at::Tensor& table = check_table(a[3], c, B);
    const at::Tensor* start = check_per_seq(a[6], c, B, "start", true);
    const at::Tensor* lens = check_per_seq(a[7], c, B, "lens", true);
    if (!call("kq_cache_write", c.dev, [&](void* st) {
          return g.cache_write(c.c, static_cast<int32_t*>(table.data_ptr()), B, table.size(1),
                               static_cast<uint16_t*>(k.data_ptr()), ks[0], ks[1], ks[2],
                               static_cast<uint16_t*>(v.data_ptr()), vs[0], vs[1], vs[2], k.size(1),
                               static_cast<int32_t*>(ptr(start)), static_cast<int32_t*>(ptr(lens)), st);
        }))
      return nullptr;
    Py_RETURN_NONE;
  });
}

// (cache, device, tensors, block_table, lens, tokens, start, f32, k, v)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const CacheRef c = cache_ref(a[0], a[1], a[2]);
    const at::Tensor& table = check_table(a[3], c, -1);
    const int64_t B = table.size(0), T = integer(a[5], "tokens");
    if (T < 0) refuse("tokens must not be negative");
    const at::Tensor* lens = check_per_seq(a[4], c, B, "lens", true);
    const at::Tensor* start = check_per_seq(a[6], c, B, "start", true);
    const at::ScalarType type = a[7] == Py_True ? at::kFloat : at::kBFloat16;
    const std::array<int64_t, 4> shape{B, T, c.c->heads, c.c->head_dim};
    at::Tensor x[2];
    std::array<int64_t, 3> s[2];
    for (int i = 0; i < 2; ++i) {
      const char* name = i ? "v" : "k";
      const at::Tensor* given = tensor(a[8 + i], name, true);
      x[i] = given ? *given : at::empty(shape, table.options().dtype(type));
      s[i] = head_rows(x[i], type, c.dev, name);
      if (x[i].sizes() != at::IntArrayRef(shape)) refuse(std::string(name) + " must be [batch, tokens, heads, head_dim]");
      disjoint(x[i], name);
    }
    if (a[8] != Py_None && a[9] != Py_None && share(x[0], x[1])) refuse("k and v must not share memory");
    if (!call("kq_cache_read", c.dev, [&](void* st) {
          return g.cache_read(c.c, static_cast<int32_t*>(table.data_ptr()), B, table.size(1), T,
                              static_cast<int32_t*>(ptr(start)), static_cast<int32_t*>(ptr(lens)), x[0].data_ptr(),
                              s[0][0], s[0][1], s[0][2], x[1].data_ptr(), s[1][0], s[1][1], s[1][2],
                              type == at::kFloat ? KQ_OUT_F32 : KQ_OUT_BF16, st);
        }))
      return nullptr;
    return Py_BuildValue("(NN)", wrap(x[0]), wrap(x[1]));
  });
}

// (q, cache, device, tensors, block_table, lens, causal, scale, max_len, out, lse, workspace)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const CacheRef c = cache_ref(a[1], a[2], a[3]);
    const at::Tensor& q = *tensor(a[0], "q");
    const auto qs = head_rows(q, at::kBFloat16, c.dev, "q");
    const int64_t B = q.size(0), M = q.size(1), H = q.size(2), D = q.size(3);
    if (D != c.c->head_dim || H == 0 || H % c.c->heads != 0)
      refuse("q must have the cache's head_dim and a multiple of its heads");
    const at::Tensor& table = check_table(a[4], c, B);
    const at::Tensor* lens = check_per_seq(a[5], c, B, "lens", false);
    const int64_t room = table.size(1) * c.c->page_size;
    const int64_t max_len = a[8] == Py_None ? room : integer(a[8], "max_len");
    if (max_len < 1 || max_len > room) refuse("max_len must be from 1 to what the block table holds");
    const int causal = PyObject_IsTrue(a[6]);
    if (causal < 0) return nullptr;
    double scale = 1.0 / std::sqrt(static_cast<double>(D));
    if (a[7] != Py_None) {
      scale = PyFloat_AsDouble(a[7]);
      if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    }
    const at::Tensor* given = tensor(a[9], "out", true);
    at::Tensor out = given ? *given : at::empty(q.sizes(), q.options().memory_format(at::MemoryFormat::Contiguous));
    const auto os = head_rows(out, at::kBFloat16, c.dev, "out");
    if (out.sizes() != q.sizes()) refuse("out must have the shape of q");
    disjoint(out, "out");
    if (given && share(q, *given)) refuse("out and q must not share memory");
    const at::Tensor* lse = tensor(a[10], "lse", true);
    if (lse) {
      check_dense(*lse, at::kFloat, c.dev, "lse");
      if (lse->dim() != 3 || lse->size(0) != B || lse->size(1) != H || lse->size(2) != M)
        refuse("lse must be float32 [batch, heads, M]");
      if (share(*lse, q) || share(*lse, out)) refuse("lse must not share memory with q or out");
    }
    if (B > 0 && M > 0) {
      const size_t need = g.attention_workspace_bytes(B, M, H, c.c->heads, D, max_len);
      const at::Tensor* ws = tensor(a[11], "workspace", true);
      at::Tensor own;
      if (ws) {
        check_dense(*ws, at::kByte, c.dev, "workspace");
        if (share(*ws, q) || share(*ws, out) || (lse && share(*ws, *lse)))
          refuse("the workspace must not share memory with q, out or lse");
      } else if (need > 0) {
        own = at::empty({static_cast<int64_t>(need)}, q.options().dtype(at::kByte));
        ws = &own;
      }
      if (!call("kq_attention_mxfp4", c.dev, [&](void* st) {
            return g.attention(static_cast<uint16_t*>(q.data_ptr()), qs[0], qs[1], qs[2], B, M, H, c.c,
                               static_cast<int32_t*>(table.data_ptr()), table.size(1),
                               static_cast<int32_t*>(lens->data_ptr()), max_len, static_cast<float>(scale), causal,
                               static_cast<uint16_t*>(out.data_ptr()), os[0], os[1], os[2],
                               static_cast<float*>(ptr(lse)), ptr(ws), ws ? ws->nbytes() : 0, st);
          }))
        return nullptr;
    }
    if (given) {
      Py_INCREF(a[9]);
      return a[9];
    }
    return wrap(out);
  });
}

// (raise, addresses of the six entry points in Entry's order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    auto set = [&](auto& f, int i) {
      f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(static_cast<intptr_t>(integer(a[i], "address")));
    };
    set(g.epilogue, 1);
    set(g.scales_tiled_bytes, 2);
    set(g.cache_write, 3);
    set(g.cache_read, 4);
    set(g.attention, 5);
    set(g.attention_workspace_bytes, 6);
    Py_INCREF(a[0]);
    Py_XDECREF(g.raise);
    g.raise = a[0];
    Py_RETURN_NONE;
  });
}

#define KQ_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KQ_METHOD(bind),       KQ_METHOD(epilogue),  KQ_METHOD(cache_write),
                         KQ_METHOD(cache_read), KQ_METHOD(attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kq_torch() { return PyModule_Create(&module); }
