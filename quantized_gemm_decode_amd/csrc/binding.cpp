// The serving operators' Python entry points: argument checks on torch
// tensors, then the C ABI.
//
// A decode step makes these calls once a layer, each a few microseconds of GPU
// time, so what the host spends on a call counts.  Checked through ctypes a
// call takes 9.9 us of host time, 5.4 us of it the checks; here the checks take
// a fraction of a microsecond beside the launch itself.  Functions take their
// arguments by position (serving.py gives them names and defaults), raise
// ValueError for tensors that do not fit and return the library's status.
#include <torch/csrc/autograd/python_variable.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>

#include "../../include/qlinear.h"

namespace {

// Thrown once a Python error is set.
struct Refused {};

[[noreturn]] void refuse(const char* name, const char* what) {
  PyErr_Format(PyExc_ValueError, "%s %s", name, what);
  throw Refused();
}

int64_t number(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

// One call's tensors: all on the GPU that the first one names.
struct Call {
  int device = -1;

  const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type, const char* type_name) {
    if (!THPVariable_Check(o)) refuse(name, "must be a CUDA (HIP) tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda()) refuse(name, "must be a CUDA (HIP) tensor");
    if (t.layout() != at::kStrided) refuse(name, "must be a dense tensor");
    if (t.scalar_type() != type) {
      PyErr_Format(PyExc_ValueError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()), type_name);
      throw Refused();
    }
    if (device < 0)
      device = t.get_device();
    else if (t.get_device() != device)
      refuse(name, "is on another device than the call's first tensor");
    return t;
  }

  // Address of a contiguous tensor of at least `numel` elements.
  template <class T>
  T* flat(PyObject* o, const char* name, at::ScalarType type, const char* type_name, int64_t numel) {
    const at::Tensor& t = tensor(o, name, type, type_name);
    if (!t.is_contiguous()) refuse(name, "must be contiguous");
    if (t.numel() < numel) {
      PyErr_Format(PyExc_ValueError, "%s holds %lld elements; this call needs at least %lld", name,
                   (long long)t.numel(), (long long)numel);
      throw Refused();
    }
    return static_cast<T*>(t.data_ptr());
  }
  // The same for rows of `width` elements each (or the elements in one row).
  float* f32_rows(PyObject* o, const char* name, int64_t n, int64_t width) {
    float* p = f32(o, name, n * width);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.dim() > 1 && t.size(-1) != width) {
      PyErr_Format(PyExc_ValueError, "%s has rows of %lld elements, expected %lld", name, (long long)t.size(-1),
                   (long long)width);
      throw Refused();
    }
    return p;
  }
  int32_t* i32(PyObject* o, const char* name, int64_t n) { return flat<int32_t>(o, name, at::kInt, "torch.int32", n); }
  int64_t* i64(PyObject* o, const char* name, int64_t n) { return flat<int64_t>(o, name, at::kLong, "torch.int64", n); }
  float* f32(PyObject* o, const char* name, int64_t n) { return flat<float>(o, name, at::kFloat, "torch.float32", n); }
  void* bytes(PyObject* o, const char* name, int64_t n) { return flat<void>(o, name, at::kByte, "torch.uint8", n); }
  void* bf16(PyObject* o, const char* name, int64_t n) {
    return flat<void>(o, name, at::kBFloat16, "torch.bfloat16", n);
  }

  // bf16 [tokens, heads, head_dim] with contiguous heads; sizes below 0 are
  // taken from the tensor.
  ql_rows rows(PyObject* o, const char* name, int64_t& tokens, int64_t& heads, int64_t& dim) {
    const at::Tensor& t = tensor(o, name, at::kBFloat16, "torch.bfloat16");
    if (t.dim() != 3) refuse(name, "must be a [tokens, heads, head_dim] tensor");
    if (tokens < 0) tokens = t.size(0);
    if (heads < 0) heads = t.size(1);
    if (dim < 0) dim = t.size(2);
    if (t.size(0) != tokens || t.size(1) != heads || t.size(2) != dim) {
      PyErr_Format(PyExc_ValueError, "%s has shape (%lld, %lld, %lld), expected (%lld, %lld, %lld)", name,
                   (long long)t.size(0), (long long)t.size(1), (long long)t.size(2), (long long)tokens,
                   (long long)heads, (long long)dim);
      throw Refused();
    }
    if (t.stride(2) != 1 && dim > 1) refuse(name, "must have contiguous heads");
    return ql_rows{t.data_ptr(), t.stride(0), t.stride(1)};
  }

  // A cache's descriptor; `index` is the device of its tensors.
  const ql_kv_cache* cache(PyObject* address, PyObject* index) {
    if (number(index) != device) refuse("cache", "is on another device than the call's first tensor");
    return static_cast<const ql_kv_cache*>(number_ptr(address));
  }

  void* stream(PyObject* o) {
    if (o == Py_None) return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(device)).stream();
    return number_ptr(o);
  }

  static void* number_ptr(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused();
    return p;
  }
};

// Launches go to the process's current device: makes that the call's for a
// scope.  As a rule it is already, and then only asking costs anything (0.1 us
// of host time, a guard that sets it and sets it back 0.3).
struct OnDevice {
  c10::hip::OptionalHIPGuard guard;
  explicit OnDevice(const Call& c) {
    if (c10::hip::current_device() != c.device) guard.set_index(static_cast<c10::DeviceIndex>(c.device));
  }
};

ql_norm_rope rule_of(Call& c, PyObject* table, PyObject* q_weight, PyObject* k_weight, int64_t dim, PyObject* eps,
                     PyObject* interleaved) {
  ql_norm_rope r{};
  if (table != Py_None) {
    const at::Tensor& t = c.tensor(table, "cos_sin", at::kFloat, "torch.float32");
    if (t.dim() != 2) refuse("cos_sin", "must be a [max_pos, rot_dim] tensor");
    if (t.size(1) > dim) refuse("cos_sin", "rotates more values than a head has");
    r.cos_sin = c.f32(table, "cos_sin", 0);
    r.max_pos = t.size(0);
    r.rot_dim = static_cast<int32_t>(t.size(1));
  }
  if (q_weight != Py_None) r.q_weight = c.bf16(q_weight, "q_weight", dim);
  if (k_weight != Py_None) r.k_weight = c.bf16(k_weight, "k_weight", dim);
  r.interleaved = PyObject_IsTrue(interleaved);
  r.eps = static_cast<float>(PyFloat_AsDouble(eps));
  if (PyErr_Occurred()) throw Refused();
  return r;
}

// q, k, positions, cos_sin, q_out, k_out, q_weight, k_weight, eps, interleaved, stream
int64_t qk_norm_rope(PyObject* const* a) {
  Call c;
  int64_t tokens = -1, q_heads = -1, kv_heads = -1, dim = -1;
  const ql_rows q = c.rows(a[0], "q", tokens, q_heads, dim), k = c.rows(a[1], "k", tokens, kv_heads, dim);
  const ql_rows q_out = c.rows(a[4], "q_out", tokens, q_heads, dim), k_out = c.rows(a[5], "k_out", tokens, kv_heads, dim);
  const ql_norm_rope r = rule_of(c, a[3], a[6], a[7], dim, a[8], a[9]);
  const int64_t* positions = c.i64(a[2], "positions", tokens);
  const OnDevice on(c);
  return qlinear_qk_norm_rope(&r, tokens, static_cast<int32_t>(q_heads), static_cast<int32_t>(kv_heads),
                              static_cast<int32_t>(dim), &q, &k, positions, &q_out, &k_out, c.stream(a[10]));
}

// q, k, v, positions, slots, cos_sin, q_out, cache, cache device, q_weight, k_weight, eps, interleaved, stream
int64_t qkv_append(PyObject* const* a) {
  Call c;
  const ql_kv_cache* cache = static_cast<const ql_kv_cache*>(Call::number_ptr(a[7]));
  int64_t tokens = -1, q_heads = -1, kv_heads = cache->kv_heads, dim = cache->head_dim;
  const ql_rows k = c.rows(a[1], "k", tokens, kv_heads, dim), v = c.rows(a[2], "v", tokens, kv_heads, dim);
  ql_rows q{}, q_out{};
  if (a[0] != Py_None) {
    q = c.rows(a[0], "q", tokens, q_heads, dim);
    q_out = c.rows(a[6], "q_out", tokens, q_heads, dim);
  } else {
    q_heads = 0;
  }
  c.cache(a[7], a[8]);
  const ql_norm_rope r = rule_of(c, a[5], a[9], a[10], dim, a[11], a[12]);
  const int64_t* positions = c.i64(a[3], "positions", tokens);
  const int64_t* slots = c.i64(a[4], "slots", tokens);
  const OnDevice on(c);
  return qlinear_qkv_append(&r, tokens, static_cast<int32_t>(q_heads), &q, &k, &v, positions, slots, &q_out, cache,
                            c.stream(a[13]));
}

// plan, batch, tokens, q_heads, head_dim, columns, workspace bytes, q, cache, cache device, page_table, seq_lens, cu_q,
// out, lse, workspace, stream
int64_t attention(PyObject* const* a) {
  Call c;
  const int64_t batch = number(a[1]), columns = number(a[5]), need = number(a[6]);
  int64_t tokens = number(a[2]), q_heads = number(a[3]), dim = number(a[4]);
  const ql_rows q = c.rows(a[7], "q", tokens, q_heads, dim), out = c.rows(a[13], "out", tokens, q_heads, dim);
  const ql_kv_cache* cache = c.cache(a[8], a[9]);
  // rows may lie apart (the columns of a larger table), a row's entries not
  const at::Tensor& t = c.tensor(a[10], "page_table", at::kInt, "torch.int32");
  if (t.dim() != 2 || t.size(0) < batch || t.size(1) < columns) {
    PyErr_Format(PyExc_ValueError, "page_table must be a [batch, columns] tensor of at least (%lld, %lld)",
                 (long long)batch, (long long)columns);
    throw Refused();
  }
  if (t.size(1) > 1 && t.stride(1) != 1) refuse("page_table", "must have contiguous rows");
  const int32_t* table = static_cast<const int32_t*>(t.data_ptr());
  const int32_t* lens = c.i32(a[11], "seq_lens", batch);
  const int32_t* cu = c.i32(a[12], "cu_q", batch + 1);
  float* lse = a[14] == Py_None ? nullptr : c.f32_rows(a[14], "lse", tokens, q_heads);
  void* workspace = nullptr;
  if (a[15] != Py_None)
    workspace = c.bytes(a[15], "workspace", need);
  else if (need > 0)
    refuse("workspace", "is required by this plan");
  const OnDevice on(c);
  return qlinear_attention(static_cast<ql_attention_plan>(Call::number_ptr(a[0])), &q, cache, table, t.stride(0), lens, cu,
                           &out, lse, workspace, c.stream(a[16]));
}

// target_probs, draft_probs, draft_tokens, cu_drafts, uniforms, noise, out_tokens, accepted, workspace, stream
int64_t verify_draft(PyObject* const* a) {
  Call c;
  const float* noise = c.f32(a[5], "noise", 0);
  const at::Tensor& e = THPVariable_Unpack(a[5]);
  const int32_t* tokens = c.i32(a[2], "draft_tokens", 0);
  int32_t* out = c.i32(a[6], "out_tokens", 0);
  const at::Tensor& o = THPVariable_Unpack(a[6]);
  if (e.dim() != 2) refuse("noise", "must be a [batch, vocab] tensor");
  const int64_t batch = e.size(0), vocab = e.size(1), n = THPVariable_Unpack(a[2]).numel();
  if (o.dim() != 2 || o.size(0) < batch || o.size(1) < 1)
    refuse("out_tokens", "must be a [batch, max_drafts + 1] tensor");
  const float* target = c.f32_rows(a[0], "target_probs", n + batch, vocab);
  const float* draft = a[1] == Py_None ? nullptr : c.f32_rows(a[1], "draft_probs", n, vocab);
  const int32_t* cu = c.i32(a[3], "cu_drafts", batch + 1);
  const float* uniforms = c.f32(a[4], "uniforms", n);
  int32_t* accepted = c.i32(a[7], "accepted", batch);
  void* workspace = c.bytes(a[8], "workspace", qlinear_verify_workspace_bytes(batch, vocab));
  const OnDevice on(c);
  return qlinear_verify_draft(batch, n, o.size(1) - 1, vocab, target, draft, tokens, cu, uniforms, noise, out, accepted,
                              workspace, c.stream(a[9]));
}

template <int64_t (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLongLong(F(args));
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <int64_t (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {method<qk_norm_rope, 11>("qk_norm_rope"), method<qkv_append, 14>("qkv_append"),
                          method<attention, 17>("attention"), method<verify_draft, 10>("verify_draft"),
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", "Serving operators on torch tensors", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
