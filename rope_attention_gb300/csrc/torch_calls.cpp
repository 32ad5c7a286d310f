// packed_attention, paged_attention and kv_cache_read called with torch tensors: the checks of
// the binding's other calls (placement, dtype, contiguity, size) and the C call behind them.
//
// One decode step's attention runs for about 10 us on the device; the same checks written with
// a tensor's Python attributes took 14 us (twelve tensors, five calls into torch each), so the
// host bounded it.  Here they take under one.  The functions give the C call's status; the
// Python side raises for it.  Parameter structs come in as buffers (ctypes structures).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <exception>
#include <string>

#include "rope_attention.h"

namespace {

// a refusal: the ValueError (or TypeError) is set
struct Refused {};
[[noreturn]] void refuse(const std::string& what, PyObject* kind = PyExc_ValueError) {
  PyErr_SetString(kind, what.c_str());
  throw Refused{};
}

const char* dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kByte: return "torch.uint8";
    case at::kChar: return "torch.int8";
    case at::kShort: return "torch.int16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kBool: return "torch.bool";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    case at::kFloat8_e5m2: return "torch.float8_e5m2";
    default: return c10::toString(t);
  }
}

// the dtypes that an argument may have: two at most (the same twice for one); none: any, the
// parameters name none and the library answers for them
struct Types {
  at::ScalarType other, main;
  bool any;
};
constexpr Types one(at::ScalarType t) { return {t, t, false}; }
Types half_type(int32_t code) {
  return code == RA_BF16 ? one(at::kBFloat16) : code == RA_FP16 ? one(at::kHalf) : Types{at::kHalf, at::kHalf, true};
}
Types stored_type(int32_t code) {
  switch (code) {
    case RA_BF16: return one(at::kBFloat16);
    case RA_FP16: return one(at::kHalf);
    case RA_INT8: return one(at::kChar);
    case RA_FP8_E4M3: return {at::kByte, at::kFloat8_e4m3fn, false};
    case RA_FP8_E5M2: return {at::kByte, at::kFloat8_e5m2, false};
    default: return {at::kByte, at::kByte, true};
  }
}
int64_t stored_bytes(int32_t code) { return code == RA_BF16 || code == RA_FP16 ? 2 : 1; }

const at::Tensor* tensor_of(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None) {
    if (optional) return nullptr;
    refuse(std::string(name) + ": expected a tensor, got None", PyExc_TypeError);
  }
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": expected a tensor", PyExc_TypeError);
  return &THPVariable_Unpack(o);
}

// Looks a call's tensors over, one after the other, and remembers the first that is not on
// the current device: sizes, dtypes and layouts of all come before that complaint.
class Args {
 public:
  // contiguous, with at least `need` bytes
  void* flat(PyObject* o, const char* name, int64_t need, Types types, bool optional = false) {
    const at::Tensor* t = tensor_of(o, name, optional);
    if (t == nullptr) return nullptr;
    if (static_cast<int64_t>(t->nbytes()) < need)
      refuse(std::string(name) + ": the call needs " + std::to_string(need) + " bytes, the tensor holds " +
             std::to_string(t->nbytes()));
    look(*t, name, types);
    if (!t->is_contiguous()) refuse(std::string(name) + ": expected a contiguous tensor");
    return t->data_ptr();
  }
  // [tokens, heads, d] of 16-bit elements with these strides, or any tensor whose storage holds
  // what they address
  void* strided(PyObject* o, const char* name, int64_t tokens, int64_t heads, int64_t d, int64_t ts, int64_t hs, Types types) {
    const at::Tensor& t = *tensor_of(o, name);
    if (!(t.dim() == 3 && t.size(0) == tokens && t.size(1) == heads && t.size(2) == d && t.stride(0) == ts &&
          t.stride(1) == hs && t.stride(2) == 1)) {
      // (parameters out of range are the library's to refuse: no byte count overflows here)
      const __int128 need = ((static_cast<__int128>(std::max<int64_t>(tokens, 1)) - 1) * ts +
                             (static_cast<__int128>(std::max<int64_t>(heads, 1)) - 1) * hs + d) * 2;
      const int64_t held = static_cast<int64_t>(t.storage().nbytes()) - t.storage_offset() * t.element_size();
      if (held < need)
        refuse(std::string(name) + ": the call needs " + std::to_string(static_cast<int64_t>(std::min<__int128>(need, INT64_MAX))) +
               " bytes, the tensor's storage holds " + std::to_string(held));
    }
    look(t, name, types);
    return t.data_ptr();
  }
  // the stream of the call: given (an int or a Stream), or the current one
  void* stream(PyObject* o) {
    if (apart_ != nullptr) {
      if (!apart_->is_cuda()) refuse(apart_name_ + ": expected a CUDA tensor");
      refuse(apart_name_ + ": on " + apart_->device().str() + ", the current device is cuda:" +
             std::to_string(c10::cuda::current_device()));
    }
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev_).stream();
    PyObject* held = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Index(o);
    if (held == nullptr) throw Refused{};
    void* s = PyLong_AsVoidPtr(held);
    Py_DECREF(held);
    if (PyErr_Occurred()) throw Refused{};
    return s;
  }

 private:
  void look(const at::Tensor& t, const char* name, Types types) {
    if (!types.any && t.scalar_type() != types.main && t.scalar_type() != types.other)
      refuse(std::string(name) + ": expected " + dtype_name(types.main) + ", got " + dtype_name(t.scalar_type()));
    if (apart_ != nullptr || (dev_ >= 0 && t.is_cuda() && t.get_device() == dev_)) return;
    if (dev_ < 0 && t.is_cuda() && t.get_device() == c10::cuda::current_device()) {
      dev_ = t.get_device();
      return;
    }
    apart_ = &t;
    apart_name_ = name;
  }
  const at::Tensor* apart_ = nullptr;
  std::string apart_name_;
  c10::DeviceIndex dev_ = -1;
};

// a parameter struct out of the ctypes structure of that name, copied
template <class P>
P params_of(PyObject* o, const char* name) {
  Py_buffer b;
  if (std::strcmp(Py_TYPE(o)->tp_name, name) != 0) refuse(std::string("params: expected a ") + name, PyExc_TypeError);
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Refused{};
  const bool fits = b.len == static_cast<Py_ssize_t>(sizeof(P));
  P p;
  if (fits) std::copy_n(static_cast<const uint8_t*>(b.buf), sizeof(P), reinterpret_cast<uint8_t*>(&p));
  PyBuffer_Release(&b);
  if (!fits) refuse(std::string("params: ") + name + " has another size here", PyExc_TypeError);
  return p;
}

// Bytes of the caches and of each one's scale or offset.  Parameters that the library rejects
// give meaningless ones; they wrap, and its own checks answer for them.
struct CacheBytes {
  int64_t k, ckv, k_quant, ckv_quant, kw, cw;
};
CacheBytes cache_bytes(const kv_rms_norm_rope_cache_params& p) {
  const auto u = [](int64_t x) { return static_cast<uint64_t>(std::max<int64_t>(x, 0)); };
  const bool v1 = p.variant == 1;
  const uint64_t kw = v1 ? u(p.rope_size) : u(p.Dkv), cw = v1 ? u(p.Dkv - p.rope_size) : u(p.Dv);
  const uint64_t rows = (p.cache_mode == RA_CACHE_NORM ? u(p.B) * u(p.cache_seq_len) : u(p.block_num) * u(p.block_size)) * u(p.N);
  const uint64_t qk = v1 ? (p.k_quant_scalar ? 1 : kw) : u(p.N) * kw, qv = v1 ? (p.c_kv_quant_scalar ? 1 : cw) : u(p.N) * cw;
  return {static_cast<int64_t>(rows * kw) * stored_bytes(p.k_cache_dtype),
          static_cast<int64_t>(rows * cw) * stored_bytes(p.ckv_cache_dtype), static_cast<int64_t>(qk * 4),
          static_cast<int64_t>(qv * 4), static_cast<int64_t>(kw), static_cast<int64_t>(cw)};
}
int64_t times(int64_t a, int64_t b, int64_t c = 1) {  // as above
  return static_cast<int64_t>(static_cast<uint64_t>(a) * static_cast<uint64_t>(b) * static_cast<uint64_t>(c));
}

// runs f, which gives a status, behind the boundary that no C++ exception passes
template <class F>
PyObject* guarded(F&& f) {
  try {
    return PyLong_FromLong(f());
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
bool count_ok(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return n == want;
}

// (q, k, v, out, B, causal, softmax_scale or None) -> the bytes of a packed_attention_params
PyObject* packed_params(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 7)) return nullptr;
  try {
    static const char* const names[4] = {"q", "k", "v", "out"};
    const at::Tensor* t[4];
    for (int i = 0; i < 4; ++i) t[i] = tensor_of(a[i], names[i]);
    for (int i = 0; i < 4; ++i) {
      const at::Tensor &x = *t[i], &like = *t[i == 0 || i == 3 ? 0 : 1], &q = *t[0];
      if (x.dim() != 3 || like.dim() != 3 || q.dim() != 3) refuse(std::string(names[x.dim() != 3 ? i : 0]) + ": expected [tokens, heads, head_dim]");
      const at::Tensor* differs = x.sizes() != like.sizes() ? &like : x.size(2) != q.size(2) ? &q : nullptr;
      if (differs != nullptr) {
        const auto shape = [](const at::Tensor& s) {
          return "(" + std::to_string(s.size(0)) + ", " + std::to_string(s.size(1)) + ", " + std::to_string(s.size(2)) + ")";
        };
        refuse(std::string(names[i]) + ": shape " + shape(x) + " does not match " + shape(*differs));
      }
      if (x.scalar_type() != q.scalar_type())
        refuse(std::string(names[i]) + ": expected " + dtype_name(q.scalar_type()) + ", got " + dtype_name(x.scalar_type()));
      if (x.size(2) > 1 && x.stride(2) != 1) refuse(std::string(names[i]) + ": the last dimension must be contiguous");
    }
    const at::ScalarType st = t[0]->scalar_type();
    if (st != at::kBFloat16 && st != at::kHalf)
      refuse(std::string("q: expected bfloat16 or float16, got ") + dtype_name(st));
    packed_attention_params p{};
    p.B = PyLong_AsLongLong(a[4]);
    p.total_q = t[0]->size(0);
    p.total_k = t[1]->size(0);
    const int64_t heads[2] = {t[0]->size(1), t[1]->size(1)}, d = t[0]->size(2);
    for (const int64_t x : {heads[0], heads[1], d})
      if (x > INT32_MAX) refuse("q: more heads or channels than 31 bits count");
    p.num_heads = static_cast<int32_t>(heads[0]);
    p.num_kv_heads = static_cast<int32_t>(heads[1]);
    p.head_dim = static_cast<int32_t>(d);
    p.dtype = st == at::kBFloat16 ? RA_BF16 : RA_FP16;
    p.causal = PyObject_IsTrue(a[5]);
    p.softmax_scale = static_cast<float>(a[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : PyFloat_AsDouble(a[6]));
    int64_t* const strides[4] = {&p.q_token_stride, &p.k_token_stride, &p.v_token_stride, &p.out_token_stride};
    for (int i = 0; i < 4; ++i) {
      strides[i][0] = t[i]->stride(0);
      strides[i][1] = t[i]->stride(1);
    }
    if (PyErr_Occurred()) return nullptr;
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&p), sizeof(p));
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (params, q, k, v, out, workspace, lse, cu_seqlens_q, cu_seqlens_k, stream)
PyObject* packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 10)) return nullptr;
  return guarded([&] {
    const auto p = params_of<packed_attention_params>(a[0], "PackedAttentionParams");
    const Types half = p.dtype == RA_FP16 ? one(at::kHalf) : p.dtype == RA_BF16 ? one(at::kBFloat16) : Types{at::kBFloat16, at::kHalf, false};
    Args args;
    auto* q = static_cast<uint16_t*>(args.strided(a[1], "q", p.total_q, p.num_heads, p.head_dim, p.q_token_stride, p.q_head_stride, half));
    auto* k = static_cast<uint16_t*>(args.strided(a[2], "k", p.total_k, p.num_kv_heads, p.head_dim, p.k_token_stride, p.k_head_stride, half));
    auto* v = static_cast<uint16_t*>(args.strided(a[3], "v", p.total_k, p.num_kv_heads, p.head_dim, p.v_token_stride, p.v_head_stride, half));
    auto* out = static_cast<uint16_t*>(args.strided(a[4], "out", p.total_q, p.num_heads, p.head_dim, p.out_token_stride, p.out_head_stride, half));
    auto* lse = static_cast<float*>(args.flat(a[6], "lse", times(p.total_q, p.num_heads, 4), one(at::kFloat), true));
    auto* cq = static_cast<int32_t*>(args.flat(a[7], "cu_seqlens_q", times(p.B + 1, 4), one(at::kInt), true));
    auto* ck = static_cast<int32_t*>(args.flat(a[8], "cu_seqlens_k", times(p.B + 1, 4), one(at::kInt), true));
    void* ws = args.flat(a[5], "workspace", 0, one(at::kByte));
    const size_t room = THPVariable_Unpack(a[5]).nbytes();
    void* stream = args.stream(a[9]);
    ra_status st;
    Py_BEGIN_ALLOW_THREADS
    st = packed_attention(&p, q, k, v, out, lse, cq, ck, ws, room, stream);
    Py_END_ALLOW_THREADS
    return static_cast<long>(st);
  });
}

// (cache, params, q, k_cache, ckv_cache, seq_lens, out, workspace, block_table, cu_seqlens_q,
//  k_rope_scale, c_kv_scale, k_rope_offset, c_kv_offset, lse, dev_error_count, stream)
PyObject* paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 17)) return nullptr;
  return guarded([&] {
    const auto c = params_of<kv_rms_norm_rope_cache_params>(a[0], "KvRmsNormRopeCacheParams");
    auto p = params_of<paged_attention_params>(a[1], "PagedAttentionParams");
    if (const at::Tensor* t = tensor_of(a[8], "block_table", true)) {
      if (t->dim() != 2 || t->size(0) != p.B) {
        std::string shape;
        for (const int64_t s : t->sizes()) shape += (shape.empty() ? "" : ", ") + std::to_string(s);
        refuse("block_table: expected [" + std::to_string(p.B) + ", pages], got (" + shape + (t->dim() == 1 ? ",)" : ")"));
      }
      if (p.block_table_stride == 0) p.block_table_stride = t->size(1);
    }
    const Types half = half_type(c.kv_dtype);
    const CacheBytes x = cache_bytes(c);
    const int64_t rows = times(p.total_q, p.num_heads);
    Args args;
    auto* q = static_cast<uint16_t*>(args.flat(a[2], "q", times(rows, c.Dkv, 2), half));
    void* kc = args.flat(a[3], "k_cache", x.k, stored_type(c.k_cache_dtype));
    void* vc = args.flat(a[4], "ckv_cache", x.ckv, stored_type(c.ckv_cache_dtype));
    auto* lens = static_cast<int32_t*>(args.flat(a[5], "seq_lens", times(p.B, 4), one(at::kInt)));
    auto* table = static_cast<int32_t*>(args.flat(a[8], "block_table", times(p.B, p.block_table_stride, 4), one(at::kInt), true));
    auto* cq = static_cast<int32_t*>(args.flat(a[9], "cu_seqlens_q", times(p.B + 1, 4), one(at::kInt), true));
    auto* ks = static_cast<float*>(args.flat(a[10], "k_rope_scale", x.k_quant, one(at::kFloat), true));
    auto* vs = static_cast<float*>(args.flat(a[11], "c_kv_scale", x.ckv_quant, one(at::kFloat), true));
    auto* ko = static_cast<float*>(args.flat(a[12], "k_rope_offset", x.k_quant, one(at::kFloat), true));
    auto* vo = static_cast<float*>(args.flat(a[13], "c_kv_offset", x.ckv_quant, one(at::kFloat), true));
    auto* out = static_cast<uint16_t*>(args.flat(a[6], "out", times(rows, c.Dv, 2), half));
    auto* lse = static_cast<float*>(args.flat(a[14], "lse", times(rows, 4), one(at::kFloat), true));
    auto* err = static_cast<int32_t*>(args.flat(a[15], "dev_error_count", 4, one(at::kInt), true));
    void* ws = args.flat(a[7], "workspace", 0, one(at::kByte));
    const size_t room = THPVariable_Unpack(a[7]).nbytes();
    void* stream = args.stream(a[16]);
    ra_status st;
    Py_BEGIN_ALLOW_THREADS
    st = paged_attention(&c, &p, q, kc, vc, lens, table, cq, ks, vs, ko, vo, out, lse, err, ws, room, stream);
    Py_END_ALLOW_THREADS
    return static_cast<long>(st);
  });
}

// (params, index, k_cache, ckv_cache, k_out, c_kv_out, k_rope_scale, c_kv_scale, k_rope_offset,
//  c_kv_offset, dev_error_count, stream)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_ok(n, 12)) return nullptr;
  return guarded([&] {
    const auto c = params_of<kv_rms_norm_rope_cache_params>(a[0], "KvRmsNormRopeCacheParams");
    const Types half = half_type(c.kv_dtype);
    const CacheBytes x = cache_bytes(c);
    const int64_t bs = std::max<int64_t>(c.block_size, 1), rows = times(c.B, c.N, c.S);
    const int64_t entries = times(c.B, c.cache_mode == RA_CACHE_PA_BLK_BNSD ? (c.S - 1) / bs + 1 : c.S);
    Args args;
    auto* index = static_cast<int64_t*>(args.flat(a[1], "index", times(entries, 8), one(at::kLong)));
    void* kc = args.flat(a[2], "k_cache", x.k, stored_type(c.k_cache_dtype), true);
    void* vc = args.flat(a[3], "ckv_cache", x.ckv, stored_type(c.ckv_cache_dtype), true);
    auto* ks = static_cast<float*>(args.flat(a[6], "k_rope_scale", x.k_quant, one(at::kFloat), true));
    auto* vs = static_cast<float*>(args.flat(a[7], "c_kv_scale", x.ckv_quant, one(at::kFloat), true));
    auto* ko = static_cast<float*>(args.flat(a[8], "k_rope_offset", x.k_quant, one(at::kFloat), true));
    auto* vo = static_cast<float*>(args.flat(a[9], "c_kv_offset", x.ckv_quant, one(at::kFloat), true));
    auto* k = static_cast<uint16_t*>(args.flat(a[4], "k_out", times(rows, x.kw, 2), half, true));
    auto* v = static_cast<uint16_t*>(args.flat(a[5], "c_kv_out", times(rows, x.cw, 2), half, true));
    auto* err = static_cast<int32_t*>(args.flat(a[10], "dev_error_count", 4, one(at::kInt), true));
    void* stream = args.stream(a[11]);
    ra_status st;
    Py_BEGIN_ALLOW_THREADS
    st = kv_cache_read(&c, index, kc, vc, ks, vs, ko, vo, k, v, err, stream);
    Py_END_ALLOW_THREADS
    return static_cast<long>(st);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}
PyMethodDef methods[] = {{"packed_params", fast<packed_params>(), METH_FASTCALL, nullptr},
                         {"packed_attention", fast<packed>(), METH_FASTCALL, nullptr},
                         {"paged_attention", fast<paged>(), METH_FASTCALL, nullptr},
                         {"kv_cache_read", fast<read>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module_def); }
