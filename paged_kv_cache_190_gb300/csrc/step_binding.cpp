// Python binding of the calls that a serving loop issues every step on small tensors: the
// rotating appends, the windowed / page-scaled / 4-bit decodes, pages read back, and prompts.  Their arguments are checked
// and handed to the C ABI here, in C++: the same checks cost 7 to 15 us a call in Python
// (about 70 attribute reads and a ctypes call of 26 arguments on a Grace core), more than
// the kernels of a small step run; here they cost about one.
//
// Nothing is kept between calls.  Errors: TypeError for a wrong type, ValueError for a
// wrong shape, layout or device; a status of the C ABI is returned for the caller to
// raise.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <string>

#include "../../include/pa.h"

namespace {

struct Refused {
  PyObject* kind;
  std::string what;
};
struct Raised {};   // a Python exception is set

[[noreturn]] void refuse_type(const std::string& what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void refuse(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    PyObject* i = PyNumber_Index(o);                       // numpy integers and the like
    if (!i) {
      PyErr_Clear();
      refuse_type(std::string(name) + " must be an integer");
    }
    const long long w = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (w == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse(std::string(name) + " is out of range");
    }
    return w;
  }
  return v;
}

int int32(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return static_cast<int>(v);
}

// A CUDA tensor on `device` (any CUDA device for < 0), contiguous.
void on_device(const at::Tensor& t, const char* name, int device) {
  if (!t.is_cuda() || !t.is_contiguous() || (device >= 0 && t.get_device() != device))
    refuse(std::string(name) + " must be a contiguous CUDA tensor" + (device >= 0 ? " on the pools' device" : ""));
}

void* vector(PyObject* o, const char* name, int device, at::ScalarType type, int64_t n) {
  const at::Tensor& t = tensor(o, name);
  on_device(t, name, device);
  if (t.scalar_type() != type) refuse_type(std::string(name) + " must be " + c10::toString(type));
  if (t.numel() != n) refuse(std::string(name) + " must have " + std::to_string(n) + " entries");
  return t.data_ptr();
}

int32_t* error_word(PyObject* o, int device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "device_errors");
  on_device(t, "device_errors", device);
  if (t.scalar_type() != at::kInt || t.numel() < 1) refuse_type("device_errors must be an int32 tensor");
  return static_cast<int32_t*>(t.data_ptr());
}

void* stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
  if (!s) throw Raised{};
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!p && PyErr_Occurred()) throw Raised{};
  return p;
}

struct Pools {
  int device;
  int64_t blocks, heads, block_size, head_dim;
  at::ScalarType type;
  void* k;
  void* v;
};

enum Codes { kNoCodes, kE4m3, kE2m1 };

Pools pools(PyObject* ok, PyObject* ov, Codes codes) {
  const at::Tensor &k = tensor(ok, "k_cache"), &v = tensor(ov, "v_cache");
  on_device(k, "k_cache", -1);
  on_device(v, "v_cache", k.get_device());
  if (k.dim() != 4 || v.sizes() != k.sizes())
    refuse("k_cache and v_cache must be [blocks, kv heads, block size, head_dim], alike");
  if (v.scalar_type() != k.scalar_type()) refuse_type("k_cache and v_cache differ in type");
  if (codes == kE4m3 && k.element_size() != 1)
    refuse_type("k_cache and v_cache must hold one-byte e4m3 codes (uint8 or float8_e4m3fn)");
  if (codes == kE2m1) {
    if (k.scalar_type() != at::kByte) refuse_type("k_cache and v_cache must be uint8");
    if (k.size(3) != 72) refuse("k_cache and v_cache must have rows of 72 bytes (128 columns)");
    return {static_cast<int>(k.get_device()), k.size(0), k.size(1), k.size(2), 128, k.scalar_type(),
            k.data_ptr(), v.data_ptr()};
  }
  return {static_cast<int>(k.get_device()), k.size(0), k.size(1), k.size(2), k.size(3), k.scalar_type(),
          k.data_ptr(), v.data_ptr()};
}

float* page_scales(PyObject* o, const char* name, const Pools& p) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != p.blocks || t.size(1) != p.heads)
    refuse_type(std::string(name) + " must be float32 [num_blocks, num_kv_heads]");
  on_device(t, name, p.device);
  return static_cast<float*>(t.data_ptr());
}

// [tokens, heads, head_dim] rows with contiguous heads and columns: their token stride.
int64_t rows(const at::Tensor& t, const char* name, const Pools& p, at::ScalarType type, int64_t tokens, int64_t heads) {
  if (!t.is_cuda() || t.get_device() != p.device || t.dim() != 3)
    refuse(std::string(name) + " must be a CUDA tensor [tokens, heads, head_dim] on the pools' device");
  if (t.scalar_type() != type) refuse_type(std::string(name) + " must be " + c10::toString(type));
  if (t.size(0) != tokens || t.size(1) != heads || t.size(2) != p.head_dim)
    refuse(std::string(name) + " must have " + std::to_string(tokens) + " tokens and " + std::to_string(heads) +
           " heads of head_dim " + std::to_string(p.head_dim));
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != p.head_dim))
    refuse(std::string(name) + ": heads and columns must be contiguous");
  return tokens > 1 ? t.stride(0) : heads * p.head_dim;
}

pa_dtype code_of(at::ScalarType t) {
  if (t == at::kBFloat16) return PA_BF16;
  if (t == at::kFloat) return PA_F32;
  refuse_type("unsupported element type");
}

// A C call with its tensors' device current and the GIL released.
template <typename F>
PyObject* issue(int device, F f) {
  int rc;
  {
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
  }
  return PyLong_FromLong(rc);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// The arguments of a C call as a tuple, for a prepared call.
PyObject* item(const void* p) { return p ? PyLong_FromVoidPtr(const_cast<void*>(p)) : Py_NewRef(Py_None); }
PyObject* item(int64_t v) { return PyLong_FromLongLong(v); }
PyObject* item(int v) { return PyLong_FromLong(v); }
PyObject* item(size_t v) { return PyLong_FromSize_t(v); }
PyObject* item(float v) { return PyFloat_FromDouble(v); }
PyObject* item(pa_dtype v) { return PyLong_FromLong(v); }

template <typename... A>
PyObject* arguments(A... a) {
  PyObject* t = PyTuple_New(sizeof...(A));
  if (!t) throw Raised{};
  Py_ssize_t i = 0;
  bool ok = true;
  ((ok = ok && [&] {
     PyObject* o = item(a);
     if (o) PyTuple_SET_ITEM(t, i++, o);
     return o != nullptr;
   }()), ...);
  if (!ok) {
    Py_DECREF(t);
    throw Raised{};
  }
  return t;
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.kind, r.what.c_str());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// rope_append(kind, q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin,
//             k_scale(s), v_scale(s), interleaved, device_errors, stream, prepare)
// kind 0: pools of the rows' type; 1: e4m3, a scale per head; 2: e4m3, one per page and head; 3: 4-bit rows
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 16) refuse_type("rope_append takes 16 arguments");
    const int kind = int32(integer(a[0], "kind"), "kind");
    const Pools p = pools(a[5], a[6], kind == 3 ? kE2m1 : kind ? kE4m3 : kNoCodes);
    const at::Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
    const at::ScalarType type = kind ? at::kBFloat16 : k.scalar_type();
    const pa_dtype dtype = code_of(type);
    if (kind == 0 && p.type != type) refuse_type("the pools must have the type of k");
    if (k.dim() != 3) refuse("k must be [tokens, heads, head_dim]");
    const int64_t tokens = k.size(0);
    const int64_t ks = rows(k, "k", p, type, tokens, p.heads), vs = rows(v, "v", p, type, tokens, p.heads);
    int64_t heads = 0, qs = 0, rot = 0, most = 0;
    const void* q_ptr = nullptr;
    void* out_ptr = nullptr;
    if (a[1] != Py_None || a[2] != Py_None) {
      if (a[1] == Py_None || a[2] == Py_None) refuse("q and q_out go together");
      const at::Tensor &q = tensor(a[2], "q"), &out = tensor(a[1], "q_out");
      if (q.dim() != 3) refuse("q must be [tokens, heads, head_dim]");
      heads = q.size(1);
      qs = rows(q, "q", p, type, tokens, heads);
      on_device(out, "q_out", p.device);
      if (out.scalar_type() != type) refuse_type("q_out must have q's type");
      if (out.sizes() != q.sizes()) refuse("q_out must have q's shape");
      q_ptr = q.data_ptr();
      out_ptr = out.data_ptr();
    }
    if ((a[8] == Py_None) != (a[9] == Py_None)) refuse("positions and cos_sin go together");
    const int64_t* pos = nullptr;
    const float* table = nullptr;
    if (a[9] != Py_None) {
      const at::Tensor& t = tensor(a[9], "cos_sin");
      if (t.scalar_type() != at::kFloat || t.dim() != 2) refuse_type("cos_sin must be float32 [max_position, rot_dim]");
      on_device(t, "cos_sin", p.device);
      most = t.size(0);
      rot = t.size(1);
      table = static_cast<const float*>(t.data_ptr());
      pos = static_cast<const int64_t*>(vector(a[8], "positions", p.device, at::kLong, tokens));
    }
    const int64_t* slots = static_cast<const int64_t*>(vector(a[7], "slot_mapping", p.device, at::kLong, tokens));
    float *s0 = nullptr, *s1 = nullptr;
    if (kind == 1) {
      s0 = static_cast<float*>(vector(a[10], "k_scale", p.device, at::kFloat, p.heads));
      s1 = static_cast<float*>(vector(a[11], "v_scale", p.device, at::kFloat, p.heads));
    } else if (kind == 2) {
      s0 = page_scales(a[10], "k_scales", p);
      s1 = page_scales(a[11], "v_scales", p);
    }
    const int inter = truth(a[12]);
    int32_t* errs = error_word(a[13], p.device);
    void* stream = stream_of(a[14], p.device);
    const int T = int32(tokens, "tokens"), hq = int32(heads, "heads"), hkv = int32(p.heads, "kv heads"),
              d = int32(p.head_dim, "head_dim"), r = int32(rot, "rot_dim"), m = int32(most, "max_position"),
              bs = int32(p.block_size, "block_size"), nb = int32(p.blocks, "blocks");
    if (truth(a[15])) {
      if (kind == 0)
        return arguments(out_ptr, q_ptr, k.data_ptr(), v.data_ptr(), p.k, p.v, slots, pos, table, qs, ks, vs, T, hq,
                         hkv, d, r, inter, m, bs, nb, dtype, errs, stream);
      if (kind == 3)
        return arguments(out_ptr, q_ptr, k.data_ptr(), v.data_ptr(), p.k, p.v, slots, pos, table, qs, ks, vs, T, hq,
                         hkv, d, r, inter, m, bs, nb, errs, stream);
      return arguments(out_ptr, q_ptr, k.data_ptr(), v.data_ptr(), p.k, p.v, slots, pos, table, s0, s1, qs, ks, vs, T,
                       hq, hkv, d, r, inter, m, bs, nb, errs, stream);
    }
    const void *kp = k.data_ptr(), *vp = v.data_ptr();
    return issue(p.device, [&] {
      if (kind == 0)
        return pa_rope_and_cache(out_ptr, q_ptr, kp, vp, p.k, p.v, slots, pos, table, qs, ks, vs, T, hq, hkv, d, r,
                                 inter, m, bs, nb, dtype, errs, stream);
      if (kind == 1)
        return pa_rope_and_cache_fp8(out_ptr, q_ptr, kp, vp, p.k, p.v, slots, pos, table, s0, s1, qs, ks, vs, T, hq,
                                     hkv, d, r, inter, m, bs, nb, errs, stream);
      if (kind == 3)
        return pa_rope_and_cache_fp4(out_ptr, q_ptr, kp, vp, p.k, p.v, slots, pos, table, qs, ks, vs, T, hq, hkv, d, r,
                                     inter, m, bs, nb, errs, stream);
      return pa_rope_and_cache_fp8_block(out_ptr, q_ptr, kp, vp, p.k, p.v, slots, pos, table, s0, s1, qs, ks, vs, T,
                                         hq, hkv, d, r, inter, m, bs, nb, errs, stream);
    });
  });
}

// span_decode(kind, out, q, k_cache, v_cache, block_tables, context_lens, scale, k_scales,
//             v_scales, num_kv_heads, max_context_len, window, sinks, workspace,
//             device_errors, stream, prepare)
// kind 0: pools of q's type; 1: e4m3, a scale for each page and head; 2: 4-bit rows
PyObject* span_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 18) refuse_type("span_decode takes 18 arguments");
    const int kind = int32(integer(a[0], "kind"), "kind");
    const bool fp8 = kind == 1, fp4 = kind == 2;
    const at::Tensor &out = tensor(a[1], "out"), &q = tensor(a[2], "q");
    const Pools p = pools(a[3], a[4], fp4 ? kE2m1 : fp8 ? kE4m3 : kNoCodes);
    on_device(q, "q", p.device);
    on_device(out, "out", p.device);
    const at::ScalarType type = q.scalar_type();
    const pa_dtype dtype = code_of(type);
    if (kind && dtype != PA_BF16) refuse_type("q and out must be bf16");
    if (!kind && p.type != type) refuse_type("the pools must have the type of q");
    if (q.dim() != 3 && q.dim() != 4) refuse("q must be [B, Hq, D] or [B, q_len, Hq, D]");
    if (out.scalar_type() != type) refuse_type("out must have q's type");
    if (out.sizes() != q.sizes()) refuse("out must have q's shape");
    if (q.size(-1) != p.head_dim) refuse("the pools have another head_dim than q");
    const int64_t heads = integer(a[10], "num_kv_heads");
    if (heads != p.heads) refuse("num_kv_heads does not match the cache shape");
    const int64_t seqs = q.size(0), q_len = q.dim() == 4 ? q.size(1) : 1;
    const at::Tensor& tables = tensor(a[5], "block_tables");
    on_device(tables, "block_tables", p.device);
    if (tables.scalar_type() != at::kInt) refuse_type("block_tables must be int32");
    if (tables.dim() != 2 || tables.size(0) != seqs) refuse("block_tables must have a row for each sequence");
    const int32_t* lens = static_cast<const int32_t*>(vector(a[6], "context_lens", p.device, at::kInt, seqs));
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const float *s0 = nullptr, *s1 = nullptr;
    if (fp8) {
      s0 = page_scales(a[8], "k_scales", p);
      s1 = page_scales(a[9], "v_scales", p);
    }
    const at::Tensor& ws = tensor(a[14], "workspace");
    on_device(ws, "workspace", p.device);
    const size_t ws_bytes = ws.nbytes();
    int32_t* errs = error_word(a[15], p.device);
    void* stream = stream_of(a[16], p.device);
    const int B = int32(seqs, "sequences"), ql = int32(q_len, "q_len"), hq = int32(q.size(-2), "heads"),
              hkv = int32(heads, "num_kv_heads"), d = int32(p.head_dim, "head_dim"),
              bs = int32(p.block_size, "block_size"), nb = int32(p.blocks, "blocks"),
              mb = int32(tables.size(1), "block_tables"), ml = int32(integer(a[11], "max_context_len"), "max_context_len"),
              win = int32(integer(a[12], "window"), "window"), sinks = int32(integer(a[13], "sinks"), "sinks");
    const float sc = static_cast<float>(scale);
    void *op = out.data_ptr(), *wp = ws.data_ptr();
    const void* qp = q.data_ptr();
    const int32_t* tp = static_cast<const int32_t*>(tables.data_ptr());
    if (truth(a[17])) {
      if (fp8)
        return arguments(op, qp, p.k, p.v, tp, lens, sc, s0, s1, hkv, B, hq, ql, d, bs, nb, mb, ml, win, sinks, wp,
                         ws_bytes, errs, stream);
      if (fp4)
        return arguments(op, qp, p.k, p.v, tp, lens, sc, hkv, B, hq, ql, d, bs, nb, mb, ml, win, sinks, wp, ws_bytes,
                         errs, stream);
      return arguments(op, qp, p.k, p.v, tp, lens, sc, hkv, B, hq, ql, d, bs, nb, mb, ml, win, sinks, dtype, wp,
                       ws_bytes, errs, stream);
    }
    return issue(p.device, [&] {
      if (fp8)
        return pa_decode_fp8_block(op, qp, p.k, p.v, tp, lens, sc, s0, s1, hkv, B, hq, ql, d, bs, nb, mb, ml, win,
                                   sinks, wp, ws_bytes, errs, stream);
      if (fp4)
        return pa_decode_fp4(op, qp, p.k, p.v, tp, lens, sc, hkv, B, hq, ql, d, bs, nb, mb, ml, win, sinks, wp,
                             ws_bytes, errs, stream);
      return pa_decode_window(op, qp, p.k, p.v, tp, lens, sc, hkv, B, hq, ql, d, bs, nb, mb, ml, win, sinks, dtype, wp,
                              ws_bytes, errs, stream);
    });
  });
}

// read_pages(k_out, v_out, k_cache, v_cache, src_dst_pairs, device_errors, stream, prepare)
PyObject* read_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) refuse_type("read_pages takes 8 arguments");
    const Pools p = pools(a[2], a[3], kE2m1);
    const at::Tensor &ko = tensor(a[0], "k_out"), &vo = tensor(a[1], "v_out"), &pairs = tensor(a[4], "src_dst_pairs");
    on_device(ko, "k_out", p.device);
    on_device(vo, "v_out", p.device);
    if (ko.scalar_type() != at::kBFloat16 || vo.scalar_type() != at::kBFloat16)
      refuse_type("k_out and v_out must be bf16");
    if (ko.dim() != 4 || vo.sizes() != ko.sizes() || ko.size(1) != p.heads || ko.size(2) != p.block_size ||
        ko.size(3) != p.head_dim)
      refuse("k_out and v_out must be [blocks, kv heads, block size, 128], alike");
    on_device(pairs, "src_dst_pairs", p.device);
    if (pairs.scalar_type() != at::kLong) refuse_type("src_dst_pairs must be int64");
    if (pairs.dim() != 2 || pairs.size(1) != 2) refuse("src_dst_pairs must be [pairs, 2]");
    int32_t* errs = error_word(a[5], p.device);
    void* stream = stream_of(a[6], p.device);
    void *kp = ko.data_ptr(), *vp = vo.data_ptr();
    const int64_t* pp = static_cast<const int64_t*>(pairs.data_ptr());
    const int np = int32(pairs.size(0), "pairs"), hkv = int32(p.heads, "kv heads"), d = int32(p.head_dim, "head_dim"),
              bs = int32(p.block_size, "block_size"), ns = int32(p.blocks, "blocks"), nd = int32(ko.size(0), "blocks");
    if (truth(a[7])) return arguments(kp, vp, p.k, p.v, pp, np, hkv, d, bs, ns, nd, errs, stream);
    return issue(p.device, [&] {
      return pa_read_pages_fp4(kp, vp, p.k, p.v, pp, np, hkv, d, bs, ns, nd, errs, stream);
    });
  });
}

// prefill(out, q, k_cache, v_cache, block_tables, context_lens, q_starts, scale, num_kv_heads,
//         max_context_len, window, sinks, workspace, device_errors, stream, prepare)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 16) refuse_type("prefill takes 16 arguments");
    const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "q");
    const Pools p = pools(a[2], a[3], kNoCodes);
    on_device(q, "q", p.device);
    on_device(out, "out", p.device);
    const at::ScalarType type = q.scalar_type();
    const pa_dtype dtype = code_of(type);
    if (p.type != type) refuse_type("the pools must have the type of q");
    if (q.dim() != 3) refuse("q must be [tokens, Hq, D]");
    if (out.scalar_type() != type) refuse_type("out must have q's type");
    if (out.sizes() != q.sizes()) refuse("out must have q's shape");
    if (q.size(2) != p.head_dim) refuse("the pools have another head_dim than q");
    const int64_t heads = integer(a[8], "num_kv_heads");
    if (heads != p.heads) refuse("num_kv_heads does not match the cache shape");
    const at::Tensor& tables = tensor(a[4], "block_tables");
    on_device(tables, "block_tables", p.device);
    if (tables.scalar_type() != at::kInt) refuse_type("block_tables must be int32");
    if (tables.dim() != 2) refuse("block_tables must be [sequences, pages]");
    const int64_t seqs = tables.size(0);
    const int32_t* lens = static_cast<const int32_t*>(vector(a[5], "context_lens", p.device, at::kInt, seqs));
    const int32_t* starts = static_cast<const int32_t*>(vector(a[6], "q_starts", p.device, at::kInt, seqs + 1));
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const at::Tensor& ws = tensor(a[12], "workspace");
    on_device(ws, "workspace", p.device);
    const size_t ws_bytes = ws.nbytes();
    int32_t* errs = error_word(a[13], p.device);
    void* stream = stream_of(a[14], p.device);
    const int B = int32(seqs, "sequences"), T = int32(q.size(0), "tokens"), hq = int32(q.size(1), "heads"),
              hkv = int32(heads, "num_kv_heads"), d = int32(p.head_dim, "head_dim"),
              bs = int32(p.block_size, "block_size"), nb = int32(p.blocks, "blocks"),
              mb = int32(tables.size(1), "block_tables"), ml = int32(integer(a[9], "max_context_len"), "max_context_len"),
              win = int32(integer(a[10], "window"), "window"), sinks = int32(integer(a[11], "sinks"), "sinks");
    const float sc = static_cast<float>(scale);
    void *op = out.data_ptr(), *wp = ws.data_ptr();
    const void* qp = q.data_ptr();
    const int32_t* tp = static_cast<const int32_t*>(tables.data_ptr());
    if (truth(a[15]))
      return arguments(op, qp, p.k, p.v, tp, lens, starts, sc, hkv, B, T, hq, d, bs, nb, mb, ml, win, sinks, dtype, wp,
                       ws_bytes, errs, stream);
    return issue(p.device, [&] {
      return pa_prefill(op, qp, p.k, p.v, tp, lens, starts, sc, hkv, B, T, hq, d, bs, nb, mb, ml, win, sinks, dtype, wp,
                        ws_bytes, errs, stream);
    });
  });
}

PyMethodDef methods[] = {
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope_append)), METH_FASTCALL, nullptr},
    {"span_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(span_decode)), METH_FASTCALL, nullptr},
    {"read_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(read_pages)), METH_FASTCALL, nullptr},
    {"prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prefill)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step", "Checked per-step calls of libpagedattn.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step() { return PyModule_Create(&module); }
