// Python binding of the cache operators: argument checks, outputs and the call
// of the C ABI (include/mla_dcp.h), in one native step.  Their kernels are as
// short as a launch, and a call through ctypes spent 10 to 20 us on its checks
// and on converting thirty arguments; here it is the launch and about 2 us.
//
// Each function takes its arguments by position (api.py gives them names and
// documents them) and returns the library's status first, then its tensors.
// Wrong types raise TypeError, wrong shapes, strides and devices ValueError.
#include <ATen/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <mutex>
#include <optional>
#include <string>
#include <vector>

#include "../../include/mla_dcp.h"

namespace {

constexpr int64_t kLatent = MLA_D_LATENT, kRope = MLA_D_ROPE, kQk = MLA_D_QK, kE2m1 = MLA_E2M1_ROW_BYTES;

struct Error {
  PyObject* type;
  std::string text;
};
[[noreturn]] void bad_value(std::string s) { throw Error{PyExc_ValueError, std::move(s)}; }
[[noreturn]] void bad_type(std::string s) { throw Error{PyExc_TypeError, std::move(s)}; }
struct PythonError {};   // one that the interpreter has set already

using Shape = std::initializer_list<int64_t>;

std::string words(c10::IntArrayRef s) {
  std::string o = "[";
  for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
  return o + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// None: nullptr
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}

int small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) bad_value(std::string(name) + " is out of range");
  return static_cast<int>(v);
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(v);
}

int fits(int64_t v, const char* name) {
  if (v > INT32_MAX) bad_value(std::string(name) + " is too large");
  return static_cast<int>(v);
}

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) bad_value(std::string(name) + " must be a CUDA tensor");
  return t.get_device();
}

void on(const at::Tensor& t, int dev, const char* name) {
  if (!t.is_cuda() || t.get_device() != dev)
    bad_value(std::string(name) + " must be a CUDA tensor on device " + std::to_string(dev));
}

void on(const at::Tensor& t, int dev, const char* name, at::ScalarType dt) {
  on(t, dev, name);
  if (t.scalar_type() != dt)
    bad_type(std::string(name) + " must be " + c10::toString(dt) + ", not " + c10::toString(t.scalar_type()));
}

void dense(const at::Tensor& t, int dev, const char* name, at::ScalarType dt, Shape shape) {
  on(t, dev, name, dt);
  if (t.sizes() != c10::IntArrayRef(shape) || !t.is_contiguous())
    bad_value(std::string(name) + " must be a contiguous tensor of shape " + words(shape) + ", not " + words(t.sizes()));
}

int32_t* error_word(const at::Tensor* t, int dev) {
  if (!t) return nullptr;
  on(*t, dev, "err_flag", at::kInt);
  if (t->numel() < 1) bad_value("err_flag must hold one int32");
  return static_cast<int32_t*>(t->data_ptr());
}

// Elements from one index of dimension d to the next (a dimension of one may
// have any stride: none is needed).
int64_t step(const at::Tensor& t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

int dtype_code(at::ScalarType dt) {
  switch (dt) {
    case at::kBFloat16: return MLA_BF16;
    case at::kHalf: return MLA_FP16;
    case at::kFloat: return MLA_FP32;
    default: bad_type(std::string("unsupported dtype ") + c10::toString(dt));
  }
}

// The library takes the stream's handle; None is the device's current stream.
struct Stream {
  c10::cuda::CUDAStream s;
  mla_stream_t raw() const { return reinterpret_cast<mla_stream_t>(s.stream()); }
};

Stream stream_of(PyObject* o, int dev) {
  if (o == Py_None) return {c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev))};
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw PythonError{};
  const int64_t v = PyLong_AsLongLong(h);
  Py_DECREF(h);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return {c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(v), static_cast<c10::DeviceIndex>(dev))};
}

// (past the dispatcher, which has nothing to choose here)
at::Tensor make(c10::IntArrayRef shape, at::ScalarType dt, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(shape, dt, like.device(), std::nullopt));
}

// A new tensor of the call's stream, whose work orders its memory: a block of the
// current stream could be one that it has given up but still works on.
at::Tensor make_on(const Stream& stream, c10::IntArrayRef shape, at::ScalarType dt, const at::Tensor& like) {
  const c10::cuda::CUDAStreamGuard guard(stream.s);
  return make(shape, dt, like);
}

// An output for the caller: made on the call's stream, and, where another one is
// current, marked as used there too, as that is where a caller goes on with it.
at::Tensor output(const Stream& stream, c10::IntArrayRef shape, at::ScalarType dt, const at::Tensor& like) {
  const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(like.get_device());
  if (current.stream() == stream.s.stream()) return make(shape, dt, like);
  at::Tensor t = make_on(stream, shape, dt, like);
  if (t.numel() > 0) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
  return t;
}

PyObject* result(int status, std::initializer_list<std::optional<at::Tensor>> out) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(out.size()) + 1);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (const auto& t : out) {
    PyObject* o = t ? THPVariable_Wrap(*t) : (Py_INCREF(Py_None), Py_None);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Runs f and turns its exceptions into Python's: none leaves a C entry.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const PythonError&) {
  } catch (const Error& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ---------------------------------------------------------------- append
// c_kv, k_pe, kv_cache, slots, positions, cos_sin, norm_weight, eps, q_pe, q_out,
// kv_out (None, "new" or a tensor), kv_scale, interleaved, sections, err_flag, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const at::Tensor &c_kv = tensor(a[0], "c_kv"), &k_pe = tensor(a[1], "k_pe"), &cache = tensor(a[2], "kv_cache");
    const at::Tensor &slots = tensor(a[3], "slots"), &positions = tensor(a[4], "positions");
    const at::Tensor& cos_sin = tensor(a[5], "cos_sin");
    const at::Tensor *weight = maybe(a[6], "norm_weight"), *q_pe = maybe(a[8], "q_pe"), *err = maybe(a[14], "err_flag");
    const int dev = device_of(c_kv, "c_kv");
    const at::ScalarType dt = c_kv.scalar_type();
    const int code = dtype_code(dt);
    if (c_kv.dim() != 2 || c_kv.size(1) != kLatent || c_kv.stride(1) != 1)
      bad_value("c_kv must be [T, 512] with unit stride along its rows");
    const int64_t T = c_kv.size(0);
    on(k_pe, dev, "k_pe", dt);
    if (k_pe.dim() != 2 || k_pe.size(0) != T || k_pe.size(1) != kRope || k_pe.stride(1) != 1)
      bad_value("k_pe must be [T, 64] with unit stride along its rows");
    on(cache, dev, "kv_cache");
    if (cache.dim() != 3 || !cache.is_contiguous())
      bad_value("kv_cache must be a contiguous [num_blocks, block_size, W] tensor");
    const int64_t W = cache.size(2);
    const at::ScalarType ct = cache.scalar_type();
    int fmt;
    if (ct == at::kByte && W == kE2m1) fmt = MLA_KV_E2M1;
    else if (ct == dt && W == kQk) fmt = MLA_KV_MODEL;
    else if ((ct == at::kByte || ct == at::kFloat8_e4m3fn) && W == kQk) fmt = MLA_KV_E4M3;
    else bad_type("no cache format has rows of " + std::to_string(W) + " " + c10::toString(ct) + " for " + c10::toString(dt));
    if (fmt == MLA_KV_MODEL && a[11] != Py_None) bad_type("kv_scale applies to an E4M3 or E2M1 cache only");
    dense(slots, dev, "slots", at::kInt, {T});
    if (!PyTuple_Check(a[13])) bad_type("sections must be a tuple");
    const int64_t axes = PyTuple_GET_SIZE(a[13]);
    if (axes < 1 || axes > 3) bad_value("one to three position axes");
    int32_t sections[3] = {0, 0, 0};
    for (int64_t i = 0; i < axes; ++i) sections[i] = small(PyTuple_GET_ITEM(a[13], i), "sections");
    if (positions.dim() == 1 && axes == 1) dense(positions, dev, "positions", at::kInt, {T});
    else dense(positions, dev, "positions", at::kInt, {axes, T});
    on(cos_sin, dev, "cos_sin", at::kFloat);
    if (cos_sin.dim() != 2 || cos_sin.size(1) != kRope || !cos_sin.is_contiguous())
      bad_value("cos_sin must be a contiguous [max_pos, 64] tensor");
    if (weight) dense(*weight, dev, "norm_weight", dt, {kLatent});
    int32_t* err_word = error_word(err, dev);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const Stream stream = stream_of(a[15], dev);
    std::optional<at::Tensor> q_out, kv_out;
    int64_t H = 0, qs = 0, qh = 0, os = 0, oh = 0;
    if (q_pe) {
      on(*q_pe, dev, "q_pe", dt);
      if (q_pe->dim() != 3 || q_pe->size(0) != T || q_pe->size(2) != kRope || q_pe->stride(2) != 1)
        bad_value("q_pe must be [T, H, 64] with unit stride along its heads");
      H = q_pe->size(1);
      if (a[9] == Py_None) {
        q_out = output(stream, {T, H, kRope}, dt, c_kv);
      } else {
        q_out = tensor(a[9], "q_out");
        on(*q_out, dev, "q_out", dt);
        if (q_out->sizes() != q_pe->sizes() || q_out->stride(2) != 1)
          bad_value("q_out must be [T, H, 64] with unit stride along its heads");
      }
      qs = step(*q_pe, 0), qh = step(*q_pe, 1), os = step(*q_out, 0), oh = step(*q_out, 1);
    } else if (a[9] != Py_None) {
      bad_value("q_out without q_pe");
    }
    const at::ScalarType kt = fmt == MLA_KV_E4M3 ? ct : dt;
    if (PyUnicode_Check(a[10])) {
      if (PyUnicode_CompareWithASCIIString(a[10], "new") != 0) bad_value("kv_out must be None, 'new' or a tensor");
      kv_out = output(stream, {T, kQk}, kt, c_kv);
    } else if (a[10] != Py_None) {
      kv_out = tensor(a[10], "kv_out");
      on(*kv_out, dev, "kv_out", kt);
      if (kv_out->numel() != T * kQk || !kv_out->is_contiguous()) bad_value("kv_out must be a contiguous [T, 576] tensor");
    }
    const int interleaved = PyObject_IsTrue(a[12]);
    if (interleaved < 0) throw PythonError{};
    int st = MLA_OK;
    if (T > 0)
      st = mla_kv_append(c_kv.data_ptr(), step(c_kv, 0), k_pe.data_ptr(), step(k_pe, 0), ptr(weight), number(a[7]),
                         ptr(q_pe), qs, qh, static_cast<const int32_t*>(positions.data_ptr()), static_cast<int>(axes),
                         sections, static_cast<const float*>(cos_sin.data_ptr()), fits(cos_sin.size(0), "max_pos"),
                         interleaved, static_cast<const int32_t*>(slots.data_ptr()), fits(T, "T"),
                         fits(H, "H"), fits(cache.size(0), "num_blocks"), fits(cache.size(1), "block_size"), code, fmt,
                         a[11] == Py_None ? 1.f : number(a[11]), cache.data_ptr(), q_out ? q_out->data_ptr() : nullptr, os,
                         oh, kv_out ? kv_out->data_ptr() : nullptr, err_word, stream.raw());
    return result(st, {q_out, kv_out});
  });
}

// ---------------------------------------------------------------- partials over E2M1 pages
// The default workspace: one per (device, stream), as calls on one stream run
// one after another; its size depends on the device alone.  A captured call gets
// one of its own, from its graph's memory: graphs captured on one stream may
// replay at once on others.  (Never destroyed: at the interpreter's end the
// allocator may be gone first.)
at::Tensor default_workspace(const at::Tensor& like, int dev, const Stream& stream, int B, int q_len, int shards, int cur) {
  static auto* kept = new std::map<std::pair<int, const void*>, at::Tensor>();
  static std::mutex mu;
  const std::pair<int, const void*> key{dev, stream.raw()};
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaStreamIsCapturing(stream.s.stream(), &capture);
  const bool keep = capture == cudaStreamCaptureStatusNone;
  std::lock_guard<std::mutex> lock(mu);
  const auto it = kept->find(key);
  if (keep && it != kept->end()) return it->second;
  const uint64_t need = mla_dcp_decode_partial_fp4_workspace_size(B, q_len, shards, cur);
  if (need == 0) return at::Tensor();   // invalid sizes: the call itself reports them
  at::Tensor t = make_on(stream, {static_cast<int64_t>(need)}, at::kByte, like);
  if (keep) kept->emplace(key, t);
  return t;
}

// q_abs, q_pe, kv_cache, block_table, seq_lens, num_shards, kv_cur, scale, part_dtype
// (a torch dtype or None), o_part, lse_part, err_flag, workspace ("default", a tensor
// or None), head_slices, kv_scale, stream
PyObject* partial_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const at::Tensor &q_abs = tensor(a[0], "q_abs"), &q_pe = tensor(a[1], "q_pe"), &cache = tensor(a[2], "kv_cache");
    const at::Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
    const at::Tensor *cur = maybe(a[6], "kv_cur"), *err = maybe(a[11], "err_flag");
    const int dev = device_of(q_abs, "q_abs");
    const at::ScalarType dt = q_abs.scalar_type();
    if (q_abs.dim() != 4) bad_value("q_abs must be [B, q, H, 512]");
    const int64_t B = q_abs.size(0), q_len = q_abs.size(1), H = q_abs.size(2);
    const int64_t shards = small(a[5], "num_shards"), slices = small(a[13], "head_slices");
    dense(q_abs, dev, "q_abs", dt, {B, q_len, H, kLatent});
    dense(q_pe, dev, "q_pe", dt, {B, q_len, H, kRope});
    if (cache.dim() != 3) bad_value("kv_cache must be [num_blocks, block_size, 324]");
    dense(cache, dev, "kv_cache", at::kByte, {cache.size(0), cache.size(1), kE2m1});
    if (table.dim() != 2) bad_value("block_table must be [B, max_blocks]");
    dense(table, dev, "block_table", at::kInt, {B, table.size(1)});
    dense(lens, dev, "seq_lens", at::kInt, {B});
    if (cur) dense(*cur, dev, "kv_cur", dt, {B, q_len, kQk});
    int32_t* err_word = error_word(err, dev);
    const int64_t P = shards + (cur ? 1 : 0);
    const int64_t hs = slices > 0 ? H / slices : H;
    const std::vector<int64_t> rows = slices == 1 ? std::vector<int64_t>{B, q_len, P, H}
                                                  : std::vector<int64_t>{std::max<int64_t>(slices, 0), B * q_len, P, hs};
    std::vector<int64_t> wide = rows;
    wide.push_back(kLatent);
    at::ScalarType pt = dt;
    if (a[8] != Py_None) {
      if (!THPDtype_Check(a[8])) bad_type("part_dtype must be a torch dtype");
      pt = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
    } else if (a[9] != Py_None) {
      pt = tensor(a[9], "o_part").scalar_type();
    }
    const int in_code = dtype_code(dt), part_code = dtype_code(pt);
    if (P < 0) bad_value("num_shards is negative");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const Stream stream = stream_of(a[15], dev);
    const at::Tensor o = a[9] == Py_None ? output(stream, wide, pt, q_abs) : tensor(a[9], "o_part");
    const at::Tensor lse = a[10] == Py_None ? output(stream, rows, at::kFloat, q_abs) : tensor(a[10], "lse_part");
    on(o, dev, "o_part", pt);
    on(lse, dev, "lse_part", at::kFloat);
    if (o.sizes() != c10::IntArrayRef(wide) || !o.is_contiguous() || lse.sizes() != c10::IntArrayRef(rows) || !lse.is_contiguous())
      bad_value("o_part and lse_part must be contiguous, of shapes " + words(wide) + " and " + words(rows));
    at::Tensor ws;
    if (PyUnicode_Check(a[12])) {
      if (PyUnicode_CompareWithASCIIString(a[12], "default") != 0) bad_value("workspace must be 'default', a tensor or None");
      ws = default_workspace(q_abs, dev, stream, fits(B, "B"), fits(q_len, "q_len"), static_cast<int>(shards), cur ? 1 : 0);
    } else if (a[12] != Py_None) {
      ws = tensor(a[12], "workspace");
      on(ws, dev, "workspace");
      if (!ws.is_contiguous()) bad_value("workspace must be contiguous");
    }
    const int st = mla_dcp_decode_partial_fp4(
        q_abs.data_ptr(), q_pe.data_ptr(), cache.data_ptr(), static_cast<const int32_t*>(table.data_ptr()),
        static_cast<const int32_t*>(lens.data_ptr()), ptr(cur), fits(B, "B"), fits(q_len, "q_len"), fits(H, "H"),
        fits(cache.size(0), "num_blocks"), fits(cache.size(1), "block_size"), fits(table.size(1), "max_blocks"),
        static_cast<int>(shards), number(a[7]), number(a[14]), in_code, part_code, o.data_ptr(),
        static_cast<float*>(lse.data_ptr()), err_word, ws.defined() ? ws.data_ptr() : nullptr,
        ws.defined() ? static_cast<uint64_t>(ws.numel()) * ws.element_size() : 0, static_cast<int>(slices), stream.raw());
    return result(st, {o, lse});
  });
}

// ---------------------------------------------------------------- pages
struct Pools {
  int layers, pages, bs;
  uint64_t stride, page_bytes;   // between layers, of a page
};

// A pool [num_blocks, bs, W] or the layers' pools [layers, num_blocks, bs, W].
Pools pools(const at::Tensor& t, const char* name) {
  const std::string s(name);
  const int64_t d = t.dim();
  if (d != 3 && d != 4) bad_value(s + " must be a tensor [(layers,) num_blocks, block_size, W]");
  const int64_t n = t.size(d - 3), bs = t.size(d - 2), w = t.size(d - 1), size = t.element_size();
  if (t.stride(d - 1) != 1 || t.stride(d - 2) != w || t.stride(d - 3) != bs * w)
    bad_value("the pages of " + s + " must be contiguous");
  const int64_t layers = d == 4 ? t.size(0) : 1, stride = layers > 1 ? t.stride(0) * size : 0;
  if (layers > 1 && stride < n * bs * w * size) bad_value("the layers of " + s + " overlap");
  return {fits(layers, "layers"), fits(n, "num_blocks"), fits(bs, "block_size"), static_cast<uint64_t>(stride),
          static_cast<uint64_t>(bs * w * size)};
}

const int32_t* ids(const at::Tensor& t, int dev, const char* name, int64_t n) {
  dense(t, dev, name, at::kInt, {n});
  return static_cast<const int32_t*>(t.data_ptr());
}

// src, dst, src_ids, dst_ids, err_flag, stream
PyObject* kv_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor &src = tensor(a[0], "src"), &dst = tensor(a[1], "dst"), &si = tensor(a[2], "src_ids");
    const at::Tensor& di = tensor(a[3], "dst_ids");
    const int dev = device_of(src, "src");
    on(dst, dev, "dst");
    const Pools s = pools(src, "src"), d = pools(dst, "dst");
    if (s.layers != d.layers || s.page_bytes != d.page_bytes || src.scalar_type() != dst.scalar_type())
      bad_value("src and dst must hold pages of one size and type in as many layers");
    const int64_t count = si.numel();
    const int32_t *from = ids(si, dev, "src_ids", count), *to = ids(di, dev, "dst_ids", count);
    int32_t* err_word = error_word(maybe(a[4], "err_flag"), dev);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const Stream stream = stream_of(a[5], dev);
    const int st = count == 0 ? MLA_OK
                              : mla_kv_copy_pages(src.data_ptr(), s.stride, s.pages, dst.data_ptr(), d.stride, d.pages,
                                                  s.page_bytes, s.layers, from, to, fits(count, "n"), err_word, stream.raw());
    return result(st, {});
  });
}

struct PageState {
  int dev, rows, max_blocks, pages;
  int32_t *table, *lens, *refs;
};

PageState page_state(PyObject* t, PyObject* l, PyObject* r) {
  const at::Tensor &table = tensor(t, "block_table"), &lens = tensor(l, "seq_lens"), &refs = tensor(r, "ref_counts");
  const int dev = device_of(table, "block_table");
  if (table.dim() != 2) bad_value("block_table must be [rows, max_blocks]");
  dense(table, dev, "block_table", at::kInt, {table.size(0), table.size(1)});
  dense(lens, dev, "seq_lens", at::kInt, {table.size(0)});
  dense(refs, dev, "ref_counts", at::kInt, {refs.numel()});
  return {dev, fits(table.size(0), "rows"), fits(table.size(1), "max_blocks"), fits(refs.numel(), "num_blocks"),
          static_cast<int32_t*>(table.data_ptr()), static_cast<int32_t*>(lens.data_ptr()), static_cast<int32_t*>(refs.data_ptr())};
}

// block_table, seq_lens, ref_counts, rows, block_size, err_flag, stream
PyObject* kv_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const PageState p = page_state(a[0], a[1], a[2]);
    const at::Tensor& rows = tensor(a[3], "rows");
    const int64_t count = rows.numel();
    const int32_t* which = ids(rows, p.dev, "rows", count);
    int32_t* err_word = error_word(maybe(a[5], "err_flag"), p.dev);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(p.dev));
    const Stream stream = stream_of(a[6], p.dev);
    const int st = count == 0 ? MLA_OK
                              : mla_kv_free(p.table, p.lens, p.refs, which, fits(count, "n"), p.rows, p.pages,
                                            small(a[4], "block_size"), p.max_blocks, err_word, stream.raw());
    return result(st, {});
  });
}

// kv_cache, block_table, seq_lens, ref_counts, parents, children, workspace, err_flag, stream
PyObject* kv_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& cache = tensor(a[0], "kv_cache");
    const PageState p = page_state(a[1], a[2], a[3]);
    on(cache, p.dev, "kv_cache");
    const Pools c = pools(cache, "kv_cache");
    if (c.pages != p.pages)
      bad_value("ref_counts of " + std::to_string(p.pages) + " pages for a pool of " + std::to_string(c.pages));
    const at::Tensor &parents = tensor(a[4], "parents"), &children = tensor(a[5], "children");
    const int64_t count = parents.numel();
    const int32_t *from = ids(parents, p.dev, "parents", count), *to = ids(children, p.dev, "children", count);
    int32_t* err_word = error_word(maybe(a[7], "err_flag"), p.dev);
    if (count == 0) return result(MLA_OK, {});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(p.dev));
    const Stream stream = stream_of(a[8], p.dev);
    at::Tensor ws;
    if (a[6] == Py_None) {
      ws = make_on(stream, {std::max<int64_t>(16, static_cast<int64_t>(mla_kv_fork_workspace_size(fits(count, "n"))))},
                   at::kByte, cache);
    } else {
      ws = tensor(a[6], "workspace");
      on(ws, p.dev, "workspace");
      if (!ws.is_contiguous()) bad_value("workspace must be contiguous");
    }
    const int st = mla_kv_fork(cache.data_ptr(), c.stride, c.page_bytes, c.layers, p.table, p.lens, p.refs, from, to,
                               fits(count, "n"), p.rows, p.pages, c.bs, p.max_blocks, ws.data_ptr(),
                               static_cast<uint64_t>(ws.numel()) * ws.element_size(), err_word, stream.raw());
    return result(st, {});
  });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(kv_append), METHOD(partial_fp4), METHOD(kv_copy_pages), METHOD(kv_free), METHOD(kv_fork),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module_def); }
