// Argument marshalling of the per-token calls of a decoder layer (norm, append
// to the 4-bit cache, attention over it): reads the tensors' types, sizes, strides and
// addresses, checks them, and calls the C ABI.  The same steps in Python take
// about 10 us a call on the host of a GB300, several times the small calls'
// GPU time; here they take about 1 us.  No computation and no fallback: what does
// not fit raises ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "gathered_rank_gemm.h"

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const char* name, const char* what) {
  throw Refused(std::string(name) + " " + what);
}

const at::Tensor* optional(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(name, "must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& required(PyObject* o, const char* name) {
  const at::Tensor* t = optional(o, name);
  if (!t) refuse(name, "must be a tensor");
  return *t;
}
double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, "must be a number");
  }
  return v;
}
int64_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, "must be a whole number");
  }
  return v;
}

// The call's 16-bit type and device, taken from its main operand (of a call without 16-bit
// data, the cache).
struct Like {
  at::ScalarType type;
  c10::Device device;
  bool f16;
  Like(const at::Tensor& t, const char* name) : type(t.scalar_type()), device(t.device()) {
    if (!t.is_cuda()) refuse(name, "must be a CUDA tensor (there is no CPU path)");
    if (type != at::kBFloat16 && type != at::kHalf) refuse(name, "must be bfloat16 or float16");
    f16 = type == at::kHalf;
  }
  explicit Like(const at::Tensor& cache) : type(at::kByte), device(cache.device()), f16(false) {
    if (!cache.is_cuda()) refuse("cache", "must be a CUDA tensor (there is no CPU path)");
  }
};

void on(const at::Tensor& t, const char* name, const Like& like) {
  if (t.device() != like.device) refuse(name, "must be on the device of the other operands");
}
// A contiguous operand of one type and shape; its address.
template <typename T>
T* vec(const at::Tensor& t, const char* name, const Like& like, at::ScalarType type,
       at::IntArrayRef shape) {
  if (t.scalar_type() != type) refuse(name, "has the wrong type");
  if (t.sizes() != shape) refuse(name, "has the wrong shape");
  if (!t.is_contiguous()) refuse(name, "must be contiguous");
  on(t, name, like);
  return static_cast<T*>(t.data_ptr());
}
// An operand [rows][...] that is contiguous behind its row stride.
template <typename T>
T* rows(const at::Tensor& t, const char* name, const Like& like, at::ScalarType type,
        at::IntArrayRef shape, int64_t& stride) {
  if (t.scalar_type() != type) refuse(name, "has the wrong type");
  if (t.sizes() != shape) refuse(name, "has the wrong shape");
  const size_t d = shape.size();
  if (t.stride(d - 1) != 1 || (d == 3 && t.stride(1) != shape[2] && shape[1] != 1))
    refuse(name, "must be contiguous behind its row stride");
  on(t, name, like);
  stride = t.stride(0);
  // one row needs no stride; a view may report any
  if (shape[0] == 1) stride = d == 3 ? shape[1] * shape[2] : shape[1];
  return static_cast<T*>(t.data_ptr());
}
uint32_t* status_word(PyObject* o, const Like& like) {
  const at::Tensor* t = optional(o, "status");
  if (!t) return nullptr;
  on(*t, "status", like);
  if (t->numel() * t->element_size() < 4) refuse("status", "must hold an int32");
  return static_cast<uint32_t*>(t->data_ptr());
}
struct Cache {
  uint8_t* ptr;
  int64_t pages, heads, page_size, dim;
  Cache(const at::Tensor& t, const Like& like) {
    if (t.scalar_type() != at::kByte || t.dim() != 4 || !t.is_contiguous() || t.size(3) % 18)
      refuse("cache", "must be a contiguous uint8 tensor [pages][kv heads][page_size / 16][18 * head_dim]");
    on(t, "cache", like);
    ptr = static_cast<uint8_t*>(t.data_ptr());
    pages = t.size(0), heads = t.size(1), page_size = 16 * t.size(2), dim = t.size(3) / 18;
    if (heads > INT32_MAX || page_size > INT32_MAX || dim > INT32_MAX)
      refuse("cache", "has a size out of range");
  }
};
// The sequences' rows, keys and pages.
struct Sequences {
  int32_t *start, *kv, *table;
  int64_t count, wide;
  Sequences(PyObject* q_start, PyObject* kv_len, PyObject* page_table, const Like& like) {
    const at::Tensor& t = required(page_table, "page_table");
    if (t.dim() != 2) refuse("page_table", "must be [sequences][pages]");
    count = t.size(0), wide = t.size(1);
    start = vec<int32_t>(required(q_start, "q_start"), "q_start", like, at::kInt, {count + 1});
    kv = vec<int32_t>(required(kv_len, "kv_len"), "kv_len", like, at::kInt, {count});
    table = vec<int32_t>(t, "page_table", like, at::kInt, {count, wide});
  }
};
bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(name, "must be true or false");
  }
  return v != 0;
}
// The stream's handle: of the device's current one, of a torch stream, or the number itself.
void* stream_of(PyObject* o, c10::Device device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device.index()).stream();
  PyObject* p = PyObject_GetAttrString(o, "cuda_stream");
  if (!p) PyErr_Clear();
  void* s = PyLong_AsVoidPtr(p ? p : o);
  Py_XDECREF(p);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse("stream", "must be a CUDA stream, its handle as a whole number, or None");
  }
  return s;
}

using Args = PyObject* const*;
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& body) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(body());  // (body leaves no Python error behind: it refuses)
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* add_rmsnorm(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const at::Tensor& x = required(a[0], "x");
    const Like like(x, "x");
    if (x.dim() != 2) refuse("x", "must be [rows][hidden]");
    const at::IntArrayRef shape = x.sizes();
    const int64_t count = shape[0], hidden = shape[1];
    int64_t xs, rs = 0, os = 0, ys = 0, es = 0, group = hidden;
    auto* xp = rows<uint16_t>(x, "x", like, like.type, shape, xs);
    auto* wp = vec<uint16_t>(required(a[1], "weight"), "weight", like, like.type, {hidden});
    const float eps = static_cast<float>(number(a[2], "eps"));
    auto* np = vec<int32_t>(required(a[3], "num_tokens"), "num_tokens", like, at::kInt, {1});
    const at::Tensor *r = optional(a[4], "residual"), *o = optional(a[5], "residual_out"),
                     *y = optional(a[6], "y"), *y8 = optional(a[7], "y8"),
                     *sc = optional(a[8], "y8_scale");
    uint16_t* rp = r ? rows<uint16_t>(*r, "residual", like, like.type, shape, rs) : nullptr;
    uint16_t* op = o ? rows<uint16_t>(*o, "residual_out", like, like.type, shape, os) : nullptr;
    uint16_t* yp = y ? rows<uint16_t>(*y, "y", like, like.type, shape, ys) : nullptr;
    uint8_t* ep = nullptr;
    float* sp = nullptr;
    if (y8) {
      if (!sc || sc->dim() != 2) refuse("y8", "must come with y8_scale, [rows][1] or [rows][hidden / 128]");
      ep = rows<uint8_t>(*y8, "y8", like, at::kFloat8_e4m3fn, shape, es);
      const int64_t groups = sc->size(1);
      if (groups != 1) group = 128;
      sp = vec<float>(*sc, "y8_scale", like, at::kFloat, {count, groups == 1 ? 1 : hidden / 128});
    }
    uint32_t* st = status_word(a[9], like);
    const c10::cuda::CUDAGuard guard(like.device);
    return (like.f16 ? lora_add_rmsnorm_f16 : lora_add_rmsnorm)(
        xp, xs, rp, rs, wp, eps, hidden, op, os, yp, ys, ep, es, sp, group, np, count, st,
        stream_of(a[10], like.device));
  });
}

PyObject* kv4_append(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    const at::Tensor& k = required(a[1], "k");
    const Like like(k, "k");
    const Cache c(required(a[0], "cache"), like);
    const at::Tensor& slots = required(a[3], "slots");
    if (slots.dim() != 1) refuse("slots", "must be [rows]");
    const int64_t count = slots.size(0);
    const int64_t shape[3] = {count, c.heads, c.dim};
    int64_t ks, vs, qs = 0, os = 0, qh = 0;
    auto* kp = rows<uint16_t>(k, "k", like, like.type, shape, ks);
    auto* vp = rows<uint16_t>(required(a[2], "v"), "v", like, like.type, shape, vs);
    auto* sp = vec<int32_t>(slots, "slots", like, at::kInt, {count});
    auto* np = vec<int32_t>(required(a[4], "num_tokens"), "num_tokens", like, at::kInt, {1});
    const at::Tensor *q = optional(a[5], "q"), *qo = optional(a[6], "q_out"),
                     *pos = optional(a[7], "positions"), *rope = optional(a[8], "rope"),
                     *kh = optional(a[12], "k_held"), *vh = optional(a[13], "v_held");
    uint16_t *qp = nullptr, *op = nullptr;
    if (q) {
      if (!qo || q->dim() != 3) refuse("q", "must be [rows][heads][head_dim] and come with q_out");
      qh = q->size(1);
      const int64_t qshape[3] = {count, qh, c.dim};
      qp = rows<uint16_t>(*q, "q", like, like.type, qshape, qs);
      op = rows<uint16_t>(*qo, "q_out", like, like.type, qshape, os);
    }
    float* rp = nullptr;
    int32_t* pp = nullptr;
    int64_t positions = 0, rope_dim = 0;
    if (rope) {
      if (!pos || rope->dim() != 2) refuse("rope", "must be [positions][rope_dim] and come with positions");
      positions = rope->size(0), rope_dim = rope->size(1);
      rp = vec<float>(*rope, "rope", like, at::kFloat, {positions, rope_dim});
      pp = vec<int32_t>(*pos, "positions", like, at::kInt, {count});
    }
    const int interleaved = truth(a[9], "interleaved") ? 1 : 0;
    const float k_scale = static_cast<float>(number(a[10], "k_scale"));
    const float v_scale = static_cast<float>(number(a[11], "v_scale"));
    uint16_t* khp = kh ? vec<uint16_t>(*kh, "k_held", like, like.type, shape) : nullptr;
    uint16_t* vhp = vh ? vec<uint16_t>(*vh, "v_held", like, like.type, shape) : nullptr;
    uint32_t* st = status_word(a[14], like);
    const c10::cuda::CUDAGuard guard(like.device);
    return (like.f16 ? lora_kv4_append_f16 : lora_kv4_append)(
        qp, qs, op, os, static_cast<int>(std::min<int64_t>(qh, INT32_MAX)), kp, ks, vp, vs, rp,
        positions, static_cast<int>(std::min<int64_t>(rope_dim, INT32_MAX)), interleaved, pp, sp, c.ptr,
        c.pages, static_cast<int>(c.heads), static_cast<int>(c.page_size), static_cast<int>(c.dim),
        k_scale, v_scale, khp, vhp, np, count, st, stream_of(a[15], like.device));
  });
}

// The attention of causal rows (15 arguments), and that of trees (16: a mask behind max_q_len).
PyObject* attention(Args a, Py_ssize_t n, bool tree) {
  return guarded(n, tree ? 16 : 15, [&] {
    const at::Tensor& q = required(a[1], "q");
    const Like like(q, "q");
    if (q.dim() != 3) refuse("q", "must be [rows][heads][head_dim]");
    const Cache c(required(a[0], "cache"), like);
    const int64_t count = q.size(0), qh = q.size(1);
    const int64_t shape[3] = {count, qh, c.dim};
    int64_t qs, os;
    auto* qp = rows<uint16_t>(q, "q", like, like.type, shape, qs);
    auto* op = rows<uint16_t>(required(a[2], "out"), "out", like, like.type, shape, os);
    const Sequences s(a[3], a[4], a[5], like);
    const int64_t max_q = whole(a[6], "max_q_len");
    int64_t words = 0;
    uint32_t* mask = nullptr;
    if (tree) {
      const at::Tensor& t = required(a[7], "tree_mask");
      if (t.dim() != 2) refuse("tree_mask", "must be [rows][words]");
      words = t.size(1);
      mask = vec<uint32_t>(t, "tree_mask", like, at::kInt, {count, words});
      ++a;
    }
    const float scale = static_cast<float>(number(a[7], "softmax_scale"));
    const at::Tensor& ws = required(a[8], "workspace");
    on(ws, "workspace", like);
    if (!ws.is_contiguous()) refuse("workspace", "must be contiguous");
    const int64_t window = whole(a[9], "window");
    const float k_scale = static_cast<float>(number(a[10], "k_scale"));
    const float v_scale = static_cast<float>(number(a[11], "v_scale"));
    const at::Tensor* lse = optional(a[12], "lse");
    float* lp = lse ? vec<float>(*lse, "lse", like, at::kFloat, {count, qh}) : nullptr;
    uint32_t* st = status_word(a[13], like);
    const c10::cuda::CUDAGuard guard(like.device);
    const int heads = static_cast<int>(std::min<int64_t>(qh, INT32_MAX));
    const int kvh = static_cast<int>(c.heads), page = static_cast<int>(c.page_size), dim = static_cast<int>(c.dim);
    const size_t bytes = static_cast<size_t>(ws.numel() * ws.element_size());
    void* stream = stream_of(a[14], like.device);
    if (tree)
      return (like.f16 ? lora_kv4_tree_attention_f16 : lora_kv4_tree_attention)(
          qp, qs, op, os, lp, heads, c.ptr, c.pages, kvh, page, dim, k_scale, v_scale, s.start, s.kv,
          s.table, s.wide, s.count, count, max_q, mask, words, scale, window, ws.data_ptr(), bytes, st,
          stream);
    return (like.f16 ? lora_kv4_attention_f16 : lora_kv4_attention)(
        qp, qs, op, os, lp, heads, c.ptr, c.pages, kvh, page, dim, k_scale, v_scale, s.start, s.kv,
        s.table, s.wide, s.count, count, max_q, scale, window, ws.data_ptr(), bytes, st, stream);
  });
}
PyObject* kv4_attention(PyObject*, Args a, Py_ssize_t n) { return attention(a, n, false); }
PyObject* kv4_tree_attention(PyObject*, Args a, Py_ssize_t n) { return attention(a, n, true); }

// Accepted paths of the sequences' trees.
struct Paths {
  int32_t *path, *len;
  int64_t longest;
  Paths(const at::Tensor& t, const at::Tensor& l, int64_t seqs, const Like& like) {
    if (t.dim() != 2) refuse("path", "must be [sequences][longest path]");
    longest = t.size(1);
    path = vec<int32_t>(t, "path", like, at::kInt, {seqs, longest});
    len = vec<int32_t>(l, "path_len", like, at::kInt, {seqs});
  }
};

PyObject* kv4_accept(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const at::Tensor& cache = required(a[0], "cache");
    const Like like(cache);
    const Cache c(cache, like);
    const Sequences s(a[1], a[2], a[3], like);
    const Paths p(required(a[4], "path"), required(a[5], "path_len"), s.count, like);
    auto* out = vec<int32_t>(required(a[6], "kv_len_out"), "kv_len_out", like, at::kInt, {s.count});
    uint32_t* st = status_word(a[7], like);
    const c10::cuda::CUDAGuard guard(like.device);
    return lora_kv4_accept(c.ptr, c.pages, static_cast<int>(c.heads), static_cast<int>(c.page_size),
                           static_cast<int>(c.dim), s.start, s.kv, s.table, s.wide, s.count, p.path,
                           p.len, p.longest, out, st, stream_of(a[8], like.device));
  });
}

PyObject* kv4_key_weights(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const at::Tensor& q = required(a[2], "q");
    const Like like(q, "q");
    if (q.dim() != 3) refuse("q", "must be [rows][heads][head_dim]");
    const Cache c(required(a[1], "cache"), like);
    const int64_t count = q.size(0), qh = q.size(1);
    int64_t qs;
    auto* qp = rows<uint16_t>(q, "q", like, like.type, {count, qh, c.dim}, qs);
    auto* lp = vec<float>(required(a[3], "lse"), "lse", like, at::kFloat, {count, qh});
    const Sequences s(a[4], a[5], a[6], like);
    const at::Tensor& w = required(a[0], "weights");
    if (w.dim() != 3) refuse("weights", "must be [sequences][kv heads][capacity]");
    const int64_t capacity = w.size(2);
    auto* wp = vec<float>(w, "weights", like, at::kFloat, {s.count, c.heads, capacity});
    const int64_t max_q = whole(a[7], "max_q_len");
    const float scale = static_cast<float>(number(a[8], "softmax_scale"));
    const int64_t window = whole(a[9], "window");
    const float k_scale = static_cast<float>(number(a[10], "k_scale"));
    const at::Tensor *path = optional(a[11], "path"), *len = optional(a[12], "path_len");
    if (!path != !len) refuse("path", "must come with path_len");
    int32_t *pp = nullptr, *np = nullptr;
    int64_t longest = 0;
    if (path) {
      const Paths p(*path, *len, s.count, like);
      pp = p.path, np = p.len, longest = p.longest;
    }
    uint32_t* st = status_word(a[13], like);
    const c10::cuda::CUDAGuard guard(like.device);
    return (like.f16 ? lora_kv4_key_weights_f16 : lora_kv4_key_weights)(
        wp, capacity, qp, qs, lp, static_cast<int>(std::min<int64_t>(qh, INT32_MAX)), c.ptr, c.pages,
        static_cast<int>(c.heads), static_cast<int>(c.page_size), static_cast<int>(c.dim), k_scale,
        s.start, s.kv, s.table, s.wide, s.count, count, max_q, scale, window, pp, np, longest, st,
        stream_of(a[14], like.device));
  });
}

PyObject* kv4_evict(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const at::Tensor& cache = required(a[0], "cache");
    const Like like(cache);
    const Cache c(cache, like);
    const at::Tensor& table = required(a[5], "page_table");
    if (table.dim() != 2) refuse("page_table", "must be [sequences][pages]");
    const int64_t seqs = table.size(0), wide = table.size(1);
    auto* tp = vec<int32_t>(table, "page_table", like, at::kInt, {seqs, wide});
    const at::Tensor& w = required(a[1], "weights");
    if (w.dim() != 3) refuse("weights", "must be [sequences][kv heads][capacity]");
    const int64_t capacity = w.size(2);
    auto* wp = vec<float>(w, "weights", like, at::kFloat, {seqs, c.heads, capacity});
    auto* pp = vec<int32_t>(required(a[2], "key_pos"), "key_pos", like, at::kInt, {seqs, c.heads, capacity});
    auto* kp = vec<int32_t>(required(a[3], "kv_len"), "kv_len", like, at::kInt, {seqs});
    auto* lp = vec<int32_t>(required(a[4], "last_pos"), "last_pos", like, at::kInt, {seqs});
    const int64_t budget = whole(a[6], "budget");
    auto* out = vec<int32_t>(required(a[7], "kv_len_out"), "kv_len_out", like, at::kInt, {seqs});
    const int64_t sink = whole(a[8], "sink"), recent = whole(a[9], "recent");
    uint32_t* st = status_word(a[10], like);
    const c10::cuda::CUDAGuard guard(like.device);
    return lora_kv4_evict(c.ptr, c.pages, static_cast<int>(c.heads), static_cast<int>(c.page_size),
                          static_cast<int>(c.dim), wp, pp, capacity, kp, lp, tp, wide, seqs, budget,
                          sink, recent, out, st, stream_of(a[11], like.device));
  });
}

PyMethodDef kMethods[] = {
    {"add_rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(add_rmsnorm)),
     METH_FASTCALL, nullptr},
    {"kv4_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv4_append)),
     METH_FASTCALL, nullptr},
    {"kv4_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv4_attention)),
     METH_FASTCALL, nullptr},
    {"kv4_tree_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv4_tree_attention)),
     METH_FASTCALL, nullptr},
    {"kv4_accept", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv4_accept)),
     METH_FASTCALL, nullptr},
    {"kv4_key_weights", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv4_key_weights)),
     METH_FASTCALL, nullptr},
    {"kv4_evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv4_evict)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__native(void) {
  return PyModule_Create(&kModule);
}
