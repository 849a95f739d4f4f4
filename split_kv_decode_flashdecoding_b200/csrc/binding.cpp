// Argument marshalling of the serving calls (prompt and tree attention, page operators) for the Python
// package: a CPython module over the C ABI of include/fd.h. These calls are made once a scheduling
// step and layer, and on short batches the host is what they wait for: through ctypes an append took
// 10.7 us of host time and a prompt or tree call 16 to 18, here 3.5 to 5.1 and 6 to 9 (the kernels: 3.7 and
// 10 to 13).
#include <Python.h>

#include <ATen/Functions.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <limits>
#include <optional>
#include <utility>

#include "fd.h"

namespace {

PyObject* g_raise = nullptr;  // (status, name): raises the package's error

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

fd_tensor desc(const at::Tensor& t) {
  TORCH_CHECK_VALUE(t.dim() <= 4, "at most 4 dimensions");
  fd_tensor d{};
  d.data = t.data_ptr();
  const auto type = t.scalar_type();
  // an E4M3 cache may be passed as torch.float8_e4m3fn or as its uint8 codes
  d.dtype = type == at::kFloat ? FD_F32
            : type == at::kBFloat16 ? FD_BF16
            : type == at::kFloat8_e4m3fn || type == at::kByte ? FD_E4M3 : -1;
  d.ndim = static_cast<int32_t>(t.dim());
  for (int64_t i = 0; i < t.dim(); ++i) {
    d.shape[i] = t.size(i);
    d.stride[i] = t.stride(i);
  }
  return d;
}

// Address of a contiguous int32 tensor of this shape on the device.
int32_t* int32s(PyObject* o, const char* name, c10::Device dev, at::IntArrayRef shape) {
  const at::Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.sizes() == shape && t.device() == dev && t.is_contiguous(),
                    name, " must be a contiguous int32 tensor ", shape, " on ", dev);
  for (const int64_t n : shape) TORCH_CHECK_VALUE(n <= std::numeric_limits<int32_t>::max(), name, " has 2^31 or more entries");
  return static_cast<int32_t*>(t.data_ptr());
}

using Named = std::pair<const char*, const at::Tensor*>;
void need(const at::Tensor& like, std::initializer_list<Named> others) {
  TORCH_CHECK_VALUE(like.is_cuda(), "CUDA tensors are needed, not ", c10::DeviceTypeName(like.device().type(), true));
  for (const Named& n : others)
    TORCH_CHECK_VALUE(n.second->device() == like.device(), n.first, " is on ", n.second->device(), ", not on ", like.device());
}

int32_t to_int32(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  TORCH_CHECK_VALUE(x >= std::numeric_limits<int32_t>::min() && x <= std::numeric_limits<int32_t>::max(), name, " is out of range");
  return static_cast<int32_t>(x);
}

float to_float(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(x);
}

int64_t attribute(PyObject* o, const char* name) {
  PyObject* x = PyObject_GetAttrString(o, name);
  if (!x) throw python_error();
  const long long v = PyLong_AsLongLong(x);
  Py_DECREF(x);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// The stream of a call: the device's current one (None), a torch stream, or a raw handle (an integer, or
// another library's object with one). `side` is a torch stream other than the current one: the
// allocator, which takes the memory of a dropped tensor back for the stream that it came from, has to
// know that the call's tensors are used there too. A raw handle says nothing about how long its stream
// lives; its caller keeps the tensors until the work is done, as in C.
struct Lane {
  void* handle = nullptr;
  std::optional<c10::cuda::CUDAStream> side;
  Lane(PyObject* o, c10::Device dev) {
    const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(dev.index());
    if (o == Py_None) {
      handle = now.stream();
    } else if (PyObject_HasAttrString(o, "stream_id")) {
      const int64_t type = attribute(o, "device_type"), index = attribute(o, "device_index");
      TORCH_CHECK_VALUE(type == static_cast<int64_t>(c10::DeviceType::CUDA) && index == dev.index(), "the stream is not one of ", dev);
      const auto s = c10::cuda::CUDAStream::unpack3(attribute(o, "stream_id"), dev.index(), c10::DeviceType::CUDA);
      handle = s.stream();
      if (handle != now.stream()) side = s;
    } else {
      PyObject* x = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Index(o);
      if (!x) throw python_error();
      handle = PyLong_AsVoidPtr(x);
      Py_DECREF(x);
      if (!handle && PyErr_Occurred()) throw python_error();
    }
  }
};

void record(const at::Tensor& t, c10::cuda::CUDAStream s) { c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), s); }

// call(stream) on the tensor's device, without the interpreter lock. args: the call's n arguments.
template <typename Call>
void run(const char* name, const at::Tensor& like, const Lane& lane, PyObject* const* args, Py_ssize_t n, Call call) {
  if (lane.side)
    for (Py_ssize_t i = 0; i < n; ++i)
      if (THPVariable_Check(args[i])) record(THPVariable_Unpack(args[i]), *lane.side);
  fd_status st;
  {
    const c10::cuda::CUDAGuard guard(like.device());
    Py_BEGIN_ALLOW_THREADS
    st = call(lane.handle);
    Py_END_ALLOW_THREADS
  }
  if (st == FD_OK) return;
  PyObject* r = PyObject_CallFunction(g_raise, "is", static_cast<int>(st), name);
  Py_XDECREF(r);
  if (!r) throw python_error();
  TORCH_CHECK(false, name, " failed with status ", static_cast<int>(st));
}

void count(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// out [T, Hq, D] and lse [T, Hq] of an attention call: the caller's, or new ones. New ones are the
// stream's: memory that the current stream has still to write would be free to it otherwise.
struct RowsOut {
  at::Tensor out, lse;
  RowsOut(const at::Tensor& q, PyObject* o, PyObject* l, const Lane& lane) {
    const at::IntArrayRef rows = q.sizes().slice(0, 2);
    const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(q.device().index());
    const c10::cuda::CUDAStreamGuard guard(lane.side ? *lane.side : now);
    if (o != Py_None) {
      out = tensor(o, "out");
    } else {
      out = at::empty(q.sizes(), q.options());
      if (lane.side) record(out, now);
    }
    if (l != Py_None) {
      lse = tensor(l, "lse");
      TORCH_CHECK_VALUE(lse.scalar_type() == at::kFloat && lse.is_contiguous() && lse.sizes() == rows,
                        "lse must be a contiguous float32 tensor [T, Hq]");
    } else {
      lse = at::empty(rows, q.options().dtype(at::kFloat));
      if (lane.side) record(lse, now);
    }
    need(q, {{"out", &out}, {"lse", &lse}});
  }
  PyObject* give() const {
    PyObject* a = THPVariable_Wrap(out);
    PyObject* b = a ? THPVariable_Wrap(lse) : nullptr;
    if (!b) {
      Py_XDECREF(a);
      throw python_error();
    }
    PyObject* pair = PyTuple_Pack(2, a, b);
    Py_DECREF(a);
    Py_DECREF(b);
    return pair;
  }
};

// A block table [B, pages_per_seq].
struct Table {
  int32_t *data, batch, per;
  Table(PyObject* o, c10::Device dev) {
    const at::Tensor& t = tensor(o, "block_table");
    TORCH_CHECK_VALUE(t.dim() == 2, "block_table must be [B, pages_per_seq]");
    data = int32s(o, "block_table", dev, t.sizes());
    batch = static_cast<int32_t>(t.size(0));
    per = static_cast<int32_t>(t.size(1));
  }
};

int64_t numel(PyObject* o, const char* name) { return tensor(o, name).numel(); }
int64_t last(const at::Tensor& t) { return t.dim() > 0 ? t.size(-1) : 0; }

// (q, k, v, seq_lens, out, lse, stream)
PyObject* prompt_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const int64_t batch = numel(a[3], "seq_lens");
  const int32_t* lens = int32s(a[3], "seq_lens", q.device(), {batch});
  TORCH_CHECK_VALUE(q.dim() == 3, "q must be [T, Hq, D]");
  need(q, {{"k", &k}, {"v", &v}});
  const Lane lane(a[6], q.device());
  const RowsOut o(q, a[4], a[5], lane);
  const fd_tensor dq = desc(q), dk = desc(k), dv = desc(v);
  fd_tensor d = desc(o.out);
  float* lse = static_cast<float*>(o.lse.data_ptr());
  run("fd_prompt_attention", q, lane, a, n,
      [&](void* s) { return fd_prompt_attention(&dq, &dk, &dv, lens, static_cast<int32_t>(batch), &d, lse, s); });
  return o.give();
  END_HANDLE_TH_ERRORS
}

// (q, k, v, block_table or None, prefix_lens, tree_lens, tree_mask, out, lse, stream)
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const bool paged = a[3] != Py_None;
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], paged ? "k_pages" : "k_cache"),
                   &v = tensor(a[2], paged ? "v_pages" : "v_cache"), &m = tensor(a[6], "tree_mask");
  const c10::Device dev = q.device();
  TORCH_CHECK_VALUE(q.dim() == 3 && k.dim() > 0, "q must be [T, Hq, D], k a cache or a page pool");
  int32_t *table = nullptr, per = 0;
  int64_t batch = k.size(0);
  if (paged) {
    const Table t(a[3], dev);
    table = t.data;
    per = t.per;
    batch = t.batch;
  }
  const int32_t *prefix = int32s(a[4], "prefix_lens", dev, {batch}), *lens = int32s(a[5], "tree_lens", dev, {batch});
  const int64_t words = last(m);
  const int32_t* mask = int32s(a[6], "tree_mask", dev, {q.size(0), words});
  need(q, {{paged ? "k_pages" : "k_cache", &k}, {paged ? "v_pages" : "v_cache", &v}});
  const Lane lane(a[9], dev);
  const RowsOut o(q, a[7], a[8], lane);
  const fd_tensor dq = desc(q), dk = desc(k), dv = desc(v);
  fd_tensor d = desc(o.out);
  float* lse = static_cast<float*>(o.lse.data_ptr());
  const int32_t w = static_cast<int32_t>(words), b = static_cast<int32_t>(batch);
  run(paged ? "fd_tree_attention_paged" : "fd_tree_attention", q, lane, a, n, [&](void* s) {
    return paged ? fd_tree_attention_paged(&dq, &dk, &dv, table, per, b, prefix, lens, mask, w, &d, lse, s)
                 : fd_tree_attention(&dq, &dk, &dv, prefix, lens, mask, w, &d, lse, s);
  });
  return o.give();
  END_HANDLE_TH_ERRORS
}

// (k_new, v_new, k_pages, v_pages, k_scale, v_scale, block_table, start_lens, new_lens, stream); scales None:
// pages of the new rows' type
PyObject* pages_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const bool fp8 = a[4] != Py_None;
  const at::Tensor &k = tensor(a[0], "k_new"), &v = tensor(a[1], "v_new"), &kp = tensor(a[2], "k_pages"), &vp = tensor(a[3], "v_pages");
  const float ks = fp8 ? to_float(a[4]) : 1.f, vs = fp8 ? to_float(a[5]) : 1.f;
  const Table t(a[6], kp.device());
  const int32_t *start = int32s(a[7], "start_lens", kp.device(), {t.batch}), *lens = int32s(a[8], "new_lens", kp.device(), {t.batch});
  need(kp, {{"k_new", &k}, {"v_new", &v}, {"v_pages", &vp}});
  const fd_tensor dk = desc(k), dv = desc(v);
  fd_tensor pk = desc(kp), pv = desc(vp);
  run(fp8 ? "fd_pages_append_fp8" : "fd_pages_append", kp, Lane(a[9], kp.device()), a, n, [&](void* s) {
    return fp8 ? fd_pages_append_fp8(&dk, &dv, &pk, &pv, ks, vs, t.data, t.per, t.batch, start, lens, s)
               : fd_pages_append(&dk, &dv, &pk, &pv, t.data, t.per, t.batch, start, lens, s);
  });
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (page_refs, block_table, want_lens, page_size, stream)
PyObject* pages_reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 5);
  const at::Tensor& r = tensor(a[0], "page_refs");
  const c10::Device dev = r.device();
  int32_t* refs = int32s(a[0], "page_refs", dev, {r.numel()});
  const Table t(a[1], dev);
  const int32_t *want = int32s(a[2], "want_lens", dev, {t.batch}), size = to_int32(a[3], "page_size");
  need(r, {});
  run("fd_pages_reserve", r, Lane(a[4], dev), a, n, [&](void* s) {
    return fd_pages_reserve(refs, static_cast<int32_t>(r.numel()), t.data, t.per, t.batch, want, size, s);
  });
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (k_pages, v_pages, page_refs, block_table, cache_lens, src_seqs, dst_seqs, stream)
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const at::Tensor &k = tensor(a[0], "k_pages"), &v = tensor(a[1], "v_pages");
  const c10::Device dev = k.device();
  TORCH_CHECK_VALUE(k.dim() > 0, "k_pages must be a page pool");
  int32_t* refs = int32s(a[2], "page_refs", dev, {k.size(0)});
  const Table t(a[3], dev);
  int32_t* lens = int32s(a[4], "cache_lens", dev, {t.batch});
  const int64_t pairs = numel(a[5], "src_seqs");
  const int32_t *src = int32s(a[5], "src_seqs", dev, {pairs}), *dst = int32s(a[6], "dst_seqs", dev, {pairs});
  need(k, {{"v_pages", &v}});
  fd_tensor dk = desc(k), dv = desc(v);
  run("fd_pages_fork", k, Lane(a[7], dev), a, n, [&](void* s) {
    return fd_pages_fork(&dk, &dv, refs, t.data, t.per, t.batch, lens, src, dst, static_cast<int32_t>(pairs), s);
  });
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (page_refs, block_table, cache_lens, seqs, stream)
PyObject* pages_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 5);
  const at::Tensor& r = tensor(a[0], "page_refs");
  const c10::Device dev = r.device();
  int32_t* refs = int32s(a[0], "page_refs", dev, {r.numel()});
  const Table t(a[1], dev);
  int32_t* lens = int32s(a[2], "cache_lens", dev, {t.batch});
  const int64_t listed = numel(a[3], "seqs");
  const int32_t* seqs = int32s(a[3], "seqs", dev, {listed});
  need(r, {});
  run("fd_pages_free", r, Lane(a[4], dev), a, n, [&](void* s) {
    return fd_pages_free(refs, static_cast<int32_t>(r.numel()), t.data, t.per, t.batch, lens, seqs, static_cast<int32_t>(listed), s);
  });
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (k_pages, v_pages, page_refs, block_table, cache_lens, start_lens, keep, keep_lens, stream)
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const at::Tensor &k = tensor(a[0], "k_pages"), &v = tensor(a[1], "v_pages"), &lists = tensor(a[6], "keep");
  const c10::Device dev = k.device();
  TORCH_CHECK_VALUE(k.dim() > 0, "k_pages must be a page pool");
  int32_t* refs = int32s(a[2], "page_refs", dev, {k.size(0)});
  const Table t(a[3], dev);
  int32_t* lens = int32s(a[4], "cache_lens", dev, {t.batch});
  const int32_t *start = int32s(a[5], "start_lens", dev, {t.batch}), *kept = int32s(a[7], "keep_lens", dev, {t.batch});
  const int64_t most = last(lists);
  const int32_t* keep = int32s(a[6], "keep", dev, {t.batch, most});
  need(k, {{"v_pages", &v}});
  fd_tensor dk = desc(k), dv = desc(v);
  run("fd_pages_compact", k, Lane(a[8], dev), a, n, [&](void* s) {
    return fd_pages_compact(&dk, &dv, refs, t.data, t.per, t.batch, lens, start, keep, static_cast<int32_t>(most), kept, s);
  });
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (callable): called as callable(status, name) for a status that is not FD_OK; has to raise
PyObject* set_raise(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_raise, f);
  Py_RETURN_NONE;
}

#define FD_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    FD_FAST(prompt_attention), FD_FAST(tree_attention), FD_FAST(pages_append), FD_FAST(pages_reserve), FD_FAST(pages_fork),
    FD_FAST(pages_free), FD_FAST(pages_compact), {"set_raise", set_raise, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fd_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__fd_binding() {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "torch_version", FD_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
