// The Python binding of the paged latent cache's calls: argument checks, outputs
// and workspaces, and the C entry points of include/dsa_cp.h on the tensors'
// device and stream.  In C++ because these are calls of a decode step, a few of
// them every few microseconds: the same checks and allocations from Python through
// ctypes took 21 us for the attention of one token whose kernels take 13.
//
// Each function takes its arguments in order, raises ValueError for tensors or
// sizes that do not fit, and returns its result, or the dsa_status of a call that
// the library refused as an int.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <optional>

#include "../../include/dsa_cp.h"

namespace {

struct Refused {};  // a Python error is set

template <typename... A>
[[noreturn]] void refuse(const char *form, A... args) {
  PyErr_Format(PyExc_ValueError, form, args...);
  throw Refused{};
}

const char *type_name(at::ScalarType t) {
  return t == at::kBFloat16 ? "torch.bfloat16" : t == at::kFloat ? "torch.float32" : t == at::kInt ? "torch.int32" : "torch.uint8";
}

// The call's tensors lie on one device, that of the first.
struct Call {
  c10::DeviceIndex device = -1;

  const at::Tensor &any(PyObject *o, at::ScalarType type, const char *name) {
    if (!THPVariable_Check(o)) refuse("%s must be a CUDA tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    if (t.scalar_type() != type) refuse("%s must be %s", name, type_name(type));
    if (device < 0) device = t.get_device();
    if (t.get_device() != device)
      refuse("tensors on different devices: cuda:%d and %s on cuda:%d", static_cast<int>(device), name,
             static_cast<int>(t.get_device()));
    return t;
  }
  const at::Tensor &full(PyObject *o, at::ScalarType type, int dims, const char *name, const char *form) {
    const at::Tensor &t = any(o, type, name);
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    if (t.dim() != dims) refuse("%s must be %s", name, form);
    return t;
  }
  const at::Tensor &ints(PyObject *o, int64_t n, const char *name) {
    const at::Tensor &t = full(o, at::kInt, 1, name, "one-dimensional");
    if (t.size(0) != n) refuse("%s must be [%lld]", name, static_cast<long long>(n));
    return t;
  }
  const int32_t *maybe_ints(PyObject *o, int64_t n, const char *name) {
    return o == Py_None ? nullptr : ints(o, n, name).const_data_ptr<int32_t>();
  }
  const at::Tensor &table(PyObject *o) {
    const at::Tensor &t = full(o, at::kInt, 2, "page_table", "[batch, max_pages]");
    if (t.size(1) < 1 || t.numel() > INT32_MAX)
      refuse("page_table must be [batch, max_pages] with a page at least and fewer than 2^31 entries");
    return t;
  }
};

int64_t integer(PyObject *o, const char *name) {
  PyObject *i = PyNumber_Index(o);
  if (!i) throw Refused{};
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(i, &over);
  Py_DECREF(i);
  if (over || v < INT32_MIN || v > INT32_MAX) refuse("%s is not below 2^31", name);
  return v;
}

int32_t below(int64_t v, const char *name) {
  if (v > INT32_MAX) refuse("%s = %lld is not below 2^31", name, static_cast<long long>(v));
  return static_cast<int32_t>(v);
}

int32_t rows_of_page(int64_t p) {
  if (p != 16 && p != 32 && p != 64 && p != 128)
    refuse("pages of %lld rows: a page has 16, 32, 64 or 128", static_cast<long long>(p));
  return static_cast<int32_t>(p);
}

// A cache [num_pages, P, D] whose rows are contiguous and start on 16-byte boundaries.
struct Pages {
  void *data;
  int32_t pages, rows;
  int64_t D, page_stride, row_stride;
};
Pages pages(Call &c, PyObject *o) {
  const at::Tensor &t = c.any(o, at::kBFloat16, "cache");
  if (t.dim() != 3) refuse("cache must be [num_pages, page_size, D]");
  Pages p{t.data_ptr(), 0, rows_of_page(t.size(1)), t.size(2), 0, t.stride(1)};
  p.pages = below(t.size(0), "num_pages");
  below(t.size(0) * p.rows, "the number of rows of cache");
  p.page_stride = p.pages > 1 ? t.stride(0) : p.row_stride * p.rows;
  if (t.stride(2) != 1 || p.row_stride < p.D || p.row_stride % 8 || p.page_stride % 8 ||
      p.page_stride < (p.rows - 1) * p.row_stride + p.D || reinterpret_cast<uintptr_t>(p.data) % 16)
    refuse("the rows of cache must be contiguous, not overlap and start on 16-byte boundaries");
  return p;
}

// The device and stream of a call made current, so that what it allocates belongs
// to the stream its kernels run on.
class Launch {
 public:
  Launch(const Call &c, PyObject *stream) {
    if (stream == Py_None) {
      guard_.emplace(c.device);
      stream_ = c10::cuda::getCurrentCUDAStream(c.device).stream();
      return;
    }
    const int64_t id = attribute(stream, "stream_id"), index = attribute(stream, "device_index"),
                  type = attribute(stream, "device_type");
    if (index != c.device)
      refuse("the stream is on cuda:%d, the tensors on cuda:%d", static_cast<int>(index), static_cast<int>(c.device));
    const auto s = c10::cuda::CUDAStream::unpack3(id, static_cast<c10::DeviceIndex>(index), static_cast<c10::DeviceType>(type));
    on_.emplace(s);
    stream_ = s.stream();
  }
  dsa_stream_t stream() const { return reinterpret_cast<dsa_stream_t>(stream_); }
  static at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Call &c) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, c.device)));
  }

 private:
  static int64_t attribute(PyObject *o, const char *name) {
    PyObject *v = PyObject_GetAttrString(o, name);
    if (!v) throw Refused{};
    const long long x = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (x == -1 && PyErr_Occurred()) throw Refused{};
    return x;
  }
  std::optional<c10::cuda::CUDAGuard> guard_;
  std::optional<c10::cuda::CUDAStreamGuard> on_;
  cudaStream_t stream_ = nullptr;
};

// The status of a library call, made without the interpreter's lock.
template <typename F>
dsa_status unlocked(F f) {
  PyThreadState *state = PyEval_SaveThread();
  const dsa_status st = f();
  PyEval_RestoreThread(state);
  return st;
}

PyObject *status(dsa_status st) { return PyLong_FromLong(st); }
PyObject *same(PyObject *o) { return Py_NewRef(o); }

PyObject *pages_update(PyObject *const *a) {
  Call c;
  const at::Tensor &table = c.table(a[0]);
  const int64_t B = table.size(0);
  const int32_t *held = c.ints(a[1], B, "held_lens").const_data_ptr<int32_t>();
  const int32_t *seq = c.ints(a[2], B, "seq_lens").const_data_ptr<int32_t>();
  const at::Tensor &pool = c.full(a[3], at::kInt, 1, "free_pages", "[num_pages]");
  const int32_t num_pages = below(pool.numel(), "num_pages");
  int32_t *count = c.ints(a[4], 1, "free_count").data_ptr<int32_t>();
  const int32_t P = rows_of_page(integer(a[5], "page_size"));
  const Launch on(c, a[6]);
  const dsa_status st = unlocked([&] {
    return dsa_pages_update(table.data_ptr<int32_t>(), static_cast<int32_t>(B), static_cast<int32_t>(table.size(1)), held, seq,
                            P, pool.data_ptr<int32_t>(), num_pages, count, on.stream());
  });
  return st == DSA_OK ? same(a[0]) : status(st);
}

PyObject *pages_slots(PyObject *const *a) {
  Call c;
  const at::Tensor &table = c.table(a[0]);
  const int64_t B = table.size(0);
  const int32_t *first = c.maybe_ints(a[1], B, "first");
  const int32_t *seq = c.ints(a[2], B, "seq_lens").const_data_ptr<int32_t>();
  const int32_t P = rows_of_page(integer(a[3], "page_size"));
  const int64_t n = integer(a[4], "num_slots");
  if (n < 0) refuse("num_slots = %lld", static_cast<long long>(n));
  at::Tensor out;
  if (a[5] != Py_None) out = c.ints(a[5], n, "out");
  const Launch on(c, a[6]);
  if (!out.defined()) out = Launch::empty({n}, at::kInt, c);
  const dsa_status st = unlocked([&] {
    return dsa_pages_slots(table.const_data_ptr<int32_t>(), static_cast<int32_t>(B), static_cast<int32_t>(table.size(1)), first,
                           seq, P, out.data_ptr<int32_t>(), static_cast<int32_t>(n), on.stream());
  });
  return st != DSA_OK ? status(st) : a[5] != Py_None ? same(a[5]) : THPVariable_Wrap(std::move(out));
}

PyObject *pages_append(PyObject *const *a) {
  Call c;
  const Pages cache = pages(c, a[3]);
  const at::Tensor &kv = c.any(a[0], at::kBFloat16, "kv");
  if (kv.dim() != 2 || kv.size(1) != cache.D) refuse("kv must be [n, %lld]", static_cast<long long>(cache.D));
  const int32_t n = below(kv.size(0), "n");
  const int64_t stride = n > 1 ? kv.stride(0) : cache.D;
  if (kv.stride(1) != 1 || stride < cache.D || stride % 8 || reinterpret_cast<uintptr_t>(kv.data_ptr()) % 16)
    refuse("the rows of kv must be contiguous, not overlap and start on 16-byte boundaries");
  if (cache.D < 8 || cache.D % 8 || cache.D > INT32_MAX) refuse("D must be a multiple of 8");
  const int32_t *slots = c.ints(a[2], n, "slots").const_data_ptr<int32_t>();
  if ((a[1] == Py_None) != (a[4] == Py_None) || (a[1] == Py_None) != (a[5] == Py_None))
    refuse("k_idx, key_cache and block_keys come together");
  const void *k_idx = nullptr;
  void *keys = nullptr, *means = nullptr;
  int32_t DI = 8;
  if (a[1] != Py_None) {
    const at::Tensor &k = c.full(a[1], at::kBFloat16, 2, "k_idx", "[n, DI]");
    const at::Tensor &kc = c.full(a[4], at::kBFloat16, 3, "key_cache", "[num_pages, page_size, DI]");
    const at::Tensor &bk = c.full(a[5], at::kBFloat16, 2, "block_keys", "[num_pages, DI]");
    DI = below(k.size(1), "DI");
    if (k.size(0) != n || kc.size(0) != cache.pages || kc.size(1) != cache.rows || kc.size(2) != DI ||
        bk.size(0) != cache.pages || bk.size(1) != DI)
      refuse("k_idx must be [%d, DI], key_cache [%d, %d, DI] and block_keys [%d, DI]", n, cache.pages, cache.rows, cache.pages);
    k_idx = k.const_data_ptr();
    keys = kc.data_ptr();
    means = bk.data_ptr();
  }
  const Launch on(c, a[6]);
  const dsa_status st = unlocked([&] {
    return dsa_pages_append(kv.const_data_ptr(), stride, k_idx, slots, n, static_cast<int32_t>(cache.D), DI, cache.data, cache.page_stride, cache.row_stride, cache.pages, cache.rows, keys, means, on.stream());
  });
  return st == DSA_OK ? same(Py_None) : status(st);
}

PyObject *block_select(PyObject *const *a) {
  Call c;
  const at::Tensor &q = c.full(a[0], at::kBFloat16, 3, "q_idx", "[n, HI, DI]");
  const int32_t n = below(q.size(0), "n"), HI = below(q.size(1), "HI"), DI = below(q.size(2), "DI");
  const at::Tensor &w = c.full(a[1], at::kFloat, 2, "w", "[n, HI]");
  if (w.size(0) != n || w.size(1) != HI) refuse("w must be [%d, %d]", n, HI);
  const at::Tensor &keys = c.full(a[2], at::kBFloat16, 2, "block_keys", "[num_pages, DI]");
  if (keys.size(1) != DI) refuse("block_keys must be [num_pages, %d]", DI);
  const at::Tensor &table = c.table(a[3]);
  const int32_t *lens = c.ints(a[4], n, "lens").const_data_ptr<int32_t>();
  const int32_t P = rows_of_page(integer(a[5], "page_size"));
  const int64_t nsel = integer(a[6], "nsel"), keep_first = integer(a[7], "keep_first"), keep_last = integer(a[8], "keep_last");
  const int32_t *req = c.maybe_ints(a[9], n, "req");
  if (!req && n > table.size(0) && a[9] == Py_None) refuse("more queries than requests (pass req)");
  below(keys.size(0) * P, "the number of rows");
  below(n * std::max<int64_t>(nsel, 1), "n * nsel");
  at::Tensor out;
  if (a[10] != Py_None) {
    out = c.full(a[10], at::kInt, 2, "out", "[n, nsel]");
    if (out.size(0) != n || out.size(1) != nsel) refuse("out must be [%d, %lld]", n, static_cast<long long>(nsel));
  }
  const Launch on(c, a[11]);
  if (!out.defined()) out = Launch::empty({n, std::max<int64_t>(nsel, 0)}, at::kInt, c);
  const dsa_status st = unlocked([&] {
    return dsa_block_select(q.const_data_ptr(), w.const_data_ptr<float>(), n, HI, DI, keys.const_data_ptr(),
                            static_cast<int32_t>(keys.size(0)), P, table.const_data_ptr<int32_t>(),
                            static_cast<int32_t>(table.size(0)), static_cast<int32_t>(table.size(1)), lens, req,
                            static_cast<int32_t>(nsel), static_cast<int32_t>(keep_first), static_cast<int32_t>(keep_last),
                            out.data_ptr<int32_t>(), on.stream());
  });
  return st != DSA_OK ? status(st) : a[10] != Py_None ? same(a[10]) : THPVariable_Wrap(std::move(out));
}

PyObject *paged_attn(PyObject *const *a) {
  Call c;
  const at::Tensor &q = c.full(a[0], at::kBFloat16, 3, "q", "[n, H, D]");
  const int32_t n = below(q.size(0), "n"), H = below(q.size(1), "H"), D = below(q.size(2), "D");
  const Pages cache = pages(c, a[1]);
  if (cache.D != D) refuse("q / cache do not match in D");
  const at::Tensor &table = c.table(a[2]);
  const int32_t *lens = c.ints(a[3], n, "lens").const_data_ptr<int32_t>();
  const double scale = PyFloat_AsDouble(a[4]);
  if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
  const int32_t Dv = static_cast<int32_t>(integer(a[5], "Dv"));
  int32_t nsel = 0;
  const int32_t *blocks = nullptr;
  if (a[6] != Py_None) {
    const at::Tensor &b = c.full(a[6], at::kInt, 2, "blocks", "[n, nsel]");
    if (b.size(0) != n || b.size(1) < 1) refuse("blocks must be [%d, nsel]", n);
    below(b.numel(), "n * nsel");
    nsel = static_cast<int32_t>(b.size(1));
    blocks = b.const_data_ptr<int32_t>();
  }
  const int32_t *req = c.maybe_ints(a[7], n, "req");
  if (a[7] == Py_None && n > table.size(0)) refuse("more queries than requests (pass req)");
  const float *sink = nullptr;
  if (a[8] != Py_None) {
    const at::Tensor &s = c.full(a[8], at::kFloat, 1, "attn_sink", "[H]");
    if (s.size(0) != H) refuse("attn_sink must be [%d]", H);
    sink = s.const_data_ptr<float>();
  }
  at::Tensor out, ws;
  if (a[9] != Py_None) {
    out = c.full(a[9], at::kBFloat16, 3, "out", "[n, H, Dv]");
    if (out.size(0) != n || out.size(1) != H || out.size(2) != Dv) refuse("out must be [%d, %d, %d]", n, H, Dv);
  }
  if (a[10] != Py_None) {
    ws = c.any(a[10], at::kByte, "workspace");
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
  }
  if (Dv < 0) refuse("Dv = %d", Dv);
  const Launch on(c, a[11]);
  if (!ws.defined()) {
    size_t bytes = 0;
    const dsa_status st = dsa_paged_attn_workspace_size(n, H, static_cast<int32_t>(table.size(1)), nsel, cache.rows, &bytes);
    if (st != DSA_OK) return status(st);
    ws = Launch::empty({static_cast<int64_t>(bytes)}, at::kByte, c);
  }
  if (!out.defined()) out = Launch::empty({n, H, Dv}, at::kBFloat16, c);
  const dsa_status st = unlocked([&] {
    return dsa_paged_attn(q.const_data_ptr(), n, cache.data, cache.page_stride, cache.row_stride, cache.pages, cache.rows,
                          table.const_data_ptr<int32_t>(), static_cast<int32_t>(table.size(0)),
                          static_cast<int32_t>(table.size(1)), lens, req, blocks, nsel, sink, static_cast<float>(scale), H, D,
                          Dv, out.data_ptr(), ws.data_ptr(), static_cast<size_t>(ws.numel()), on.stream());
  });
  return st != DSA_OK ? status(st) : a[9] != Py_None ? same(a[9]) : THPVariable_Wrap(std::move(out));
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", N, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS  // what PyTorch throws, out of memory, say, is raised as its own calls raise it
  try {
    return F(args);
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(pages_update, 7),  ENTRY(pages_slots, 7), ENTRY(pages_append, 7),
                         ENTRY(block_select, 12), ENTRY(paged_attn, 12), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
