// The paged calls' short way from Python to the library: the same checks as
// in paged.py, made on the tensors themselves, then the call.
//
// A decode step's calls take 4 to 15 us of device time, and a Python call that
// reads device, type, shape, strides and address of a dozen tensors one
// attribute at a time takes longer than that (a page map 10 us, a decode 20).
// Each function here takes the arguments of its namesake in paged.py but for
// the stream (it launches on the current one of the current device) and returns
// kNotPlain, having done nothing, for whatever it does not handle: arguments
// that are wrong, tensors of a subclass or of another device, cells that are
// neither a list nor an integer array.  The caller then goes the long way, which
// explains what is wrong.  Otherwise the result is the library's status (decode:
// the output tensor on success).  Nothing is kept between calls.
//
// The library's functions are given as addresses (bind), so this module needs
// no link to it.

#include <Python.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <climits>
#include <cstdint>
#include <initializer_list>

#include "loopkv.h"

namespace {

constexpr int kNotPlain = -1;

decltype(&loopkv_page_map) page_map_fn;
decltype(&loopkv_page_release) page_release_fn;
decltype(&loopkv_paged_append) append_fn;
decltype(&loopkv_paged_workspace) workspace_fn;
decltype(&loopkv_paged_decode) decode_fn;

PyObject* status(long rc) { return PyLong_FromLong(rc); }

const at::Tensor* tensor(PyObject* o, int64_t dim) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.defined() && t.layout() == at::kStrided && t.dim() == dim ? &t : nullptr;
}

bool on(const at::Tensor& t, at::ScalarType type, int index) {
  return t.scalar_type() == type && t.is_cuda() && t.get_device() == index;
}

// A contiguous tensor of a type and shape on a device.
bool full(PyObject* o, at::ScalarType type, int index, at::IntArrayRef shape, void** at_) {
  const at::Tensor* t = tensor(o, (int64_t)shape.size());
  if (t == nullptr || !on(*t, type, index) || t->sizes() != shape || !t->is_contiguous()) return false;
  *at_ = t->data_ptr();
  return true;
}

template <typename T>
bool ints(PyObject* o, int index, std::initializer_list<int64_t> shape, T** at_) {
  void* p = nullptr;
  if (!full(o, at::kInt, index, at::IntArrayRef(shape.begin(), shape.size()), &p)) return false;
  *at_ = static_cast<T*>(p);
  return true;
}

// The same or None (nullptr).
template <typename T>
bool ints_or_none(PyObject* o, int index, std::initializer_list<int64_t> shape, T** at_) {
  if (o == Py_None) {
    *at_ = nullptr;
    return true;
  }
  return ints(o, index, shape, at_);
}

bool small(int64_t n) { return n >= 0 && n <= INT32_MAX; }

bool count(PyObject* o, int32_t* n) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &over);
  if (over != 0 || !small(x)) return false;
  *n = (int32_t)x;
  return true;
}

// The device all tensors of a call are on, if it is the current one.
bool current_device(const at::Tensor& t, int* index) {
  if (!t.is_cuda()) return false;
  *index = t.get_device();
  return *index == c10::cuda::current_device();
}

struct Cells {
  int32_t n = 0;
  int32_t cell[LOOPKV_MAX_CELLS_PER_CALL];

  bool take(PyObject* o) {
    if (PyList_CheckExact(o)) {
      const Py_ssize_t size = PyList_GET_SIZE(o);
      if (size < 1 || size > LOOPKV_MAX_CELLS_PER_CALL) return false;
      for (Py_ssize_t i = 0; i < size; ++i) {
        PyObject* x = PyList_GET_ITEM(o, i);
        int over = 0;
        if (!PyLong_CheckExact(x) || !put(PyLong_AsLongLongAndOverflow(x, &over)) || over != 0) return false;
      }
      return true;
    }
    if (!PyObject_CheckBuffer(o)) return false;
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) != 0) {
      PyErr_Clear();
      return false;
    }
    const char* f = b.format;
    bool good = b.ndim == 1 && f != nullptr && f[0] != 0 && f[1] == 0 && b.shape[0] >= 1 &&
                b.shape[0] <= LOOPKV_MAX_CELLS_PER_CALL;
    if (good && f[0] == 'i' && b.itemsize == 4) {
      for (Py_ssize_t i = 0; i < b.shape[0]; ++i) put(static_cast<const int32_t*>(b.buf)[i]);
    } else if (good && (f[0] == 'l' || f[0] == 'q') && b.itemsize == 8) {
      for (Py_ssize_t i = 0; good && i < b.shape[0]; ++i) good = put(static_cast<const int64_t*>(b.buf)[i]);
    } else {
      good = false;
    }
    PyBuffer_Release(&b);
    return good;
  }

  bool put(long long x) {
    if (x < INT32_MIN || x > INT32_MAX) return false;
    cell[n++] = (int32_t)x;
    return true;
  }
};

struct Pool {
  loopkv_page_pool c{};
  at::ScalarType vectors;
  int index = 0;

  bool take(PyObject* k_pages, PyObject* v_pages, PyObject* meta) {
    const at::Tensor* k = tensor(k_pages, 5);
    if (k == nullptr || !current_device(*k, &index)) return false;
    const at::ScalarType type = k->scalar_type();
    if (type == at::kBFloat16) c.format = LOOPKV_PAGE_BF16;
    else if (type == at::kHalf) c.format = LOOPKV_PAGE_F16;
    else if (type == at::kByte) c.format = LOOPKV_PAGE_Q8;
    else return false;
    vectors = type == at::kHalf ? at::kHalf : at::kBFloat16;
    const at::IntArrayRef shape = k->sizes();
    for (int64_t n : shape)
      if (!small(n)) return false;
    void* m = nullptr;
    if (!full(k_pages, type, index, shape, &c.k) || !full(v_pages, type, index, shape, &c.v)) return false;
    if ((meta == Py_None) != (type != at::kByte)) return false;
    if (meta != Py_None) {
      const int64_t per[5] = {shape[0], shape[1], shape[2], shape[3], 4};
      if (!full(meta, at::kFloat, index, per, &m)) return false;
    }
    c.meta = static_cast<float*>(m);
    c.n_cells = (int32_t)shape[0];
    c.n_pages = (int32_t)shape[1];
    c.n_kv_heads = (int32_t)shape[2];
    c.page_size = (int32_t)shape[3];
    c.head_dim = (int32_t)shape[4];
    return true;
  }
};

// [cells, rows, heads, head dim] vectors; heads < 0: any number.
struct Rows {
  loopkv_rows c{};
  int64_t heads = 0;

  bool take(PyObject* o, at::ScalarType type, int index, int64_t cells, int64_t rows, int64_t want_heads, int64_t dim) {
    const at::Tensor* t = tensor(o, 4);
    if (t == nullptr || !on(*t, type, index)) return false;
    const at::IntArrayRef n = t->sizes(), s = t->strides();
    if (n[0] != cells || n[1] != rows || (want_heads >= 0 && n[2] != want_heads) || n[3] != dim || s[3] != 1) return false;
    heads = n[2];
    c.data = t->data_ptr();
    c.cell_stride = n[0] <= 1 ? 0 : s[0];
    c.row_stride = n[1] <= 1 ? 0 : s[1];
    c.head_stride = n[2] <= 1 ? 0 : s[2];
    return ((c.cell_stride | c.row_stride | c.head_stride) & 7) == 0 && (reinterpret_cast<uintptr_t>(c.data) & 15) == 0;
  }
};

void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }

PyObject* page_map(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12) return status(kNotPlain);
  try {
    const at::Tensor *table = tensor(a[2], 2), *free = tensor(a[3], 1), *slots = tensor(a[6], 1);
    int index;
    int32_t page_size;
    if (table == nullptr || free == nullptr || slots == nullptr || !current_device(*table, &index) || !count(a[5], &page_size))
      return status(kNotPlain);
    const int64_t batch = table->size(0), width = table->size(1), pages = free->numel(), rows = slots->numel();
    int32_t *len, *add, *tab, *fre, *cnt, *slo, *sta, *newest, *len_out, *cnt_out;
    uint32_t* st;
    if (!small(batch) || !small(width) || !small(pages) || !small(rows) || !ints(a[0], index, {batch}, &len) ||
        !ints(a[1], index, {batch}, &add) || !ints(a[2], index, {batch, width}, &tab) ||
        !ints(a[3], index, {pages}, &fre) || !ints(a[4], index, {1}, &cnt) || !ints(a[6], index, {rows}, &slo) ||
        !ints(a[7], index, {batch + 1}, &sta) || !ints_or_none(a[8], index, {batch}, &newest) ||
        !ints_or_none(a[9], index, {batch}, &len_out) || !ints_or_none(a[10], index, {1}, &cnt_out) ||
        !ints_or_none(a[11], index, {1}, &st))
      return status(kNotPlain);
    return status(page_map_fn((int32_t)batch, page_size, (int32_t)width, (int32_t)pages, (int32_t)rows, len, add, tab, fre,
                              cnt, slo, sta, newest, len_out ? len_out : len, cnt_out ? cnt_out : cnt, st,
                              stream_of(index)));
  } catch (...) {
    return status(kNotPlain);
  }
}

PyObject* page_release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) return status(kNotPlain);
  try {
    const at::Tensor *table = tensor(a[2], 2), *free = tensor(a[3], 1);
    int index;
    int32_t page_size;
    if (table == nullptr || free == nullptr || !current_device(*table, &index) || !count(a[5], &page_size))
      return status(kNotPlain);
    const int64_t batch = table->size(0), width = table->size(1), pages = free->numel();
    int32_t *len, *cut, *tab, *fre, *cnt, *len_out, *cnt_out;
    uint32_t* st;
    if (!small(batch) || !small(width) || !small(pages) || !ints(a[0], index, {batch}, &len) ||
        !ints(a[1], index, {batch}, &cut) || !ints(a[2], index, {batch, width}, &tab) ||
        !ints(a[3], index, {pages}, &fre) || !ints(a[4], index, {1}, &cnt) ||
        !ints_or_none(a[6], index, {batch}, &len_out) || !ints_or_none(a[7], index, {1}, &cnt_out) ||
        !ints_or_none(a[8], index, {1}, &st))
      return status(kNotPlain);
    return status(page_release_fn((int32_t)batch, page_size, (int32_t)width, (int32_t)pages, len, cut, tab, fre, cnt,
                                  len_out ? len_out : len, cnt_out ? cnt_out : cnt, st, stream_of(index)));
  } catch (...) {
    return status(kNotPlain);
  }
}

PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) return status(kNotPlain);
  try {
    Cells cells;
    Pool pool;
    Rows k, v;
    const at::Tensor* slots = tensor(a[3], 1);
    int32_t* slo;
    uint32_t* st;
    if (slots == nullptr || !small(slots->numel()) || !cells.take(a[0]) || !pool.take(a[4], a[5], a[6]))
      return status(kNotPlain);
    const int64_t rows = slots->numel();
    if (!k.take(a[1], pool.vectors, pool.index, cells.n, rows, pool.c.n_kv_heads, pool.c.head_dim) ||
        !v.take(a[2], pool.vectors, pool.index, cells.n, rows, pool.c.n_kv_heads, pool.c.head_dim) ||
        !ints(a[3], pool.index, {rows}, &slo) || !ints_or_none(a[7], pool.index, {1}, &st))
      return status(kNotPlain);
    return status(append_fn(&pool.c, cells.cell, cells.n, (int32_t)rows, slo, &k.c, &v.c, st, stream_of(pool.index)));
  } catch (...) {
    return status(kNotPlain);
  }
}

PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 14) return status(kNotPlain);
  try {
    Cells cells;
    Pool pool;
    Rows q, cur_k, cur_v;
    const at::Tensor* table = tensor(a[4], 2);
    if (table == nullptr || !cells.take(a[0]) || !pool.take(a[2], a[3], a[6])) return status(kNotPlain);
    const int64_t batch = table->size(0), width = table->size(1);
    const int index = pool.index;
    int32_t *tab, *len;
    uint32_t* st;
    if (!small(batch) || !small(width) || pool.c.n_kv_heads < 1 ||
        !q.take(a[1], pool.vectors, index, cells.n, batch, -1, pool.c.head_dim) || q.heads % pool.c.n_kv_heads != 0 ||
        !ints(a[4], index, {batch, width}, &tab) || !ints(a[5], index, {batch}, &len) ||
        !ints_or_none(a[13], index, {1}, &st) || (!PyFloat_CheckExact(a[12]) && !PyLong_CheckExact(a[12])))
      return status(kNotPlain);
    const bool with_cur = a[7] != Py_None;
    if (with_cur != (a[8] != Py_None)) return status(kNotPlain);
    uint8_t current[LOOPKV_MAX_CELLS_PER_CALL];
    for (int i = 0; i < cells.n; ++i) current[i] = with_cur;
    if (a[9] != Py_None) {  // a truth value (or byte) per listed cell
      Py_buffer b;
      if (!PyObject_CheckBuffer(a[9])) return status(kNotPlain);
      if (PyObject_GetBuffer(a[9], &b, PyBUF_C_CONTIGUOUS) != 0) {
        PyErr_Clear();
        return status(kNotPlain);
      }
      bool good = b.ndim == 1 && b.itemsize == 1 && b.len == cells.n;
      for (int i = 0; good && i < cells.n; ++i) {
        current[i] = static_cast<const uint8_t*>(b.buf)[i];
        good = with_cur || current[i] == 0;
      }
      PyBuffer_Release(&b);
      if (!good) return status(kNotPlain);
    }
    if (with_cur && (!cur_k.take(a[7], pool.vectors, index, cells.n, batch, pool.c.n_kv_heads, pool.c.head_dim) ||
                     !cur_v.take(a[8], pool.vectors, index, cells.n, batch, pool.c.n_kv_heads, pool.c.head_dim)))
      return status(kNotPlain);
    const int64_t shape[4] = {cells.n, batch, q.heads, pool.c.head_dim};
    void *out = nullptr, *lse = nullptr;
    if (a[10] != Py_None && !full(a[10], pool.vectors, index, shape, &out)) return status(kNotPlain);
    if (a[11] != Py_None && !full(a[11], at::kFloat, index, at::IntArrayRef(shape, 3), &lse)) return status(kNotPlain);
    const double scale = PyFloat_AsDouble(a[12]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      return status(kNotPlain);
    }
    if (scale > 0 && static_cast<float>(scale) == 0.f) return status(kNotPlain);
    const loopkv_paged_desc desc{(int32_t)batch, (int32_t)width, (int32_t)(q.heads / pool.c.n_kv_heads), (float)scale};
    size_t bytes = 0;
    loopkv_status rc = workspace_fn(&pool.c, &desc, &bytes);
    if (rc != LOOPKV_OK) return status(rc);
    at::Tensor made;
    if (out == nullptr) {
      made = at::empty(at::IntArrayRef(shape, 4), THPVariable_Unpack(a[1]).options());
      out = made.data_ptr();
    }
    // the workspace goes back to the allocator at once: what gets it next on this stream runs behind the call
    const c10::cuda::CUDAStream stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index);
    void* work = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, stream.stream());
    rc = decode_fn(&pool.c, &desc, cells.cell, current, cells.n, tab, len, &q.c, with_cur ? &cur_k.c : nullptr,
                   with_cur ? &cur_v.c : nullptr, out, static_cast<float*>(lse), work, bytes, st, stream.stream());
    c10::cuda::CUDACachingAllocator::raw_delete(work);
    if (rc != LOOPKV_OK) return status(rc);
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[10]);
    return a[10];
  } catch (...) {
    return status(kNotPlain);
  }
}

// bind(address, ...) of the five library functions, in the order below.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* fn[5];
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "five addresses");
    return nullptr;
  }
  for (int i = 0; i < 5; ++i) {
    fn[i] = PyLong_AsVoidPtr(a[i]);
    if (fn[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  page_map_fn = reinterpret_cast<decltype(page_map_fn)>(fn[0]);
  page_release_fn = reinterpret_cast<decltype(page_release_fn)>(fn[1]);
  append_fn = reinterpret_cast<decltype(append_fn)>(fn[2]);
  workspace_fn = reinterpret_cast<decltype(workspace_fn)>(fn[3]);
  decode_fn = reinterpret_cast<decltype(decode_fn)>(fn[4]);
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(page_map), METHOD(page_release), METHOD(paged_append),
                         METHOD(paged_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
