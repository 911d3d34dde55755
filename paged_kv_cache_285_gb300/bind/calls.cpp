// The block-scaled, microscaled, gather, window and moving calls from Python
// tensors straight to the C ABI: the argument checks of the package's Python functions on the tensors
// themselves.
//
// What bounds a small call is the host: its kernel takes 2 to 8 us, the ABI call
// with its launch 3.4 to 5, and a dozen tensors looked at from Python another 7
// (shape, dtype, device, contiguity and pointer of each are Python objects made
// and dropped).  Here the same checks are reads of the tensors' fields.
//
// A function returns the call's status, or None without having called anything
// where an argument is not of the plain kind it knows (a check that fails, a
// number outside its type, a tensor subclass, another current device); the
// Python function then goes its own way, which refuses the argument by name or
// converts it.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstdint>
#include <utility>
#include <vector>

#include "pkv.h"

namespace {

struct Unplain {};  // an argument for the Python function

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_CheckExact(o)) throw Unplain();
  return THPVariable_Unpack(o);
}

int32_t i32(int64_t v) {
  if (v < INT32_MIN || v > INT32_MAX) throw Unplain();
  return (int32_t)v;
}

int32_t integer(PyObject* o) {
  if (!PyLong_CheckExact(o)) throw Unplain();
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (over) throw Unplain();
  return i32(v);
}

float number(PyObject* o) {
  if (PyFloat_CheckExact(o)) return (float)PyFloat_AS_DOUBLE(o);
  return (float)integer(o);
}

pkv_dtype code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kHalf: return PKV_F16;
    case at::kBFloat16: return PKV_BF16;
    case at::kByte:
    case at::kFloat8_e4m3fn: return PKV_FP8_E4M3;
    default: throw Unplain();
  }
}

// Pointer of a contiguous tensor of this shape and dtype on this device.
void* data(PyObject* o, at::IntArrayRef shape, at::ScalarType dtype, int device) {
  const at::Tensor& t = tensor(o);
  if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != device ||
      t.scalar_type() != dtype || t.sizes() != shape || !t.is_contiguous())
    throw Unplain();
  return t.data_ptr();
}

template <typename T>
T* array(PyObject* o, at::IntArrayRef shape, int device) {
  return static_cast<T*>(data(o, shape, c10::CppTypeToScalarType<T>::value, device));
}

// What a call's pools hold: values with a scale per tensor (or none), codes with
// fp32 scales per block and head, or e2m1 codes with microscales.
enum Kind { PLAIN, SCALED, MX4 };

struct Pools {
  pkv_cache_desc desc;
  void *k, *v;
  int64_t blocks, heads, dim;
  int device;

  Pools(PyObject* ko, PyObject* vo, float k_scale, float v_scale, bool mx4 = false) {
    const at::Tensor& t = tensor(ko);
    if (t.dim() != 4 || !t.is_cuda()) throw Unplain();
    device = t.get_device();
    blocks = t.size(0);
    heads = t.size(1);
    dim = mx4 ? 2 * t.size(3) : t.size(3);
    if (mx4 && t.scalar_type() != at::kByte) throw Unplain();
    desc.num_blocks = i32(blocks);
    desc.block_size = i32(t.size(2));
    desc.num_kv_heads = i32(heads);
    desc.head_dim = i32(dim);
    desc.cache_dtype = mx4 ? PKV_MX4 : code(t);
    desc.k_scale = k_scale;
    desc.v_scale = v_scale;
    k = data(ko, t.sizes(), t.scalar_type(), device);
    v = data(vo, t.sizes(), t.scalar_type(), device);
    if (c10::cuda::current_device() != device) throw Unplain();
  }
  float* scales(PyObject* o) const { return array<float>(o, {blocks, heads}, device); }
  uint8_t* microscales(PyObject* o) const {
    return array<uint8_t>(o, {blocks, heads, desc.block_size, dim / 32}, device);
  }
};

// A pair of activation tensors [rows][heads][dim] of one 16-bit dtype.
struct Rows {
  void *a, *b;
  int64_t rows, heads;
  pkv_dtype dtype;

  Rows(PyObject* ao, PyObject* bo, const Pools& c, bool kv) {
    const at::Tensor& t = tensor(ao);
    if (t.dim() != 3) throw Unplain();
    rows = t.size(0);
    heads = kv ? c.heads : t.size(1);
    i32(rows);
    i32(heads);
    dtype = code(t);
    a = data(ao, {rows, heads, c.dim}, t.scalar_type(), c.device);
    b = data(bo, {rows, heads, c.dim}, t.scalar_type(), c.device);
  }
};

struct Table {
  int32_t* blocks;
  int64_t batch, width;

  Table(PyObject* o, int device) {
    const at::Tensor& t = tensor(o);
    if (t.dim() != 2) throw Unplain();
    batch = t.size(0);
    width = t.size(1);
    i32(batch);
    i32(width);
    blocks = array<int32_t>(o, {batch, width}, device);
  }
};

// Where the rows of each request lie: indptr [batch + 1], starts [batch].
struct Layout : Table {
  int32_t *indptr, *starts;

  Layout(PyObject* indptr_o, PyObject* starts_o, PyObject* table_o, int device)
      : Table(table_o, device) {
    indptr = array<int32_t>(indptr_o, {batch + 1}, device);
    starts = array<int32_t>(starts_o, {batch}, device);
  }
};

struct Workspace {
  void* at = nullptr;
  size_t bytes = 0;

  Workspace(PyObject* o, int device) {
    if (o == Py_None) return;
    const at::Tensor& t = tensor(o);
    at = data(o, t.sizes(), t.scalar_type(), device);
    bytes = t.nbytes();
  }
};

float* lse(PyObject* o, int64_t rows, int64_t heads, int device) {
  return o == Py_None ? nullptr : array<float>(o, {rows, heads}, device);
}

cudaStream_t stream(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw Unplain();
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) throw Unplain();
  return static_cast<cudaStream_t>(p);
}

// The ABI call itself runs without the interpreter's lock, as under ctypes.
template <typename F>
PyObject* call(Py_ssize_t got, Py_ssize_t want, F f) {
  if (got != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

template <typename F>
long unlocked(F f) {
  long st;
  Py_BEGIN_ALLOW_THREADS
  st = (long)f();
  Py_END_ALLOW_THREADS
  return st;
}

// k, v, k_scales, v_scales, k_new, v_new, q_indptr, prefix_lens, block_tables,
// max_suffix_len, stream
PyObject* append_block_scaled(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&] {
    const Pools c(a[0], a[1], 1.f, 1.f);
    float *ks = c.scales(a[2]), *vs = c.scales(a[3]);
    const Rows r(a[4], a[5], c, true);
    const Layout l(a[6], a[7], a[8], c.device);
    const int32_t longest = integer(a[9]);
    const cudaStream_t s = stream(a[10], c.device);
    return unlocked([&] {
      return pkv_kv_append_block_scaled(&c.desc, c.k, c.v, ks, vs, r.a, r.b, r.dtype, l.indptr,
                                        l.starts, l.blocks, (int32_t)l.width, (int32_t)l.batch,
                                        (int32_t)r.rows, longest, s);
    });
  });
}

// The same arguments, over microscaled codes.
PyObject* append_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&] {
    const Pools c(a[0], a[1], 1.f, 1.f, true);
    uint8_t *ks = c.microscales(a[2]), *vs = c.microscales(a[3]);
    const Rows r(a[4], a[5], c, true);
    const Layout l(a[6], a[7], a[8], c.device);
    const int32_t longest = integer(a[9]);
    const cudaStream_t s = stream(a[10], c.device);
    return unlocked([&] {
      return pkv_kv_append_mx4(&c.desc, c.k, c.v, ks, vs, r.a, r.b, r.dtype, l.indptr, l.starts,
                               l.blocks, (int32_t)l.width, (int32_t)l.batch, (int32_t)r.rows, longest, s);
    });
  });
}

// k, v, k_scales, v_scales, k_out, v_out, row_indptr, start_positions,
// block_tables, stream
PyObject* gather_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&] {
    const Pools c(a[0], a[1], 1.f, 1.f, true);
    const uint8_t *ks = c.microscales(a[2]), *vs = c.microscales(a[3]);
    const Rows r(a[4], a[5], c, true);
    const Layout l(a[6], a[7], a[8], c.device);
    const cudaStream_t s = stream(a[9], c.device);
    return unlocked([&] {
      return pkv_kv_gather_mx4(&c.desc, c.k, c.v, ks, vs, r.a, r.b, r.dtype, l.indptr, l.starts,
                               l.blocks, (int32_t)l.width, (int32_t)l.batch, (int32_t)r.rows, s);
    });
  });
}

// tuple of pools -> (bytes of their pkv_pool structs, the bytes' address, device), or
// None (64 pools: 120 us when read from Python).
PyObject* pools(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 1 || !PyTuple_CheckExact(a[0])) Py_RETURN_NONE;
  const Py_ssize_t count = PyTuple_GET_SIZE(a[0]);
  try {
    std::vector<pkv_pool> got((size_t)count);
    std::vector<std::pair<uintptr_t, uintptr_t>> spans((size_t)count);
    int device = -1;
    for (Py_ssize_t i = 0; i < count; ++i) {
      const at::Tensor& t = tensor(PyTuple_GET_ITEM(a[0], i));
      if (t.layout() != at::kStrided || t.dim() < 2 || !t.is_cuda() || !t.is_contiguous()) throw Unplain();
      if (i == 0) device = t.get_device();
      int64_t row = (int64_t)t.element_size();
      for (int64_t d = 3; d < t.dim(); ++d) row = i32(row * i32(t.size(d)));
      pkv_pool& q = got[(size_t)i];
      q.base = t.data_ptr();
      q.num_blocks = i32(t.size(0));
      q.num_kv_heads = i32(t.size(1));
      q.block_size = t.dim() > 2 ? i32(t.size(2)) : 1;
      q.row_bytes = i32(row);
      if (t.get_device() != device || q.num_blocks != got[0].num_blocks || q.num_blocks <= 0 ||
          q.num_kv_heads <= 0 || q.block_size <= 0 || q.row_bytes <= 0)
        throw Unplain();
      spans[(size_t)i] = {(uintptr_t)q.base, (uintptr_t)q.base + (uintptr_t)t.nbytes()};
    }
    std::sort(spans.begin(), spans.end());
    for (size_t i = 1; i < spans.size(); ++i)
      if (spans[i - 1].second > spans[i].first) throw Unplain();
    PyObject* bytes = PyBytes_FromStringAndSize(reinterpret_cast<const char*>(got.data()),
                                                (Py_ssize_t)(got.size() * sizeof(pkv_pool)));
    if (!bytes) return nullptr;
    return Py_BuildValue("(NNi)", bytes, PyLong_FromVoidPtr(PyBytes_AS_STRING(bytes)), device);
  } catch (...) {  // what the Python way refuses by name, or converts
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// The pools of a KvPools: the address and number of its pkv_pool structs.
struct PoolSet {
  const pkv_pool* at;
  int32_t count;

  PoolSet(PyObject* address, PyObject* count_o) {
    if (!PyLong_CheckExact(address)) throw Unplain();
    at = static_cast<const pkv_pool*>(PyLong_AsVoidPtr(address));
    if (PyErr_Occurred()) throw Unplain();
    count = integer(count_o);
  }
};

int device_of(PyObject* o) {
  const int d = integer(o);
  if (d < 0 || c10::cuda::current_device() != d) throw Unplain();
  return d;
}

int64_t length(PyObject* o) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != 1) throw Unplain();
  return i32(t.size(0));
}

// pools, count, device, src_blocks, dst_blocks, stream
PyObject* copy_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 6, [&] {
    const PoolSet p(a[0], a[1]);
    const int device = device_of(a[2]);
    const int64_t pairs = length(a[3]);
    const int32_t *src = array<int32_t>(a[3], {pairs}, device), *dst = array<int32_t>(a[4], {pairs}, device);
    const cudaStream_t s = stream(a[5], device);
    return unlocked([&] { return pkv_kv_copy_blocks(p.at, p.count, src, dst, (int32_t)pairs, s); });
  });
}

// pools, count, device, src_positions, row_indptr, dst_starts, block_tables,
// max_rows, stream
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const PoolSet p(a[0], a[1]);
    const int device = device_of(a[2]);
    const int64_t rows = length(a[3]);
    const int32_t* src = array<int32_t>(a[3], {rows}, device);
    const Layout l(a[4], a[5], a[6], device);
    const int32_t most = integer(a[7]);
    const cudaStream_t s = stream(a[8], device);
    return unlocked([&] {
      return pkv_kv_compact(p.at, p.count, src, l.indptr, l.starts, l.blocks, (int32_t)l.width,
                            (int32_t)l.batch, (int32_t)rows, most, s);
    });
  });
}

// k, v, k_out, v_out, row_indptr, start_positions, block_tables, k_scale, v_scale,
// k_scales, v_scales, stream
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 12, [&] {
    const Pools c(a[0], a[1], number(a[7]), number(a[8]));
    const bool scaled = a[9] != Py_None;
    if (!scaled && a[10] != Py_None) throw Unplain();
    const float* ks = scaled ? c.scales(a[9]) : nullptr;
    const float* vs = scaled ? c.scales(a[10]) : nullptr;
    const Rows r(a[2], a[3], c, true);
    const Layout l(a[4], a[5], a[6], c.device);
    const cudaStream_t s = stream(a[11], c.device);
    return unlocked([&] {
      return pkv_kv_gather(&c.desc, c.k, c.v, ks, vs, r.a, r.b, r.dtype, l.indptr, l.starts,
                           l.blocks, (int32_t)l.width, (int32_t)l.batch, (int32_t)r.rows, s);
    });
  });
}

// k, v, then k_scales, v_scales (SCALED, MX4) or k_scale, v_scale; q, out, block_tables,
// seq_lens, sm_scale, max_seq_len, window, sink_tokens, num_splits, lse_out,
// workspace, stream
template <Kind K>
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 16, [&] {
    const Pools c(a[0], a[1], K != PLAIN ? 1.f : number(a[2]), K != PLAIN ? 1.f : number(a[3]), K == MX4);
    const float* ks = K == SCALED ? c.scales(a[2]) : nullptr;
    const float* vs = K == SCALED ? c.scales(a[3]) : nullptr;
    const uint8_t* km = K == MX4 ? c.microscales(a[2]) : nullptr;
    const uint8_t* vm = K == MX4 ? c.microscales(a[3]) : nullptr;
    const Rows r(a[4], a[5], c, false);
    const Table t(a[6], c.device);
    if (t.batch != r.rows) throw Unplain();
    const int32_t* lens = array<int32_t>(a[7], {r.rows}, c.device);
    const float sm_scale = number(a[8]);
    const int32_t longest = integer(a[9]), window = integer(a[10]), sinks = integer(a[11]);
    const int32_t splits = integer(a[12]);
    float* l = lse(a[13], r.rows, r.heads, c.device);
    const Workspace w(a[14], c.device);
    const cudaStream_t s = stream(a[15], c.device);
    const int32_t width = (int32_t)t.width, batch = (int32_t)r.rows, heads = (int32_t)r.heads;
    return unlocked([&] {
      if constexpr (K == MX4)
        return pkv_paged_decode_attn_mx4(&c.desc, c.k, c.v, km, vm, r.a, r.b, r.dtype, t.blocks, width,
                                         lens, batch, heads, sm_scale, longest, window, sinks, splits,
                                         l, w.at, w.bytes, s);
      else if constexpr (K == SCALED)
        return pkv_paged_decode_attn_block_scaled(&c.desc, c.k, c.v, ks, vs, r.a, r.b, r.dtype,
                                                  t.blocks, width, lens, batch, heads, sm_scale,
                                                  longest, window, sinks, splits, l, w.at, w.bytes,
                                                  s);
      else
        return pkv_paged_decode_attn_window(&c.desc, c.k, c.v, r.a, r.b, r.dtype, t.blocks, width,
                                            lens, batch, heads, sm_scale, longest, window, sinks,
                                            splits, l, w.at, w.bytes, s);
    });
  });
}

// k, v, then k_scales, v_scales (SCALED, MX4) or k_scale, v_scale; q, out, q_indptr,
// prefix_lens, block_tables, sm_scale, max_suffix_len, max_total_len, window,
// sink_tokens, lse_out, workspace, stream
template <Kind K>
PyObject* extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 17, [&] {
    const Pools c(a[0], a[1], K != PLAIN ? 1.f : number(a[2]), K != PLAIN ? 1.f : number(a[3]), K == MX4);
    const float* ks = K == SCALED ? c.scales(a[2]) : nullptr;
    const float* vs = K == SCALED ? c.scales(a[3]) : nullptr;
    const uint8_t* km = K == MX4 ? c.microscales(a[2]) : nullptr;
    const uint8_t* vm = K == MX4 ? c.microscales(a[3]) : nullptr;
    const Rows r(a[4], a[5], c, false);
    const Layout y(a[6], a[7], a[8], c.device);
    const float sm_scale = number(a[9]);
    const int32_t suffix = integer(a[10]), total = integer(a[11]);
    const int32_t window = integer(a[12]), sinks = integer(a[13]);
    float* l = lse(a[14], r.rows, r.heads, c.device);
    const Workspace w(a[15], c.device);
    const cudaStream_t s = stream(a[16], c.device);
    const int32_t width = (int32_t)y.width, batch = (int32_t)y.batch, rows = (int32_t)r.rows;
    const int32_t heads = (int32_t)r.heads;
    return unlocked([&] {
      if constexpr (K == MX4)
        return pkv_paged_extend_attn_mx4(&c.desc, c.k, c.v, km, vm, r.a, r.b, r.dtype, y.indptr,
                                         y.starts, y.blocks, width, batch, heads, sm_scale, rows,
                                         suffix, total, window, sinks, l, w.at, w.bytes, s);
      else if constexpr (K == SCALED)
        return pkv_paged_extend_attn_block_scaled(&c.desc, c.k, c.v, ks, vs, r.a, r.b, r.dtype,
                                                  y.indptr, y.starts, y.blocks, width, batch, heads,
                                                  sm_scale, rows, suffix, total, window, sinks, l,
                                                  w.at, w.bytes, s);
      else
        return pkv_paged_extend_attn_window(&c.desc, c.k, c.v, r.a, r.b, r.dtype, y.indptr,
                                            y.starts, y.blocks, width, batch, heads, sm_scale, rows,
                                            suffix, total, window, sinks, l, w.at, w.bytes, s);
    });
  });
}

#define FN(name, f) \
  { name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FN("append_block_scaled", append_block_scaled),
                         FN("gather", gather),
                         FN("decode_window", decode<PLAIN>),
                         FN("decode_block_scaled", decode<SCALED>),
                         FN("extend_window", extend<PLAIN>),
                         FN("extend_block_scaled", extend<SCALED>),
                         FN("append_mx4", append_mx4),
                         FN("gather_mx4", gather_mx4),
                         FN("decode_mx4", decode<MX4>),
                         FN("extend_mx4", extend<MX4>),
                         FN("pools", pools),
                         FN("copy_blocks", copy_blocks),
                         FN("compact", compact),
                         {nullptr, nullptr, 0, nullptr}};
#undef FN

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers this was compiled with
PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", PKV_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
