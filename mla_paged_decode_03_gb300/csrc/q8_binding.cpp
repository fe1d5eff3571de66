// Python binding of the calls of the 8-bit cache and of prompt processing: argument checks, outputs,
// the current stream, and the C ABI's functions (handed over by address, so that the library is
// loaded in one place).
//
// A small step's kernels take 3 to 12 us; with checks and allocations in Python and a ctypes
// call, calls back to back took 26 us (cp_step_tables), 9 us (cp_store_q8) and 26 us
// (mla_decode_q8 of two short requests); through this they take 8, 5 and 12.5 us.  Only the
// marshalling is here: what a call means, and every check of sizes, is the C ABI's.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/CUDAContextLight.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cstdarg>
#include <optional>
#include <string>

#include "../../include/mla_decode.h"

namespace {

constexpr int64_t kDqk = 576, kDv = 512;

// The library's functions, the check that raises the error of a code, and the result type of
// step_tables (a subclass of tuple).
struct {
  decltype(&cp_step_tables) step_tables = nullptr;
  decltype(&cp_store_q8) store = nullptr;
  decltype(&mla_decode_q8) decode = nullptr;
  decltype(&mla_decode_shards_q8) decode_shards = nullptr;
  decltype(&mla_decode_q8_workspace_size) workspace_size = nullptr;
  decltype(&mla_rope) rope = nullptr;
  decltype(&cp_rope_store) rope_store = nullptr;
  decltype(&mla_expand) expand = nullptr;
  decltype(&mla_prefill) prefill = nullptr;
  decltype(&mla_prefill_workspace_size) prefill_workspace_size = nullptr;
  PyObject* check = nullptr;
  PyTypeObject* tables_type = nullptr;
} g;

// Thrown with a Python error set.
struct Raised {};

[[noreturn]] void refuse(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Raised();
}

std::string text(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

int as_int(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT_MIN || v > INT_MAX) refuse(PyExc_ValueError, "%s = %ld does not fit 32 bits", name, v);
  return (int)v;
}
bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}
float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return (float)v;
}

const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  return t;
}
void here(const at::Tensor& t, const char* name, int dev) {
  if (t.get_device() != dev)
    refuse(PyExc_ValueError, "%s is on cuda:%d, not on the current device cuda:%d", name, (int)t.get_device(), dev);
}
// A contiguous tensor of `dims` dimensions on the current device.
const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type, int64_t dims, int dev) {
  const at::Tensor& t = tensor(o, name, type);
  if (t.dim() != dims)
    refuse(PyExc_ValueError, "%s must have %d dims, got %s", name, (int)dims, text(t.sizes()).c_str());
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  here(t, name, dev);
  return t;
}
// The address of a contiguous tensor of this shape on the current device.
template <class T>
T* address(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  const at::Tensor& t = tensor(o, name, type);
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, "%s must be %s, got %s", name, text(shape).c_str(), text(t.sizes()).c_str());
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  here(t, name, dev);
  return static_cast<T*>(t.data_ptr());
}

at::Tensor made(at::ScalarType type, at::IntArrayRef shape, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
}

// New outputs of one type in one allocation (an allocation and its release take 1.4 us, a tensor
// on part of a storage 0.4): the sizes of those that the caller did not give are added up first.
struct Pool {
  at::ScalarType type;
  int64_t elements = 0, used = 0;
  at::Tensor base;
  void need(PyObject* given, int64_t n) {
    if (given == Py_None) elements += n;
  }
  at::Tensor take(at::IntArrayRef shape, int dev) {
    if (!base.defined()) base = made(type, {elements}, dev);
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), base.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(used);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    used += t.numel();
    return t;
  }
};

// An output: the caller's tensor, checked, or a new one.
struct Output {
  PyObject* obj = nullptr;                 // owned
  void* ptr = nullptr;
  Output(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev, Pool* pool = nullptr) {
    if (o != Py_None) {
      ptr = address<void>(o, name, type, shape, dev);
      obj = Py_NewRef(o);
      return;
    }
    at::Tensor t = pool != nullptr ? pool->take(shape, dev) : made(type, shape, dev);
    ptr = t.data_ptr();
    obj = THPVariable_Wrap(std::move(t));
    if (obj == nullptr) throw Raised();
  }
  Output(const Output&) = delete;
  ~Output() { Py_XDECREF(obj); }
  PyObject* release() {
    PyObject* o = obj;
    obj = nullptr;
    return o;
  }
};

struct Table {
  int32_t* ptr;
  int64_t stride;
  int columns;
};
// A block table of contiguous rows (a single row's stride is its width at least).
Table block_table(PyObject* o, int64_t rows, int dev) {
  const at::Tensor& t = tensor(o, "block_table", at::kInt);
  if (t.dim() != 2) refuse(PyExc_TypeError, "block_table must be a 2-D int32 CUDA tensor");
  const int64_t n = t.size(0), width = t.size(1);
  if (n != rows || (width > 1 && t.stride(1) != 1) || width > INT_MAX)
    refuse(PyExc_ValueError, "block_table must be [%lld, max_blocks] with contiguous rows, got %s with strides %s",
          (long long)rows, text(t.sizes()).c_str(), text(t.strides()).c_str());
  here(t, "block_table", dev);
  const int64_t stride = t.stride(0);
  return {static_cast<int32_t*>(t.data_ptr()), rows <= 1 && stride < width ? width : stride, (int)width};
}

struct Cache {
  void* rows;
  float* scales;
  int num_blocks, block_size;
};
Cache cache(PyObject* kv, PyObject* scales, int dev) {
  const at::Tensor& t = dense(kv, "kv_cache", at::kFloat8_e4m3fn, 3, dev);
  const int64_t nb = t.size(0), bs = t.size(1);
  if (t.size(2) != kDqk || bs % MLA_Q8_GROUP || nb > INT_MAX || bs > INT_MAX)
    refuse(PyExc_ValueError,
          "kv_cache must be [num_blocks, block_size, %d] with block_size a multiple of %d, got %s", (int)kDqk,
          MLA_Q8_GROUP, text(t.sizes()).c_str());
  return {t.data_ptr(), address<float>(scales, "kv_scales", at::kFloat, {nb, bs / MLA_Q8_GROUP}, dev), (int)nb,
          (int)bs};
}

int small(int64_t v, const char* name) {
  if (v > INT_MAX) refuse(PyExc_ValueError, "%s = %lld does not fit 32 bits", name, (long long)v);
  return (int)v;
}

mla_stream_t stream(int dev) {
  return reinterpret_cast<mla_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}

// Raises the library's error of a failed call.
void check(int rc) {
  if (rc == MLA_OK) return;
  PyObject* r = PyObject_CallFunction(g.check, "i", rc);
  if (r != nullptr) {
    Py_DECREF(r);
    refuse(PyExc_RuntimeError, "error code %d", rc);
  }
  throw Raised();
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "%zd arguments, not %zd", n, want);
  if (g.check == nullptr) refuse(PyExc_RuntimeError, "the library has not been bound");
}

// bind(step_tables, store, decode, decode_shards, workspace_size, abi_version, check, tables_type);
// refuses a library that was built with another ABI than this binding
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != 8) refuse(PyExc_TypeError, "%zd arguments, not 8", n);
    void* f[6];
    for (int i = 0; i < 6; ++i) {
      f[i] = PyLong_AsVoidPtr(a[i]);
      if (f[i] == nullptr) refuse(PyExc_ValueError, "no address of function %d", i);
    }
    if (!PyType_Check(a[7]) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(a[7]), &PyTuple_Type))
      refuse(PyExc_TypeError, "the result type must be a tuple");
    const int abi = reinterpret_cast<decltype(&mla_abi_version)>(f[5])();
    if (abi != MLA_ABI_VERSION)
      refuse(PyExc_ImportError, "the library has ABI version %d.%d, the binding was built for %d.%d: build both again",
             abi >> 16, abi & 0xffff, MLA_ABI_VERSION >> 16, MLA_ABI_VERSION & 0xffff);
    g.step_tables = reinterpret_cast<decltype(g.step_tables)>(f[0]);
    g.store = reinterpret_cast<decltype(g.store)>(f[1]);
    g.decode = reinterpret_cast<decltype(g.decode)>(f[2]);
    g.decode_shards = reinterpret_cast<decltype(g.decode_shards)>(f[3]);
    g.workspace_size = reinterpret_cast<decltype(g.workspace_size)>(f[4]);
    Py_XSETREF(g.check, Py_NewRef(a[6]));
    PyTypeObject* old = g.tables_type;
    g.tables_type = reinterpret_cast<PyTypeObject*>(Py_NewRef(a[7]));
    Py_XDECREF(reinterpret_cast<PyObject*>(old));
    Py_RETURN_NONE;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// step_tables(prev_lens, ctx_lens, new_lens, block_table, free_pages, free_state, block_size, N, cp_size,
//             cp_rank, n_ranks, interleave, total_lens, seq_lens, positions, slots, free_state_out)
PyObject* step_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 17);
    const at::Tensor& first = tensor(a[0], "prev_lens", at::kInt);
    if (first.dim() != 1) refuse(PyExc_TypeError, "prev_lens must be a 1-D int32 CUDA tensor");
    const int dev = c10::cuda::current_device();
    const int64_t B = first.size(0);
    const auto *prev = address<int32_t>(a[0], "prev_lens", at::kInt, {B}, dev),
               *ctx = address<int32_t>(a[1], "ctx_lens", at::kInt, {B}, dev),
               *fresh = address<int32_t>(a[2], "new_lens", at::kInt, {B}, dev);
    const Table table = block_table(a[3], B, dev);
    const at::Tensor& ring = dense(a[4], "free_pages", at::kInt, 1, dev);
    const auto* state = address<int32_t>(a[5], "free_state", at::kInt, {2}, dev);
    const int bs = as_int(a[6], "block_size"), N = as_int(a[7], "N"), cp = as_int(a[8], "cp_size"),
              rank = as_int(a[9], "cp_rank"), ranks = as_int(a[10], "n_ranks"), il = as_int(a[11], "interleave");
    if (ranks < 1 || N < 0) refuse(PyExc_ValueError, "need n_ranks >= 1 and N >= 0, got %d and %d", ranks, N);
    if (B > INT_MAX / ranks || (N > 0 && B > INT_MAX / ranks / N))
      refuse(PyExc_ValueError, "n_ranks * B * N = %d * %lld * %d does not fit 32 bits", ranks, (long long)B, N);
    Pool i32{at::kInt}, i64{at::kLong};
    i32.need(a[12], B);
    i32.need(a[13], ranks * B);
    i32.need(a[16], 2);
    i64.need(a[14], B * N);
    i64.need(a[15], ranks * B * N);
    Output total(a[12], "total_lens", at::kInt, {B}, dev, &i32);
    Output seq(a[13], "seq_lens", at::kInt, {ranks, B}, dev, &i32);
    Output positions(a[14], "positions", at::kLong, {B, N}, dev, &i64);
    Output slots(a[15], "slots", at::kLong, {ranks, B, N}, dev, &i64);
    Output state_out(a[16], "free_state_out", at::kInt, {2}, dev, &i32);
    const int cap = small(ring.size(0), "free_pages' length");
    const mla_stream_t s = stream(dev);
    auto* pages = static_cast<int32_t*>(ring.data_ptr());
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g.step_tables(prev, ctx, fresh, (int)B, N, table.ptr, table.stride, table.columns, pages, cap, state,
                       static_cast<int32_t*>(state_out.ptr), bs, cp, rank, ranks, il,
                       static_cast<int32_t*>(total.ptr), static_cast<int32_t*>(seq.ptr),
                       static_cast<int64_t*>(positions.ptr), static_cast<int64_t*>(slots.ptr), s);
    Py_END_ALLOW_THREADS
    check(rc);
    // StepTables is a tuple in this order
    PyObject* made = g.tables_type->tp_alloc(g.tables_type, 5);
    if (made == nullptr) return nullptr;
    PyTuple_SET_ITEM(made, 0, total.release());
    PyTuple_SET_ITEM(made, 1, seq.release());
    PyTuple_SET_ITEM(made, 2, positions.release());
    PyTuple_SET_ITEM(made, 3, slots.release());
    PyTuple_SET_ITEM(made, 4, state_out.release());
    return made;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// store(kv_new, ctx_lens, total_lens, block_table, kv_cache, kv_scales, cp_size, cp_rank, interleave)
PyObject* store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 9);
    tensor(a[0], "kv_new", at::kBFloat16);
    const int dev = c10::cuda::current_device();
    const at::Tensor& rows = dense(a[0], "kv_new", at::kBFloat16, 3, dev);
    const int64_t B = rows.size(0);
    if (rows.size(2) != kDqk)
      refuse(PyExc_ValueError, "kv_new must be [B, N, %d], got %s", (int)kDqk, text(rows.sizes()).c_str());
    const Table table = block_table(a[3], B, dev);
    const Cache c = cache(a[4], a[5], dev);
    const auto *ctx = address<int32_t>(a[1], "ctx_lens", at::kInt, {B}, dev),
               *total = address<int32_t>(a[2], "total_lens", at::kInt, {B}, dev);
    const int b = small(B, "B"), N = small(rows.size(1), "N"), cp = as_int(a[6], "cp_size"),
              rank = as_int(a[7], "cp_rank"), il = as_int(a[8], "interleave");
    const void* src = rows.data_ptr();
    const mla_stream_t s = stream(dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g.store(src, ctx, total, table.ptr, table.stride, table.columns, b, N, c.block_size, cp, rank, il, c.rows,
                 c.scales, c.num_blocks, s);
    Py_END_ALLOW_THREADS
    check(rc);
    return PyTuple_Pack(2, a[4], a[5]);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// decode(n_shards or None, q, kv_cache, kv_scales, block_table, seq_lens, causal_seqlens_global, q_len,
//        cp_world, cp_rank, scale, out, lse, lse_base_e, workspace, return_lse, causal, interleave)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 18);
    const bool sharded = a[0] != Py_None;
    const int64_t shards = sharded ? as_int(a[0], "n_shards") : 1;
    if (shards < 1) refuse(PyExc_ValueError, "need n_shards >= 1, got %lld", (long long)shards);
    const at::Tensor& q = tensor(a[1], "q", at::kBFloat16);
    const int dev = c10::cuda::current_device();
    const int q_len = as_int(a[7], "q_len");
    // [B, q_len, H, 576] or [B * q_len, H, 576]
    const bool flat = q.dim() == 3;
    if ((!flat && q.dim() != 4) || q.size(-1) != kDqk || q_len < 1 ||
        (flat ? q.size(0) % q_len != 0 : q.size(1) != q_len))
      refuse(PyExc_ValueError, "q must be [B, q_len=%d, H, %d] or [B*q_len, H, %d], got %s", q_len, (int)kDqk,
            (int)kDqk, text(q.sizes()).c_str());
    dense(a[1], "q", at::kBFloat16, q.dim(), dev);
    const int64_t B = flat ? q.size(0) / q_len : q.size(0), H = q.size(-2);
    const Cache c = cache(a[2], a[3], dev);
    const Table table = block_table(a[4], shards * B, dev);
    const auto* seq = address<int32_t>(a[5], "seq_lens", at::kInt, {shards * B}, dev);
    const int32_t* global =
        a[6] == Py_None ? nullptr : address<int32_t>(a[6], "causal_seqlens_global", at::kInt, {B}, dev);
    const int b = small(shards * B, "n_shards * B") / (int)shards, h = small(H, "H");
    const int cp = sharded ? 0 : as_int(a[8], "cp_world"), rank = sharded ? 0 : as_int(a[9], "cp_rank"),
              il = as_int(a[17], "interleave");
    const float scale = as_float(a[10]);
    const bool base_e = as_bool(a[13]), causal = as_bool(a[16]);
    int64_t shape[4] = {shards, B * q_len, H, kDv};
    const at::IntArrayRef out_shape(shape + (sharded ? 0 : 1), sharded ? 4 : 3);
    Output out(a[11], "out", at::kBFloat16, out_shape, dev);
    const bool with_lse = a[12] != Py_None || as_bool(a[15]);
    std::optional<Output> lse;
    if (with_lse) lse.emplace(a[12], "lse", at::kFloat, out_shape.slice(0, out_shape.size() - 1), dev);
    at::Tensor scratch;
    if (a[14] == Py_None) {
      const size_t bytes = g.workspace_size((int)(shards * B), h, q_len,
                                            at::cuda::getDeviceProperties((c10::DeviceIndex)dev)->multiProcessorCount);
      scratch = made(at::kByte, {(int64_t)bytes}, dev);
    } else {
      if (!THPVariable_Check(a[14])) refuse(PyExc_TypeError, "workspace must be a torch.Tensor");
      scratch = THPVariable_Unpack(a[14]);
      if (!scratch.is_cuda()) refuse(PyExc_ValueError, "workspace must be a CUDA tensor");
      if (!scratch.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
      here(scratch, "workspace", dev);
    }
    const void* src = q.data_ptr();
    void *ws = scratch.data_ptr(), *o = out.ptr;
    float* l = with_lse ? static_cast<float*>(lse->ptr) : nullptr;
    const size_t ws_bytes = scratch.nbytes();
    const mla_stream_t s = stream(dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = sharded ? g.decode_shards(src, c.rows, c.scales, table.ptr, table.stride, seq, global, b, h, q_len, causal,
                                   c.block_size, c.num_blocks, table.columns, (int)shards, il, scale, o, l, base_e,
                                   ws, ws_bytes, s)
                 : g.decode(src, c.rows, c.scales, table.ptr, table.stride, seq, global, b, h, q_len, causal,
                            c.block_size, c.num_blocks, table.columns, cp, rank, il, scale, o, l, base_e, ws,
                            ws_bytes, s);
    Py_END_ALLOW_THREADS
    check(rc);
    return PyTuple_Pack(2, out.obj, with_lse ? lse->obj : Py_None);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// ---- prompt processing ---------------------------------------------------------------------

// bind_prompt(rope, rope_store, expand, prefill, prefill_workspace_size), after bind
PyObject* bind_prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, 5);
    void* f[5];
    for (int i = 0; i < 5; ++i) {
      f[i] = PyLong_AsVoidPtr(a[i]);
      if (f[i] == nullptr) refuse(PyExc_ValueError, "no address of function %d", i);
    }
    g.rope = reinterpret_cast<decltype(g.rope)>(f[0]);
    g.rope_store = reinterpret_cast<decltype(g.rope_store)>(f[1]);
    g.expand = reinterpret_cast<decltype(g.expand)>(f[2]);
    g.prefill = reinterpret_cast<decltype(g.prefill)>(f[3]);
    g.prefill_workspace_size = reinterpret_cast<decltype(g.prefill_workspace_size)>(f[4]);
    Py_RETURN_NONE;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
void prompt_arguments(Py_ssize_t n, Py_ssize_t want) {
  arguments(n, want);
  if (g.prefill == nullptr) refuse(PyExc_RuntimeError, "the library has not been bound");
}

// Rows of `width` contiguous bf16 values, T tokens (or B x N, taken as one row of tokens) of H heads.
struct Rows {
  void* ptr;
  int64_t T, H, stride_t, stride_h;
};
Rows rows_of(const at::Tensor& t, const char* name, int64_t width, bool heads, int dev) {
  const int64_t dims = t.dim(), lead = dims - (heads ? 2 : 1);
  if (lead < 1 || lead > 2 || t.size(dims - 1) != width)
    refuse(PyExc_ValueError, "%s must be [T, %s%d] or [B, N, %s%d], got %s", name, heads ? "H, " : "", (int)width,
           heads ? "H, " : "", (int)width, text(t.sizes()).c_str());
  here(t, name, dev);
  Rows r;
  r.ptr = t.data_ptr();
  r.T = lead == 2 ? t.size(0) * t.size(1) : t.size(0);
  r.H = heads ? t.size(dims - 2) : 1;
  if (t.stride(dims - 1) != 1)
    refuse(PyExc_ValueError, "%s's last dimension must be contiguous, its strides are %s", name, text(t.strides()).c_str());
  r.stride_h = heads && r.H > 1 ? t.stride(dims - 2) : width;
  // two leading dimensions have to step as one
  if (lead == 2 && t.size(0) > 1 && t.size(1) > 1 && t.stride(0) != t.size(1) * t.stride(1))
    refuse(PyExc_ValueError, "%s's first two dimensions must step as one, its strides are %s", name,
           text(t.strides()).c_str());
  const int64_t step = lead == 2 && t.size(1) > 1 ? t.stride(1) : t.stride(0);
  r.stride_t = r.T > 1 ? step : width * r.H;
  if (r.stride_h % 8 || r.stride_t % 8 || reinterpret_cast<uintptr_t>(r.ptr) % 16)
    refuse(PyExc_ValueError, "%s must start on 16 bytes and step by multiples of 8 values, its strides are %s", name,
           text(t.strides()).c_str());
  return r;
}

const int64_t* freqs_of(PyObject* o, int dev) { return address<int64_t>(o, "freqs", at::kLong, {32}, dev); }

// rope(x, positions, freqs, out, half, mscale)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    prompt_arguments(n, 6);
    const at::Tensor& x = tensor(a[0], "x", at::kBFloat16);
    const int dev = c10::cuda::current_device();
    const Rows r = rows_of(x, "x", 64, true, dev);
    const auto* pos = address<int64_t>(a[1], "positions", at::kLong, x.sizes().slice(0, x.dim() - 2), dev);
    const int64_t* freqs = freqs_of(a[2], dev);
    const bool half = as_bool(a[4]);
    const float mscale = as_float(a[5]);
    const int T = small(r.T, "T"), H = small(r.H, "H");
    at::Tensor made_out;
    if (a[3] == Py_None) {
      made_out = made(at::kBFloat16, x.sizes(), dev);
    } else {
      made_out = tensor(a[3], "out", at::kBFloat16);
      if (made_out.sizes() != x.sizes())
        refuse(PyExc_ValueError, "out must be %s, got %s", text(x.sizes()).c_str(), text(made_out.sizes()).c_str());
    }
    const Rows o = rows_of(made_out, "out", 64, true, dev);
    const mla_stream_t s = stream(dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g.rope(r.ptr, r.stride_t, r.stride_h, pos, freqs, T, H, half, mscale, o.ptr, o.stride_t, o.stride_h, s);
    Py_END_ALLOW_THREADS
    check(rc);
    return a[3] == Py_None ? THPVariable_Wrap(std::move(made_out)) : Py_NewRef(a[3]);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// rope_store(latent, k_rope, positions, freqs, block_table, kv_cache, cp_size, cp_rank, interleave, half, mscale, slots)
PyObject* rope_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    prompt_arguments(n, 12);
    const at::Tensor& latent = tensor(a[0], "latent", at::kBFloat16);
    const at::Tensor& k_rope = tensor(a[1], "k_rope", at::kBFloat16);
    const int dev = c10::cuda::current_device();
    if (latent.dim() != 3 || k_rope.dim() != 3 || latent.size(0) != k_rope.size(0) || latent.size(1) != k_rope.size(1))
      refuse(PyExc_ValueError, "latent and k_rope must be [B, N, 512] and [B, N, 64], got %s and %s",
             text(latent.sizes()).c_str(), text(k_rope.sizes()).c_str());
    const int64_t B = latent.size(0), N = latent.size(1);
    const Rows c = rows_of(latent, "latent", kDv, false, dev), r = rows_of(k_rope, "k_rope", 64, false, dev);
    const auto* pos = address<int64_t>(a[2], "positions", at::kLong, {B, N}, dev);
    const int64_t* freqs = freqs_of(a[3], dev);
    const Table table = block_table(a[4], B, dev);
    const at::Tensor& kv = dense(a[5], "kv_cache", at::kBFloat16, 3, dev);
    if (kv.size(2) != kDqk)
      refuse(PyExc_ValueError, "kv_cache must be [num_blocks, block_size, %d], got %s", (int)kDqk, text(kv.sizes()).c_str());
    const int nb = small(kv.size(0), "num_blocks"), bs = small(kv.size(1), "block_size"), b = small(B, "B"), nn = small(N, "N");
    const int cp = as_int(a[6], "cp_size"), rank = as_int(a[7], "cp_rank"), il = as_int(a[8], "interleave");
    const bool half = as_bool(a[9]);
    const float mscale = as_float(a[10]);
    int64_t* slots = a[11] == Py_None ? nullptr : address<int64_t>(a[11], "slots", at::kLong, {B, N}, dev);
    void* pages = kv.data_ptr();
    const mla_stream_t s = stream(dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g.rope_store(c.ptr, c.stride_t, r.ptr, r.stride_t, pos, freqs, table.ptr, table.stride, table.columns, b, nn, bs,
                      cp, rank, il, half, mscale, pages, nb, slots, s);
    Py_END_ALLOW_THREADS
    check(rc);
    return Py_NewRef(a[5]);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// A part of kv [H, S, 256] as [S, H, 128].
at::Tensor half_head(const at::Tensor& kv, int64_t S, int64_t H, int64_t from) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(kv.storage()), kv.key_set(), kv.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(kv.storage_offset() + from);
  t.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef({S, H, 128}), at::IntArrayRef({256, S * 256, 1}));
  return t;
}

// expand(kv_cache, kv_scales, block_table, seq_lens, kv_starts, w_kv, S, kv, k_rope)
PyObject* expand(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    prompt_arguments(n, 9);
    const bool q8 = a[1] != Py_None;
    tensor(a[0], "kv_cache", q8 ? at::kFloat8_e4m3fn : at::kBFloat16);
    const int dev = c10::cuda::current_device();
    Cache c;
    if (q8) {
      c = cache(a[0], a[1], dev);
    } else {
      const at::Tensor& t = dense(a[0], "kv_cache", at::kBFloat16, 3, dev);
      if (t.size(2) != kDqk)
        refuse(PyExc_ValueError, "kv_cache must be [num_blocks, block_size, %d], got %s", (int)kDqk, text(t.sizes()).c_str());
      c = {t.data_ptr(), nullptr, small(t.size(0), "num_blocks"), small(t.size(1), "block_size")};
    }
    const at::Tensor& lens = tensor(a[3], "seq_lens", at::kInt);
    if (lens.dim() != 1) refuse(PyExc_ValueError, "seq_lens must be [B], got %s", text(lens.sizes()).c_str());
    const int64_t B = lens.size(0);
    const auto *seq = address<int32_t>(a[3], "seq_lens", at::kInt, {B}, dev),
               *starts = address<int32_t>(a[4], "kv_starts", at::kInt, {B}, dev);
    const Table table = block_table(a[2], B, dev);
    const at::Tensor& w = dense(a[5], "w_kv", at::kBFloat16, 3, dev);
    const int64_t H = w.size(0);
    if (w.size(1) != 256 || w.size(2) != kDv)
      refuse(PyExc_ValueError, "w_kv must be [H, 256, %d], got %s", (int)kDv, text(w.sizes()).c_str());
    const int S = as_int(a[6], "S"), b = small(B, "B"), h = small(H, "H");
    if (S < 0) refuse(PyExc_ValueError, "need S >= 0, got %d", S);
    at::Tensor kv;
    if (a[7] == Py_None) {
      kv = made(at::kBFloat16, {H, S, 256}, dev);
    } else {
      address<void>(a[7], "kv", at::kBFloat16, {H, S, 256}, dev);
      kv = THPVariable_Unpack(a[7]);
    }
    Output k_rope(a[8], "k_rope", at::kBFloat16, {S, 64}, dev);
    void* out = kv.data_ptr();
    const void* weights = w.data_ptr();
    const mla_stream_t s = stream(dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g.expand(c.rows, c.scales, table.ptr, table.stride, seq, starts, b, c.block_size, c.num_blocks, table.columns,
                  weights, h, S, out, k_rope.ptr, s);
    Py_END_ALLOW_THREADS
    check(rc);
    PyObject* k = THPVariable_Wrap(half_head(kv, S, H, 0));
    PyObject* v = k != nullptr ? THPVariable_Wrap(half_head(kv, S, H, 128)) : nullptr;
    PyObject* all = v != nullptr ? PyTuple_Pack(3, k, v, k_rope.obj) : nullptr;
    Py_XDECREF(k);
    Py_XDECREF(v);
    return all;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// prefill(q, k_nope, k_rope, v, cu_q_lens, kv_starts, seq_lens, causal_seqlens_global, scale, cp_world, cp_rank,
//         out, lse, lse_base_e, workspace, return_lse, causal, interleave)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    prompt_arguments(n, 18);
    const at::Tensor& tq = tensor(a[0], "q", at::kBFloat16);
    const at::Tensor& tk = tensor(a[1], "k_nope", at::kBFloat16);
    const at::Tensor& tr = tensor(a[2], "k_rope", at::kBFloat16);
    const at::Tensor& tv = tensor(a[3], "v", at::kBFloat16);
    if (tq.dim() != 3 || tk.dim() != 3 || tr.dim() != 2 || tv.dim() != 3)
      refuse(PyExc_ValueError, "need q [T, H, 192], k_nope [S, H, 128], k_rope [S, 64], v [S, H, 128], got %s, %s, %s, %s",
             text(tq.sizes()).c_str(), text(tk.sizes()).c_str(), text(tr.sizes()).c_str(), text(tv.sizes()).c_str());
    const int dev = c10::cuda::current_device();
    const Rows q = rows_of(tq, "q", 192, true, dev), k = rows_of(tk, "k_nope", 128, true, dev),
               r = rows_of(tr, "k_rope", 64, false, dev), v = rows_of(tv, "v", 128, true, dev);
    if (k.H != q.H || v.H != q.H || r.T != k.T || v.T != k.T)
      refuse(PyExc_ValueError, "heads or key rows of q %s, k_nope %s, k_rope %s and v %s differ", text(tq.sizes()).c_str(),
             text(tk.sizes()).c_str(), text(tr.sizes()).c_str(), text(tv.sizes()).c_str());
    const at::Tensor& lens = tensor(a[6], "seq_lens", at::kInt);
    if (lens.dim() != 1) refuse(PyExc_ValueError, "seq_lens must be [B], got %s", text(lens.sizes()).c_str());
    const int64_t B = lens.size(0), H = q.H;
    const auto *cu = address<int32_t>(a[4], "cu_q_lens", at::kInt, {B + 1}, dev),
               *starts = address<int32_t>(a[5], "kv_starts", at::kInt, {B}, dev),
               *seq = address<int32_t>(a[6], "seq_lens", at::kInt, {B}, dev);
    const int32_t* global =
        a[7] == Py_None ? nullptr : address<int32_t>(a[7], "causal_seqlens_global", at::kInt, {B}, dev);
    const int T = small(q.T, "T"), S = small(k.T, "S"), h = small(H, "H"), b = small(B, "B");
    const float scale = as_float(a[8]);
    const int cp = as_int(a[9], "cp_world"), rank = as_int(a[10], "cp_rank"), il = as_int(a[17], "interleave");
    const bool base_e = as_bool(a[13]), causal = as_bool(a[16]);
    Output out(a[11], "out", at::kBFloat16, {T, H, 128}, dev);
    const bool with_lse = a[12] != Py_None || as_bool(a[15]);
    std::optional<Output> lse;
    if (with_lse) lse.emplace(a[12], "lse", at::kFloat, at::IntArrayRef({T, H}), dev);
    at::Tensor scratch;
    if (a[14] == Py_None) {
      const size_t bytes = g.prefill_workspace_size(
          T, b, h, S, at::cuda::getDeviceProperties((c10::DeviceIndex)dev)->multiProcessorCount);
      scratch = made(at::kByte, {(int64_t)bytes}, dev);
    } else {
      if (!THPVariable_Check(a[14])) refuse(PyExc_TypeError, "workspace must be a torch.Tensor");
      scratch = THPVariable_Unpack(a[14]);
      if (!scratch.is_cuda()) refuse(PyExc_ValueError, "workspace must be a CUDA tensor");
      if (!scratch.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
      here(scratch, "workspace", dev);
    }
    void *ws = scratch.data_ptr(), *o = out.ptr;
    float* l = with_lse ? static_cast<float*>(lse->ptr) : nullptr;
    const size_t ws_bytes = scratch.nbytes();
    const mla_stream_t s = stream(dev);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g.prefill(q.ptr, q.stride_t, q.stride_h, k.ptr, k.stride_t, k.stride_h, r.ptr, r.stride_t, v.ptr, v.stride_t,
                   v.stride_h, cu, starts, seq, global, T, b, h, S, causal, cp, rank, il, scale, o, l, base_e, ws,
                   ws_bytes, s);
    Py_END_ALLOW_THREADS
    check(rc);
    return PyTuple_Pack(2, out.obj, with_lse ? lse->obj : Py_None);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"step_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(step_tables)), METH_FASTCALL, nullptr},
    {"store", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(store)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {"bind_prompt", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_prompt)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"rope_store", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_store)), METH_FASTCALL, nullptr},
    {"expand", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(expand)), METH_FASTCALL, nullptr},
    {"prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefill)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "q8_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_q8_binding() { return PyModule_Create(&module); }
