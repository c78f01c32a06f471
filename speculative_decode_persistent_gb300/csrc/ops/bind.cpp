// Python side of the pool's operators: checks of tensors, the calls' structs,
// outputs and workspaces from torch's allocator, torch's current stream. The work
// itself is behind include/mk_ops.h, whose entries the package hands over as
// addresses (connect), so that this file needs no library but torch.
//
// A small call is bound by the host. The same marshalling in Python (ctypes, tensor
// attributes one by one) took 11 us of a call's 15, this takes 2 to 3.
//
// Handles (pools, rows, layers, rotations) are bytes objects with the C struct and
// the device; the classes that own them keep the tensors alive.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <initializer_list>
#include <string>

#include "mk_ops.h"

namespace {

constexpr int64_t kPage = 16;

// ---------------------------------------------------------------- the library
struct Library {
  decltype(&mk_kv_write) kv_write;
  decltype(&mk_kv_read) kv_read;
  decltype(&mk_attend_work_bytes) attend_work_bytes;
  decltype(&mk_attend_tree) attend_tree;
  decltype(&mk_rope_write) rope_write;
  decltype(&mk_tree_work_bytes) tree_work_bytes;
  decltype(&mk_tree_accept) tree_accept;
  decltype(&mk_kv_copy) kv_copy;
  decltype(&mk_kv_keep) kv_keep;
} lib;
PyObject* error_type = nullptr;

// --------------------------------------------------------------------- errors
struct Refusal {
  int status;
  std::string what;
};
[[noreturn]] void refuse(std::string what) { throw Refusal{MK_ERR_INVALID, std::move(what)}; }
struct PythonError {};  // already set

template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refusal& r) {
    PyObject* e = PyObject_CallFunction(error_type, "is", r.status, r.what.c_str());
    if (e) {
      PyErr_SetObject(error_type, e);
      Py_DECREF(e);
    }
  } catch (const PythonError&) {
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// -------------------------------------------------------------------- handles
struct PoolHandle {
  mk_kv_pool c;
  int32_t device;  // index, -1: not a CUDA device
};
struct RowsHandle {
  mk_kv_rows c;  // n_rows -1: as many as the call's tensors have; max_q -1: their mean
  int32_t device;
};
struct LayersHandle {
  mk_kv_layers c;
  int32_t device;
};
struct RopeHandle {
  mk_rope c;
  int32_t device, gain;  // gain: elements of the gains, 0: none
};

template <class T>
PyObject* handle(const T& x) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&x), sizeof(T));
}
template <class T>
T get(PyObject* o) {
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != static_cast<Py_ssize_t>(sizeof(T))) refuse("a handle of another kind");
  T x;
  std::memcpy(&x, PyBytes_AS_STRING(o), sizeof(T));
  return x;
}

// -------------------------------------------------------------------- tensors
const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + " (a tensor)");
  return THPVariable_Unpack(o);
}
int cuda_index(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }
bool on(const at::Tensor& t, int device) { return cuda_index(t) == device && (device >= 0 || t.is_cpu()); }
bool half_type(at::ScalarType t) { return t == at::kHalf || t == at::kShort; }
int dtype_of(at::ScalarType t) { return t == at::kFloat ? MK_F32 : t == at::kHalf ? MK_F16 : t == at::kBFloat16 ? MK_BF16 : -1; }
void no_gradient(const at::Tensor& t, const char* what) {
  if (t.requires_grad() && c10::GradMode::is_enabled())
    refuse(std::string(what) + " (no gradient is defined: detach it or use torch.no_grad)");
}

// Whether two of the n x heads vectors of dh elements at r row + h head share an element.
bool overlap(int64_t n, int64_t heads, int64_t dh, int64_t row, int64_t head) {
  if (n == 0 || (head >= dh && (n == 1 || row >= (heads - 1) * head + dh))) return false;  // rows of heads
  if (row >= dh && (heads == 1 || head >= (n - 1) * row + dh)) return false;               // heads of rows
  if ((n > 1 && row < dh) || (heads > 1 && head < dh)) return true;
  for (int64_t b = 1; b < heads; ++b)  // the multiples of row on both sides of each multiple of head
    for (int64_t a = b * head / row; a <= b * head / row + 1; ++a)
      if (a < n && std::llabs(a * row - b * head) < dh) return true;
  return false;
}

mk_dense dense(const at::Tensor& t, int64_t heads, int64_t dh, const char* what, bool out = false) {
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != dh)
    refuse(std::string(what) + " ([rows][" + std::to_string(heads) + "][" + std::to_string(dh) + "])");
  if (t.stride(2) != 1) refuse(std::string(what) + " (contiguous head dim)");
  if (out && overlap(t.size(0), heads, dh, t.stride(0), t.stride(1))) refuse(std::string(what) + " (rows of an output must not overlap)");
  no_gradient(t, what);
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}

// Rows of dense tensors that belong together.
int same(const PoolHandle& pool, const RowsHandle& rows, std::initializer_list<const at::Tensor*> all) {
  const at::Tensor& t = **all.begin();
  const int64_t n = t.size(0);
  if (rows.c.n_rows >= 0 && rows.c.n_rows != n) refuse("rows of the dense tensors differ from KVRows.n_rows");
  for (const at::Tensor* x : all)
    if (x->size(0) != n || x->scalar_type() != t.scalar_type()) refuse("dense tensors of one type with one number of rows");
  if (dtype_of(t.scalar_type()) < 0) refuse("dense tensors are float32, float16 or bfloat16");
  bool here = pool.device >= 0 && rows.device == pool.device;
  for (const at::Tensor* x : all) here = here && cuda_index(*x) == pool.device;
  if (!here) refuse("pool, rows and dense tensors on one CUDA device");
  if (n > INT32_MAX) throw Refusal{MK_ERR_UNSUPPORTED, "dense tensors (2^31 rows)"};
  return static_cast<int>(n);
}

mk_kv_rows with(const RowsHandle& rows, int n) {
  mk_kv_rows r = rows.c;
  r.n_rows = n;
  const int seqs = r.n_seqs > 1 ? r.n_seqs : 1;
  r.max_q = rows.c.max_q < 0 ? static_cast<int>((static_cast<int64_t>(n) + seqs - 1) / seqs) : rows.c.max_q < n ? rows.c.max_q : n;
  return r;
}

// Address of a contiguous int32 tensor of n elements, nullptr for None.
const int32_t* index(PyObject* o, int64_t n, int device, const char* what) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous() || !on(t, device))
    refuse(std::string(what) + " (contiguous int32 [" + std::to_string(n) + "] on the pool's device)");
  return t.data_ptr<int32_t>();
}

PyObject* tuple(std::initializer_list<PyObject*> items) {  // takes its items' references
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (!t || !o) {
      Py_XDECREF(o);
      Py_CLEAR(t);
      continue;
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  if (!t) throw PythonError{};
  return t;
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int device) {
  return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device))));
}

// f(stream) with the device current, on its current stream.
template <class F>
void run(int device, const char* what, F f) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
  void* const stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  mk_status rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f(stream);
  Py_END_ALLOW_THREADS
  if (rc != MK_OK) throw Refusal{rc, what};
}

int64_t integer(PyObject* o) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) {
    if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw PythonError{};
    PyErr_Clear();
    return INT64_MIN;
  }
  return x;
}
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
  return x;
}

// --------------------------------------------------------------- constructors
// One layer's tensors, [pages][kv heads][16][head dim], or several layers' with those in front.
template <bool LAYERS>
PyObject* make_pool(PyObject* const* a) {
  constexpr const char* name = LAYERS ? "KVLayers" : "KVPool";
  constexpr int o = LAYERS;  // dims before a page's
  auto no = [&](const char* what) { refuse(std::string(name) + " (" + what + ")"); };
  const at::Tensor &k = tensor(a[0], name), &v = tensor(a[1], name);
  if (k.dim() != 4 + o || v.sizes() != k.sizes() || k.size(2 + o) != kPage || v.scalar_type() != k.scalar_type() || (LAYERS && k.size(0) == 0))
    no(LAYERS ? "k and v are [layers][pages][kv heads][16][head dim] of one type" : "k and v are [pages][kv heads][16][head dim] of one type");
  const int64_t pages = k.size(o), heads = k.size(1 + o), dh = k.size(3 + o), n = LAYERS ? k.size(0) : 1;
  const int64_t layer = LAYERS && n > 1 ? k.stride(0) : 0;
  // each layer contiguous (by torch's rule: strides of dimensions of size 1 say nothing), all tensors' layers equally far apart
  auto packed = [&](const at::Tensor& t, int64_t per) {
    if (!LAYERS) return t.is_contiguous();
    int64_t want = 1;
    for (int d = 4; d >= 1; want *= t.size(d--))
      if (t.numel() && t.size(d) != 1 && t.stride(d) != want) return false;
    return n == 1 || (t.stride(0) * per == layer && layer >= pages * heads * kPage * dh && layer % 256 == 0);
  };
  if (!packed(k, 1) || !packed(v, 1)) no(LAYERS ? "contiguous layers, equally far apart in all tensors" : "contiguous tensors");
  const int device = cuda_index(k);
  if (!on(v, device)) no("one device");
  if (n > INT32_MAX || pages > INT32_MAX || heads > INT32_MAX || dh > INT32_MAX) throw Refusal{MK_ERR_UNSUPPORTED, name};
  mk_kv_pool p{k.data_ptr(), v.data_ptr(), nullptr, nullptr, MK_KV_F16, static_cast<int32_t>(pages), static_cast<int32_t>(heads), static_cast<int32_t>(dh)};
  if (k.scalar_type() == at::kChar) {
    p.kv_dtype = MK_KV_Q8;
    for (int i = 0; i < 2; ++i) {
      const bool given = a[2 + i] != Py_None;
      bool fits = given;
      if (given) {
        const at::Tensor& s = tensor(a[2 + i], name);
        fits = s.dim() == 4 + o && half_type(s.scalar_type()) && (!LAYERS || s.size(0) == n) && s.size(o) == pages && s.size(1 + o) == heads &&
               s.size(2 + o) == kPage && s.size(3 + o) == dh / 32 && on(s, device);
        if (fits && !packed(s, 32)) no(LAYERS ? "contiguous layers, equally far apart in all tensors" : "contiguous scales");
        (i ? p.v_scale : p.k_scale) = s.data_ptr();
      }
      if (!fits) no("an int8 pool needs binary16 scales, of the pool's shape with head dim / 32");
    }
  } else if (!half_type(k.scalar_type()) || a[2] != Py_None || a[3] != Py_None) {
    no("binary16, or int8 codes with scales");
  }
  if (LAYERS) return handle(LayersHandle{{p, static_cast<int32_t>(n), layer}, device});
  return handle(PoolHandle{p, device});
}

PyObject* make_rows(PyObject* const* a) {  // row_start, kv_len, tables, n_rows, max_q
  const at::Tensor &start = tensor(a[0], "KVRows"), &len = tensor(a[1], "KVRows"), &tables = tensor(a[2], "KVRows");
  for (const at::Tensor* t : {&start, &len, &tables})
    if (t->scalar_type() != at::kInt || !t->is_contiguous()) refuse("KVRows (contiguous int32 tensors)");
  if (tables.dim() != 2 || len.dim() != 1 || start.dim() != 1 || start.size(0) != len.size(0) + 1 || tables.size(0) != len.size(0))
    refuse("KVRows (row_start [n + 1], kv_len [n], tables [n][pages])");
  const int device = cuda_index(len);
  if (!on(start, device) || !on(tables, device)) refuse("KVRows (one device)");
  int64_t count[2];
  for (int i = 0; i < 2; ++i) {
    count[i] = a[3 + i] == Py_None ? -1 : integer(a[3 + i]);
    if (a[3 + i] != Py_None && (count[i] < 0 || count[i] > INT32_MAX)) refuse("KVRows (counts of rows)");
  }
  if (len.size(0) > INT32_MAX || tables.size(1) > INT32_MAX) throw Refusal{MK_ERR_UNSUPPORTED, "KVRows"};
  return handle(RowsHandle{{start.data_ptr<int32_t>(), len.data_ptr<int32_t>(), tables.data_ptr<int32_t>(), static_cast<int32_t>(len.size(0)),
                            static_cast<int32_t>(count[0]), static_cast<int32_t>(tables.size(1)), static_cast<int32_t>(count[1])},
                           device});
}

PyObject* make_rope(PyObject* const* a) {  // turns, q_gain, k_gain, dims, eps
  const at::Tensor& turns = tensor(a[0], "Rope");
  RopeHandle h{{static_cast<const uint64_t*>(turns.data_ptr()), nullptr, nullptr, static_cast<int32_t>(integer(a[3])), static_cast<float>(number(a[4]))},
               cuda_index(turns), 0};
  for (int i = 0; i < 2; ++i) {
    if (a[1 + i] == Py_None) continue;
    const at::Tensor& g = tensor(a[1 + i], "Rope");
    if (g.scalar_type() != at::kFloat || g.dim() != 1 || !g.is_contiguous() || !on(g, h.device) || (h.gain && g.size(0) != h.gain) ||
        g.size(0) < 1 || g.size(0) > 65536)
      refuse("Rope (gains: contiguous float32 [head dim] on one device)");
    no_gradient(g, "Rope gains");
    if (reinterpret_cast<uintptr_t>(g.data_ptr()) % 16) refuse("Rope (gains: 16-byte aligned)");
    (i ? h.c.k_gain : h.c.q_gain) = g.data_ptr<float>();
    h.gain = static_cast<int32_t>(g.size(0));
  }
  return handle(h);
}

// ------------------------------------------------------------------ operators
PyObject* kv_write(PyObject* const* a) {  // pool, rows, k, v
  const PoolHandle pool = get<PoolHandle>(a[0]);
  const RowsHandle rows = get<RowsHandle>(a[1]);
  const at::Tensor &k = tensor(a[2], "kv_write k"), &v = tensor(a[3], "kv_write v");
  const mk_dense kd = dense(k, pool.c.hkv, pool.c.dh, "kv_write k"), vd = dense(v, pool.c.hkv, pool.c.dh, "kv_write v");
  const mk_kv_rows r = with(rows, same(pool, rows, {&k, &v}));
  run(pool.device, "mk_kv_write", [&](void* s) { return lib.kv_write(&pool.c, &r, &kd, &vd, dtype_of(k.scalar_type()), s); });
  Py_RETURN_NONE;
}

PyObject* kv_read(PyObject* const* a) {  // pool, rows, dtype, k or None, v
  const PoolHandle pool = get<PoolHandle>(a[0]);
  const RowsHandle rows = get<RowsHandle>(a[1]);
  at::Tensor k, v;
  if (a[3] == Py_None) {
    if (!THPDtype_Check(a[2])) refuse("kv_read (dtype)");
    if (rows.c.n_rows < 0) refuse("kv_read (KVRows.n_rows or out)");
    if (pool.device < 0 || rows.device != pool.device) refuse("pool, rows and dense tensors on one CUDA device");
    const auto type = reinterpret_cast<THPDtype*>(a[2])->scalar_type;
    if (dtype_of(type) < 0) refuse("dense tensors are float32, float16 or bfloat16");
    const int64_t shape[3] = {rows.c.n_rows, pool.c.hkv, pool.c.dh};
    k = empty(shape, type, pool.device);
    v = empty(shape, type, pool.device);
  } else {
    k = tensor(a[3], "kv_read out");
    v = tensor(a[4], "kv_read out");
  }
  const mk_dense kd = dense(k, pool.c.hkv, pool.c.dh, "kv_read out", true), vd = dense(v, pool.c.hkv, pool.c.dh, "kv_read out", true);
  const mk_kv_rows r = with(rows, same(pool, rows, {&k, &v}));
  run(pool.device, "mk_kv_read", [&](void* s) { return lib.kv_read(&pool.c, &r, &kd, &vd, dtype_of(k.scalar_type()), s); });
  if (a[3] != Py_None) return tuple({Py_NewRef(a[3]), Py_NewRef(a[4])});
  return tuple({THPVariable_Wrap(std::move(k)), THPVariable_Wrap(std::move(v))});
}

PyObject* attend(PyObject* const* a) {  // pool, rows, q, scale, window, sinks, gate, out, parents
  const PoolHandle pool = get<PoolHandle>(a[0]);
  const RowsHandle rows = get<RowsHandle>(a[1]);
  const at::Tensor& q = tensor(a[2], "attend q");
  const int64_t hq = q.dim() == 3 ? q.size(1) : 0, dh = pool.c.dh;
  mk_attend_args x{};
  x.q = dense(q, hq, dh, "attend q");
  const at::Tensor* gate = nullptr;
  if (a[6] != Py_None) {
    gate = &tensor(a[6], "attend gate");
    x.gate = dense(*gate, hq, dh, "attend gate");
  }
  at::Tensor out;
  int n;
  if (a[7] == Py_None) {
    n = gate ? same(pool, rows, {&q, gate}) : same(pool, rows, {&q});
    out = empty(q.sizes(), q.scalar_type(), pool.device);
    x.out = {out.data_ptr(), hq * dh, dh};
  } else {
    out = tensor(a[7], "attend out");
    x.out = dense(out, hq, dh, "attend out", true);
    n = gate ? same(pool, rows, {&q, &out, gate}) : same(pool, rows, {&q, &out});
  }
  const double scale = a[3] == Py_None ? 1.0 / std::sqrt(static_cast<double>(dh)) : number(a[3]);
  const int64_t window = integer(a[4]), sinks = integer(a[5]);
  if (!(scale > 0.0 && scale < 3.4e38) || window < 0 || window > INT32_MAX || sinks < 0 || sinks > INT32_MAX || hq > INT32_MAX)
    refuse("attend (a finite positive scale, a window and sinks of at least 0)");
  x.hq = static_cast<int32_t>(hq);
  x.dtype = dtype_of(q.scalar_type());
  x.scale = static_cast<float>(scale);
  x.window = static_cast<int32_t>(window);
  x.sinks = static_cast<int32_t>(sinks);
  const mk_kv_rows r = with(rows, n);
  const int32_t* parents = index(a[8], n, pool.device, "attend parents");
  // from torch's allocator, so calls on other streams and captured graphs have their own
  const size_t bytes = lib.attend_work_bytes(&pool.c, &r, x.hq);
  const int64_t size[1] = {static_cast<int64_t>(bytes > 256 ? bytes : 256)};
  const at::Tensor work = empty(size, at::kByte, pool.device);
  x.work = work.data_ptr();
  x.work_bytes = static_cast<uint64_t>(size[0]);
  run(pool.device, "mk_attend", [&](void* s) { return lib.attend_tree(&pool.c, &r, &x, parents, s); });
  return a[7] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[7]);
}

PyObject* rope_write(PyObject* const* a) {  // pool, rows, rope, q, k, v, parents, positions, out
  const PoolHandle pool = get<PoolHandle>(a[0]);
  const RowsHandle rows = get<RowsHandle>(a[1]);
  const RopeHandle rope = get<RopeHandle>(a[2]);
  const at::Tensor &q = tensor(a[3], "rope_write q"), &k = tensor(a[4], "rope_write k"), &v = tensor(a[5], "rope_write v");
  const int64_t hq = q.dim() == 3 ? q.size(1) : 0, dh = pool.c.dh;
  mk_rope_args x{};
  x.q = dense(q, hq, dh, "rope_write q");
  x.k = dense(k, pool.c.hkv, dh, "rope_write k");
  x.v = dense(v, pool.c.hkv, dh, "rope_write v");
  at::Tensor out;
  int n;
  if (a[8] == Py_None) {
    n = same(pool, rows, {&q, &k, &v});
    out = empty(q.sizes(), q.scalar_type(), pool.device);
    x.out = {out.data_ptr(), hq * dh, dh};
  } else {
    out = tensor(a[8], "rope_write out");
    x.out = dense(out, hq, dh, "rope_write out", true);
    n = same(pool, rows, {&q, &k, &v, &out});
  }
  if (rope.device != pool.device || rope.c.rot > dh || (rope.gain && rope.gain != dh) || hq > INT32_MAX)
    refuse("rope_write (a Rope on the pool's device, of no more dims than a head and gains for all of them)");
  if (a[6] != Py_None && a[7] != Py_None) refuse("rope_write (parents or positions)");
  x.hq = static_cast<int32_t>(hq);
  x.dtype = dtype_of(q.scalar_type());
  x.rope = rope.c;
  x.parents = index(a[6], n, pool.device, "rope_write parents");
  x.positions = index(a[7], n, pool.device, "rope_write positions");
  const mk_kv_rows r = with(rows, n);
  run(pool.device, "mk_rope_write", [&](void* s) { return lib.rope_write(&pool.c, &r, &x, s); });
  return a[8] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[8]);
}

PyObject* tree_accept(PyObject* const* a) {  // rows, parents, tokens, logits
  const RowsHandle rows = get<RowsHandle>(a[0]);
  const at::Tensor& logits = tensor(a[3], "tree_accept logits");
  if (logits.dim() != 2 || dtype_of(logits.scalar_type()) < 0 || logits.size(1) == 0 || (logits.size(1) > 1 && logits.stride(1) != 1))
    refuse("tree_accept (logits [rows][vocabulary], float32, float16 or bfloat16, a row contiguous)");
  const int64_t n = logits.size(0), vocab = logits.size(1);
  if (rows.c.n_rows >= 0 && rows.c.n_rows != n) refuse("rows of the logits differ from KVRows.n_rows");
  if (rows.device < 0 || !on(logits, rows.device)) refuse("tree_accept (rows and logits on one CUDA device)");
  if (a[2] == Py_None) refuse("tree_accept (tokens)");
  if (n > INT32_MAX || vocab > INT32_MAX) throw Refusal{MK_ERR_UNSUPPORTED, "tree_accept (2^31 rows or logits)"};
  mk_tree_args x{};
  x.parents = index(a[1], n, rows.device, "tree_accept parents");
  x.tokens = index(a[2], n, rows.device, "tree_accept tokens");
  x.logits = logits.data_ptr();
  x.row_stride = logits.stride(0);
  x.vocab = static_cast<int32_t>(vocab);
  x.dtype = dtype_of(logits.scalar_type());
  const mk_kv_rows r = with(rows, static_cast<int>(n));
  const int64_t per_row[1] = {n}, per_seq[1] = {r.n_seqs};
  at::Tensor path = empty(per_row, at::kInt, rows.device), emitted = empty(per_row, at::kInt, rows.device),
             count = empty(per_seq, at::kInt, rows.device);
  x.path = path.data_ptr<int32_t>();
  x.emitted = emitted.data_ptr<int32_t>();
  x.count = count.data_ptr<int32_t>();
  x.work_bytes = lib.tree_work_bytes(&r, x.vocab);
  at::Tensor work;
  if (x.work_bytes) {
    const int64_t size[1] = {static_cast<int64_t>(x.work_bytes)};
    work = empty(size, at::kByte, rows.device);
    x.work = work.data_ptr();
  }
  run(rows.device, "mk_tree_accept", [&](void* s) { return lib.tree_accept(&r, &x, s); });
  return tuple({THPVariable_Wrap(std::move(path)), THPVariable_Wrap(std::move(count)), THPVariable_Wrap(std::move(emitted))});
}

PyObject* kv_copy(PyObject* const* a) {  // layers, src, dst
  const LayersHandle layers = get<LayersHandle>(a[0]);
  const at::Tensor& src = tensor(a[1], "kv_copy src");
  if (src.dim() != 1 || src.size(0) > INT32_MAX) refuse("kv_copy (int32 [n])");
  if (layers.device < 0) refuse("kv_copy (a CUDA device)");
  tensor(a[2], "kv_copy dst");
  const int64_t n = src.size(0);
  const int32_t *s = index(a[1], n, layers.device, "kv_copy src"), *d = index(a[2], n, layers.device, "kv_copy dst");
  run(layers.device, "mk_kv_copy", [&](void* st) { return lib.kv_copy(&layers.c, s, d, static_cast<int32_t>(n), st); });
  Py_RETURN_NONE;
}

PyObject* kv_keep(PyObject* const* a) {  // layers, rows, keep
  const LayersHandle layers = get<LayersHandle>(a[0]);
  const RowsHandle rows = get<RowsHandle>(a[1]);
  const at::Tensor& keep = tensor(a[2], "kv_keep keep");
  if (layers.device < 0 || rows.device != layers.device) refuse("kv_keep (layers and rows on one CUDA device)");
  if (keep.dim() != 1 || keep.size(0) > INT32_MAX || (rows.c.n_rows >= 0 && rows.c.n_rows != keep.size(0))) refuse("kv_keep (an entry per row)");
  const int64_t n = keep.size(0);
  const int32_t* entries = index(a[2], n, layers.device, "kv_keep keep");
  const mk_kv_rows r = with(rows, static_cast<int>(n));
  const int64_t per_seq[1] = {r.n_seqs};
  at::Tensor kv_len = empty(per_seq, at::kInt, layers.device);
  run(layers.device, "mk_kv_keep", [&](void* s) { return lib.kv_keep(&layers.c, &r, entries, kv_len.data_ptr<int32_t>(), s); });
  return THPVariable_Wrap(std::move(kv_len));
}

// --------------------------------------------------------------------- module
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", N, n);
    return nullptr;
  }
  return guarded([&] { return F(args); });
}
template <PyObject* (*F)(PyObject* const*), int N>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<F, N>)), METH_FASTCALL, nullptr};
}

// The error class, and the library's entries by name as addresses.
PyObject* connect(PyObject* const* a) {
  if (!PyDict_Check(a[1])) refuse("connect");
  auto set = [&](auto& fn, const char* name) {
    PyObject* at = PyDict_GetItemString(a[1], name);
    if (!at) refuse(std::string("connect (") + name + ")");
    const size_t p = PyLong_AsSize_t(at);
    if (PyErr_Occurred()) throw PythonError{};
    fn = reinterpret_cast<std::decay_t<decltype(fn)>>(p);
  };
  Py_XSETREF(error_type, Py_NewRef(a[0]));
  set(lib.kv_write, "mk_kv_write");
  set(lib.kv_read, "mk_kv_read");
  set(lib.attend_work_bytes, "mk_attend_work_bytes");
  set(lib.attend_tree, "mk_attend_tree");
  set(lib.rope_write, "mk_rope_write");
  set(lib.tree_work_bytes, "mk_tree_work_bytes");
  set(lib.tree_accept, "mk_tree_accept");
  set(lib.kv_copy, "mk_kv_copy");
  set(lib.kv_keep, "mk_kv_keep");
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {method<connect, 2>("connect"),       method<make_pool<false>, 4>("pool"), method<make_pool<true>, 4>("layers"),
                         method<make_rows, 5>("rows"),        method<make_rope, 5>("rope"),        method<kv_write, 4>("kv_write"),
                         method<kv_read, 5>("kv_read"),       method<attend, 9>("attend"),         method<rope_write, 9>("rope_write"),
                         method<tree_accept, 4>("tree_accept"), method<kv_copy, 3>("kv_copy"),     method<kv_keep, 3>("kv_keep"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
