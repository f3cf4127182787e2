// The short way from torch tensors to the operators' C functions.
//
// One decoded token runs a layer's five calls in some 22 us of GPU time, while checking arguments, allocating outputs
// and converting them one by one in Python takes 12 to 25 us a call on the GPU's host.  This module does the ordinary call in
// C++: it checks what it is given, allocates the outputs on torch's current stream and calls the library.  Whatever is not
// ordinary (a wrong argument, another device or stream) it leaves to operators.py by returning None, which looks again and
// raises what is wrong.  A status other than MOE_OK goes to the function given to init().
//
// Groups and 4-bit rows come as the tuples that operators.py keeps of them, integers and tensors:
//   groups  (device, E, P, T, k, offsets, tiles, order, place), or (device, E, P, T, k, buffer, byte, None, None) with the four
//           one after another from that byte of a buffer of the library's own
//   rows    (device, G, N, K, wdtype, codes, scales, g or None, number of g)
// Addresses are read from the tensors at each call: a copy has its own memory, and a resized tensor other memory than before.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe_operators.h"

namespace {

PyObject* g_raise = nullptr;   // operators.py's, called with a status

using at::ScalarType;

struct Groups { int64_t index, E, P, T, k, offsets, tiles, order, place; };
struct Rows { int64_t index, G, N, K, wdtype, codes, scales, g, g_count; };
static_assert(sizeof(Groups) == 9 * 8 && sizeof(Rows) == 9 * 8, "nine integers each");

template <typename T> T* ptr(int64_t p) { return reinterpret_cast<T*>((uintptr_t)p); }

// a contiguous CUDA tensor of `dim` dimensions on device `index` (any where -1), or NULL
const at::Tensor* tensor(PyObject* o, int dim, int64_t index) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.dim() != dim || !t.is_contiguous() || (index >= 0 && t.get_device() != index)) return nullptr;
  return &t;
}
const at::Tensor* typed(PyObject* o, ScalarType type, int dim, int64_t index) {
  const at::Tensor* t = tensor(o, dim, index);
  return t && t->scalar_type() == type ? t : nullptr;
}
// the library's code of fp32 or bf16, or -1
int float_code(const at::Tensor& t) {
  return t.scalar_type() == ScalarType::Float ? MOE_F32 : t.scalar_type() == ScalarType::BFloat16 ? MOE_BF16 : -1;
}
ScalarType float_type(long code) { return code == MOE_F32 ? ScalarType::Float : ScalarType::BFloat16; }
bool fits(int64_t v) { return v >= 0 && v <= 0x7fffffff; }
// the library's limits: pairs of a call, matrices of a stack, K
bool pairs_fit(int64_t T, int64_t k) { return T <= 0x70000000 / (k > 0 ? k : 1); }
bool matrices_fit(int64_t G, int64_t N, int64_t K) { return G <= 65535 && fits(N) && K <= 1 << 24; }
bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// the current stream, when `index` is the current device
bool here(int64_t index, void** stream) {
  if (c10::cuda::current_device() != index) return false;
  *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
  return true;
}
at::Tensor empty(at::IntArrayRef shape, ScalarType type, int64_t index) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)index));
}
// `bytes` of memory for several tensors of one call: an allocation costs more than the tensors on it
at::Tensor room(int64_t bytes, int64_t index) { return empty({bytes}, ScalarType::Byte, index); }
// a contiguous tensor at byte `at` of b's memory, without as_strided's way through the dispatcher (2 us)
at::Tensor on(const at::Tensor& b, int64_t at, at::IntArrayRef shape, ScalarType type) {
  const auto meta = c10::scalarTypeToTypeMeta(type);
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(b.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA), meta);
  t.unsafeGetTensorImpl()->set_storage_offset(at / (int64_t)meta.itemsize());
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}
PyObject* raise(moe_status st) {
  PyObject* r = PyObject_CallFunction(g_raise, "i", (int)st);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the library refused the call");
  return nullptr;
}
int64_t address(const at::Tensor& t) { return (int64_t)(uintptr_t)t.data_ptr(); }

// the first n integers of a tuple of nine
bool integers(PyObject* o, int n, int64_t* to) {
  if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 9) return false;
  for (int i = 0; i < n; ++i) to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
  return !PyErr_Occurred();
}
// bytes of t's memory from its first element on
int64_t bytes_from(const at::Tensor& t) { return (int64_t)t.storage().nbytes() - t.storage_offset() * (int64_t)t.itemsize(); }
// where a tensor of a tuple is now; false if it is no longer the one that was checked
bool held(PyObject* o, ScalarType type, int64_t index, int64_t numel, int64_t* p) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != type || t.numel() != numel || !t.is_contiguous() ||
      bytes_from(t) < numel * (int64_t)t.itemsize())
    return false;
  *p = address(t);
  return true;
}
bool groups_in(PyObject* o, Groups& g) {
  if (!integers(o, 5, &g.index)) return false;
  PyObject *first = PyTuple_GET_ITEM(o, 5), *second = PyTuple_GET_ITEM(o, 6);
  if (PyLong_Check(second)) {
    const int64_t at = PyLong_AsLongLong(second), bins = 4 * (g.E + 1);
    if (!THPVariable_Check(first)) return false;
    const at::Tensor& b = THPVariable_Unpack(first);
    if (!b.is_cuda() || b.get_device() != g.index || bytes_from(b) < at + 2 * bins + 8 * g.P) return false;
    g.offsets = address(b) + at;
    g.tiles = g.offsets + bins;
    g.order = g.tiles + bins;
    g.place = g.order + 4 * g.P;
    return true;
  }
  return held(first, ScalarType::Int, g.index, g.E + 1, &g.offsets) && held(second, ScalarType::Int, g.index, g.E + 1, &g.tiles) &&
         held(PyTuple_GET_ITEM(o, 7), ScalarType::Int, g.index, g.P, &g.order) && held(PyTuple_GET_ITEM(o, 8), ScalarType::Int, g.index, g.P, &g.place);
}

// one fp32 scale, or `most`: pointer and number, 0 and 0 for None
bool scale_of(PyObject* o, int64_t most, int64_t index, int64_t* p, int64_t* n) {
  *p = *n = 0;
  if (o == Py_None) return true;
  const at::Tensor* t = typed(o, ScalarType::Float, 1, index);
  if (!t || (t->numel() != 1 && t->numel() != most)) return false;
  *p = address(*t);
  *n = t->numel();
  return true;
}
int64_t block_of(int64_t wdtype) { return wdtype == MOE_NVFP4 ? 16 : 32; }
int64_t block_groups(int64_t wdtype, int64_t K) { return (K + 4 * block_of(wdtype) - 1) / (4 * block_of(wdtype)); }
int64_t row_tiles(const Rows& r, const Groups* g) {
  return g ? moe_grouped_tiles(g->P, (int32_t)g->E) : r.G * ((r.N + 127) / 128);
}

// rows with the groups that they are laid out by (NULL: matrices)
bool rows_in(PyObject* o, const Groups* g, Rows& r) {
  if (!integers(o, 5, &r.index)) return false;
  PyObject *scale = PyTuple_GET_ITEM(o, 7), *count = PyTuple_GET_ITEM(o, 8);
  r.g_count = PyLong_AsLongLong(count);
  r.g = 0;
  return held(PyTuple_GET_ITEM(o, 5), ScalarType::Byte, r.index, r.G * r.N * (r.K / 2), &r.codes) &&
         held(PyTuple_GET_ITEM(o, 6), ScalarType::Byte, r.index, row_tiles(r, g) * block_groups(r.wdtype, r.K) * 512, &r.scales) &&
         (scale == Py_None || held(scale, ScalarType::Float, r.index, r.g_count, &r.g));
}
// a new tuple of rows; takes codes and scales
PyObject* rows_tuple(const Rows& r, PyObject* codes, PyObject* scales, PyObject* g) {
  return Py_BuildValue("(LLLLLNNOL)", (long long)r.index, (long long)r.G, (long long)r.N, (long long)r.K, (long long)r.wdtype, codes, scales, g, (long long)r.g_count);
}

// room for the rows r describes
void make_rows(Rows& r, const Groups* g, bool stacked, at::Tensor& codes, at::Tensor& scales) {
  const int64_t cb = (r.G * r.N * (r.K / 2) + 15) / 16 * 16, tiles = row_tiles(r, g), groups = block_groups(r.wdtype, r.K);
  const at::Tensor b = room(cb + tiles * groups * 512, r.index);
  codes = stacked ? on(b, 0, {r.G, r.N, r.K / 2}, ScalarType::Byte) : on(b, 0, {r.N, r.K / 2}, ScalarType::Byte);
  scales = on(b, cb, {tiles, groups, 512}, ScalarType::Byte);
  r.codes = address(b);
  r.scales = r.codes + cb;
}

#define OTHERWISE Py_RETURN_NONE
#define TRY try {
#define CATCH                                                   \
  }                                                             \
  catch (const std::exception& e) {                             \
    PyErr_SetString(PyExc_RuntimeError, e.what());              \
    return nullptr;                                             \
  }

// groups_of(offsets, tiles, order, place) -> tuple
PyObject* groups_of(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  if (n != 4) OTHERWISE;
  const at::Tensor* off = typed(a[0], ScalarType::Int, 1, -1);
  if (!off) OTHERWISE;
  Groups g{};
  g.index = off->get_device();
  const at::Tensor *til = typed(a[1], ScalarType::Int, 1, g.index), *order = typed(a[2], ScalarType::Int, 1, g.index),
                   *place = typed(a[3], ScalarType::Int, 2, g.index);
  if (!til || !order || !place) OTHERWISE;
  g.E = off->numel() - 1;
  g.P = order->numel();
  g.T = place->size(0);
  g.k = place->size(1);
  if (g.E < 1 || g.E > 4096 || til->numel() != g.E + 1 || g.T * g.k != g.P || !pairs_fit(g.P, 1)) OTHERWISE;
  for (const at::Tensor* t : {off, til, order, place}) (void)address(*t);   // throws where there is no memory
  return Py_BuildValue("(LLLLLOOOO)", (long long)g.index, (long long)g.E, (long long)g.P, (long long)g.T, (long long)g.k, a[0], a[1], a[2], a[3]);
  CATCH
}

// rows_of(codes, scales, wdtype, g, groups) -> tuple
PyObject* rows_of(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  if (n != 5 || !THPVariable_Check(a[0])) OTHERWISE;
  Groups gr{};
  const bool grouped = a[4] != Py_None;
  if (grouped && !groups_in(a[4], gr)) OTHERWISE;
  const int dim = grouped || THPVariable_Unpack(a[0]).dim() != 3 ? 2 : 3;
  const at::Tensor* codes = typed(a[0], ScalarType::Byte, dim, grouped ? gr.index : -1);
  if (!codes) OTHERWISE;
  Rows r{};
  r.index = codes->get_device();
  const at::Tensor* scales = typed(a[1], ScalarType::Byte, 3, r.index);
  if (!scales) OTHERWISE;
  r.wdtype = PyLong_AsLong(a[2]);
  r.G = dim == 3 ? codes->size(0) : 1;
  r.N = codes->size(dim - 2);
  r.K = 2 * codes->size(dim - 1);
  if (r.K <= 0 || r.K % 32 || !matrices_fit(r.G, r.N, r.K) || (grouped && r.N != gr.P)) OTHERWISE;
  if (scales->size(0) != row_tiles(r, grouped ? &gr : nullptr) || scales->size(1) != block_groups(r.wdtype, r.K) || scales->size(2) != 512) OTHERWISE;
  r.codes = address(*codes);
  r.scales = address(*scales);
  if ((r.codes | r.scales) % 16 || !scale_of(a[3], r.G, r.index, &r.g, &r.g_count)) OTHERWISE;
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  return rows_tuple(r, a[0], a[1], a[3]);
  CATCH
}

// route(logits, k, scoring, bias, n_group, topk_group, renormalize, scale, groups) -> (ids, w, None or groups)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  if (n != 9) OTHERWISE;
  const at::Tensor* x = tensor(a[0], 2, -1);
  if (!x) OTHERWISE;
  const int dt = float_code(*x);
  const int64_t T = x->size(0), E = x->size(1), index = x->get_device();
  const long k = PyLong_AsLong(a[1]), sc = PyLong_AsLong(a[2]), ng = PyLong_AsLong(a[4]), tg = PyLong_AsLong(a[5]);
  const int renorm = PyObject_IsTrue(a[6]), group = PyObject_IsTrue(a[8]);
  const double scale = PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred()) return nullptr;
  void* s;
  if (dt < 0 || (sc != 0 && sc != 1) || k < 1 || k > E || E > 4096 || !pairs_fit(T, k) || (sc == 0 && (a[3] != Py_None || ng != 1)) || ng < 1 || ng > 32 || E % ng || tg < 1 ||
      tg > ng || tg * (E / ng) < k || !here(index, &s))
    OTHERWISE;
  const at::Tensor* bias = nullptr;
  if (a[3] != Py_None) {
    bias = typed(a[3], ScalarType::Float, 1, index);
    if (!bias || bias->numel() != E) OTHERWISE;
  }
  // ids, gates, and with groups their four arrays: in one allocation up to 256 pairs.  Otherwise the groups have one of
  // their own, so that keeping or saving ids does not keep them.  The workspace goes when the call returns.
  const int64_t pairs = 4 * T * k, bins = 4 * (E + 1), wb = group ? moe_group_workspace((int32_t)T, (int32_t)k, (int32_t)E) : 0;
  const int64_t many = group ? 2 * bins + 2 * pairs : 0;
  const bool few = T * k <= 256;
  const at::Tensor both = room(2 * pairs + (few ? many : 0), index), buf = few || !group ? both : room(many, index);
  at::Tensor ws;
  if (wb) ws = room(wb, index);
  const at::Tensor ids = on(both, 0, {T, k}, ScalarType::Int), w = on(both, pairs, {T, k}, ScalarType::Float);
  const int64_t from = few ? 2 * pairs : 0, base = address(buf) + from;
  Groups g{};
  if (group) g = Groups{index, E, T * k, T, k, base, base + bins, base + 2 * bins, base + 2 * bins + pairs};
  const moe_status st = moe_route((int32_t)T, (int32_t)E, (int32_t)k, dt, x->data_ptr(), (int32_t)sc, bias ? bias->data_ptr<float>() : nullptr, (int32_t)ng,
                                  (int32_t)tg, renorm, (float)scale, ids.data_ptr<int32_t>(), w.data_ptr<float>(), ptr<int32_t>(g.offsets), ptr<int32_t>(g.tiles),
                                  ptr<int32_t>(g.order), ptr<int32_t>(g.place), wb ? ws.data_ptr() : nullptr, wb, s);
  if (st != MOE_OK) return raise(st);
  PyObject* third = Py_None;
  if (group)
    third = Py_BuildValue("(LLLLLNLOO)", (long long)index, (long long)E, (long long)g.P, (long long)T, (long long)k, THPVariable_Wrap(buf), (long long)from, Py_None, Py_None);
  else Py_INCREF(third);
  return Py_BuildValue("(NNN)", THPVariable_Wrap(ids), THPVariable_Wrap(w), third);
  CATCH
}

// quantize(x, wdtype, g, groups) -> rows
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  if (n != 4 || !THPVariable_Check(a[0])) OTHERWISE;
  Groups gr{};
  const bool grouped = a[3] != Py_None;
  if (grouped && !groups_in(a[3], gr)) OTHERWISE;
  const int dim = grouped || THPVariable_Unpack(a[0]).dim() != 3 ? 2 : 3;
  const at::Tensor* x = tensor(a[0], dim, grouped ? gr.index : -1);
  if (!x) OTHERWISE;
  const int dt = float_code(*x);
  Rows r{};
  r.index = x->get_device();
  r.wdtype = PyLong_AsLong(a[1]);
  r.G = dim == 3 ? x->size(0) : 1;
  r.N = grouped ? gr.P : x->size(dim - 2);
  r.K = x->size(dim - 1);
  void* s;
  if (dt < 0 || r.K <= 0 || r.K % 32 || !matrices_fit(r.G, r.N, r.K) || (grouped && x->size(0) != gr.T) || !aligned(x->data_ptr(), 16) ||
      (a[2] != Py_None && r.wdtype != MOE_NVFP4) || !scale_of(a[2], r.G, r.index, &r.g, &r.g_count) || !here(r.index, &s))
    OTHERWISE;
  at::Tensor codes, scales;
  make_rows(r, grouped ? &gr : nullptr, dim == 3, codes, scales);
  const moe_status st =
      moe_quantize_fp4((int32_t)r.G, (int32_t)r.N, (int32_t)r.K, dt, x->data_ptr(), (int32_t)r.wdtype, ptr<float>(r.g), (int32_t)r.g_count, (int32_t)gr.E,
                       (int32_t)gr.k, ptr<int32_t>(gr.offsets), ptr<int32_t>(gr.tiles), ptr<int32_t>(gr.place), ptr<uint8_t>(r.codes), ptr<uint8_t>(r.scales), s);
  if (st != MOE_OK) return raise(st);
  return rows_tuple(r, THPVariable_Wrap(codes), THPVariable_Wrap(scales), a[2]);
  CATCH
}

// dequantize(rows, groups, stacked, out dtype) -> tensor
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  Rows r{};
  Groups gr{};
  const bool grouped = n == 4 && a[1] != Py_None;
  if (n != 4 || (grouped && !groups_in(a[1], gr)) || !rows_in(a[0], grouped ? &gr : nullptr, r)) OTHERWISE;
  const long od = PyLong_AsLong(a[3]);
  void* s;
  if (!here(r.index, &s)) OTHERWISE;
  at::Tensor out = PyObject_IsTrue(a[2]) ? empty({r.G, r.N, r.K}, float_type(od), r.index) : empty({r.N, r.K}, float_type(od), r.index);
  const moe_status st = moe_dequantize_fp4((int32_t)r.G, (int32_t)r.N, (int32_t)r.K, (int32_t)r.wdtype, ptr<uint8_t>(r.codes), ptr<uint8_t>(r.scales),
                                           ptr<float>(r.g), (int32_t)r.g_count, (int32_t)gr.E, ptr<int32_t>(gr.offsets), ptr<int32_t>(gr.tiles), (int32_t)od,
                                           out.data_ptr(), s);
  if (st != MOE_OK) return raise(st);
  return THPVariable_Wrap(out);
  CATCH
}

// matmul(x, w, groups, act, gather, out dtype) -> tensor
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  Groups g{};
  if (n != 6 || !groups_in(a[2], g)) OTHERWISE;
  const at::Tensor *x = typed(a[0], ScalarType::BFloat16, 2, g.index), *w = typed(a[1], ScalarType::BFloat16, 3, g.index);
  if (!x || !w) OTHERWISE;
  const long act = PyLong_AsLong(a[3]), od = PyLong_AsLong(a[5]);
  const int gather = PyObject_IsTrue(a[4]);
  if (PyErr_Occurred()) return nullptr;
  const int64_t E = w->size(0), N = w->size(1), K = w->size(2), rows = gather ? g.T : g.P;
  void* s;
  if (E != g.E || N < 1 || K < 1 || K % 8 || (act && N % 32) || x->size(0) != rows || x->size(1) != K || !matrices_fit(E, N, K) || !fits(g.P) ||
      !aligned(x->data_ptr(), 16) || !aligned(w->data_ptr(), 16) || !here(g.index, &s))
    OTHERWISE;
  at::Tensor out = empty({g.P, act ? N / 2 : N}, float_type(od), g.index), ws;
  const int64_t wb = moe_grouped_matmul_workspace((int32_t)g.P, (int32_t)E, (int32_t)K, gather);
  if (wb) ws = empty({wb}, ScalarType::Byte, g.index);
  const moe_status st = moe_grouped_matmul((int32_t)g.P, (int32_t)E, (int32_t)N, (int32_t)K, x->data_ptr(), (int32_t)rows, gather ? ptr<int32_t>(g.order) : nullptr,
                                           gather ? ptr<int32_t>(g.place) : nullptr, (int32_t)g.k, w->data_ptr(), ptr<int32_t>(g.offsets), ptr<int32_t>(g.tiles), (int32_t)act, (int32_t)od, out.data_ptr(),
                                           wb ? ws.data_ptr() : nullptr, wb, s);
  if (st != MOE_OK) return raise(st);
  return THPVariable_Wrap(out);
  CATCH
}

// matmul_fp4(x rows, w rows, x's groups, groups, act, g_out or False, out dtype) -> tensor, or with a g_out (None = 1) rows
PyObject* matmul_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  Rows x{}, w{};
  Groups xg{}, g{};
  if (n != 7 || !groups_in(a[2], xg) || !groups_in(a[3], g) || !rows_in(a[0], &xg, x) || !rows_in(a[1], nullptr, w)) OTHERWISE;
  const long act = PyLong_AsLong(a[4]), od = PyLong_AsLong(a[6]);
  const bool quant = a[5] != Py_False;
  const int64_t cols = act ? w.N / 2 : w.N;
  void* s;
  // x's scale tiles lie by its own groups: they have to be these, or of the same tensors
  if (w.G != g.E || xg.offsets != g.offsets || xg.tiles != g.tiles || xg.E != g.E || x.index != w.index || g.index != w.index || x.wdtype != w.wdtype || x.N != g.P || x.K != w.K || x.g_count > 1 || w.N < 1 ||
      !fits(w.N) || !fits(g.P) || (act && w.N % 32) || (quant && (!act || cols % 32)) || !here(w.index, &s))
    OTHERWISE;
  at::Tensor out, codes, scales;
  Rows r{w.index, 1, g.P, cols, w.wdtype, 0, 0, 0, 0};
  if (quant) {
    if ((a[5] != Py_None && w.wdtype != MOE_NVFP4) || !scale_of(a[5], 1, w.index, &r.g, &r.g_count)) OTHERWISE;
    make_rows(r, &g, false, codes, scales);
  } else {
    out = empty({g.P, cols}, float_type(od), w.index);
  }
  const moe_status st = moe_grouped_matmul_fp4(
      (int32_t)g.P, (int32_t)g.E, (int32_t)w.N, (int32_t)w.K, (int32_t)w.wdtype, ptr<uint8_t>(x.codes), ptr<uint8_t>(x.scales), ptr<float>(x.g), ptr<uint8_t>(w.codes),
      ptr<uint8_t>(w.scales), ptr<float>(w.g), (int32_t)w.g_count, ptr<int32_t>(g.offsets), ptr<int32_t>(g.tiles), (int32_t)act, (int32_t)od,
      quant ? nullptr : out.data_ptr(), ptr<uint8_t>(r.codes), ptr<uint8_t>(r.scales), ptr<float>(r.g), s);
  if (st != MOE_OK) return raise(st);
  if (!quant) return THPVariable_Wrap(out);
  return rows_tuple(r, THPVariable_Wrap(codes), THPVariable_Wrap(scales), a[5]);
  CATCH
}

// combine(y, groups, topk_w, out dtype) -> tensor
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  Groups g{};
  if (n != 4 || !groups_in(a[1], g)) OTHERWISE;
  const at::Tensor *y = tensor(a[0], 2, g.index), *w = typed(a[2], ScalarType::Float, 2, g.index);
  if (!y || !w) OTHERWISE;
  const int dt = float_code(*y);
  const long od = PyLong_AsLong(a[3]);
  const int64_t N = y->size(1);
  void* s;
  if (dt < 0 || w->size(0) != g.T || w->size(1) != g.k || y->size(0) != g.P || N < 1 || !fits(N) || !fits(g.P) ||
      (N % 8 == 0 && !aligned(y->data_ptr(), 16)) || !here(g.index, &s))
    OTHERWISE;
  at::Tensor out = empty({g.T, N}, float_type(od), g.index);
  const moe_status st = moe_combine((int32_t)g.T, (int32_t)g.k, (int32_t)N, dt, y->data_ptr(), ptr<int32_t>(g.place), w->data_ptr<float>(), (int32_t)od, out.data_ptr(), s);
  if (st != MOE_OK) return raise(st);
  return THPVariable_Wrap(out);
  CATCH
}

// contiguous fp32 or bf16 of this shape on `index`, its code to *dt; None is fine where `none`
bool floats_in(PyObject* o, at::IntArrayRef shape, int64_t index, bool none, int* dt) {
  *dt = MOE_F32;
  if (o == Py_None) return none;
  const at::Tensor* t = tensor(o, (int)shape.size(), index);
  return t && t->sizes() == shape && (*dt = float_code(*t)) >= 0;
}
// where it is, once all else is right; false if it is not on 16 bytes where `wide`
bool pointer(PyObject* o, bool wide, const void** p) {
  *p = o == Py_None ? nullptr : THPVariable_Unpack(o).data_ptr();
  return !wide || aligned(*p, 16);
}

// codes and scales of 8-bit blocks, as they are now: [R, K] with scales [blocks of K, R], or [N, K] / [G, N, K] with a block of 128 x 128 each
struct Blocks8 { int64_t index, G, N, K; const uint8_t* codes; const float* scales; };
bool blocks8_in(PyObject* c, PyObject* s, bool rows, int dim, int64_t index, Blocks8& b) {
  const at::Tensor* codes = typed(c, ScalarType::Float8_e4m3fn, dim, index);
  if (!codes) return false;
  b.index = codes->get_device();
  b.G = dim == 3 ? codes->size(0) : 1;
  b.N = codes->size(dim - 2);
  b.K = codes->size(dim - 1);
  if (b.K < 1 || b.K % 16 || !matrices_fit(b.G, b.N, b.K)) return false;
  const at::Tensor* scales = typed(s, ScalarType::Float, dim, b.index);
  const int64_t kb = (b.K + 127) / 128, nb = (b.N + 127) / 128;
  if (!scales || (dim == 3 && scales->size(0) != b.G) || scales->size(dim - 2) != (rows ? kb : nb) || scales->size(dim - 1) != (rows ? b.N : kb)) return false;
  if (bytes_from(*codes) < b.G * b.N * b.K || bytes_from(*scales) < scales->numel() * 4) return false;
  b.codes = static_cast<const uint8_t*>(codes->data_ptr());
  b.scales = static_cast<const float*>(scales->data_ptr());
  return aligned(b.codes, 16);
}
// room for rows [R, K] and their scales
PyObject* make_rows8(int64_t R, int64_t K, int64_t index, uint8_t** codes, float** scales) {
  const int64_t cb = (R * K + 15) / 16 * 16, kb = (K + 127) / 128;
  const at::Tensor b = room(cb + kb * R * 4, index);
  *codes = static_cast<uint8_t*>(b.data_ptr());
  *scales = reinterpret_cast<float*>(*codes + cb);
  return Py_BuildValue("(NN)", THPVariable_Wrap(on(b, 0, {R, K}, ScalarType::Float8_e4m3fn)), THPVariable_Wrap(on(b, cb, {kb, R}, ScalarType::Float)));
}
PyObject* or_raise(moe_status st, PyObject* r) {
  if (st == MOE_OK) return r;
  Py_XDECREF(r);
  return raise(st);
}

// blocks8(codes, scales, rows) -> True if they are 8-bit rows, or weights
PyObject* blocks8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  Blocks8 b;
  if (n != 3 || !THPVariable_Check(a[0])) OTHERWISE;
  const bool rows = a[2] == Py_True;
  if (!blocks8_in(a[0], a[1], rows, !rows && THPVariable_Unpack(a[0]).dim() == 3 ? 3 : 2, -1, b)) OTHERWISE;
  Py_RETURN_TRUE;
  CATCH
}

// dequantize8(codes, scales, rows, out dtype) -> tensor
PyObject* dequantize8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  Blocks8 b;
  if (n != 4 || !THPVariable_Check(a[0])) OTHERWISE;
  const bool rows = a[2] == Py_True;
  const at::Tensor& codes = THPVariable_Unpack(a[0]);
  if (!blocks8_in(a[0], a[1], rows, !rows && codes.dim() == 3 ? 3 : 2, -1, b)) OTHERWISE;
  const long od = PyLong_AsLong(a[3]);
  void* s;
  if (PyErr_Occurred()) return nullptr;
  if (!here(b.index, &s)) OTHERWISE;
  const at::Tensor out = empty(codes.sizes(), float_type(od), b.index);
  PyObject* r = THPVariable_Wrap(out);
  if (out.numel() == 0) return r;
  return or_raise(moe_dequantize_fp8((int32_t)b.G, (int32_t)b.N, (int32_t)b.K, !rows, b.codes, b.scales, (int32_t)od, out.data_ptr(), s), r);
  CATCH
}

// quantize_weights8(w) -> (codes, scales)
PyObject* quantize_weights8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  if (n != 1 || !THPVariable_Check(a[0])) OTHERWISE;
  const int dim = THPVariable_Unpack(a[0]).dim() == 3 ? 3 : 2;
  const at::Tensor* w = tensor(a[0], dim, -1);
  if (!w) OTHERWISE;
  const int dt = float_code(*w);
  const int64_t G = dim == 3 ? w->size(0) : 1, N = w->size(dim - 2), K = w->size(dim - 1), index = w->get_device(), nb = (N + 127) / 128, kb = (K + 127) / 128;
  void* s;
  if (dt < 0 || K < 1 || K % 16 || !matrices_fit(G, N, K) || nb * kb > 0x7fffffff || !aligned(w->data_ptr(), 16) || !here(index, &s)) OTHERWISE;
  const at::Tensor codes = empty(w->sizes(), ScalarType::Float8_e4m3fn, index);
  const at::Tensor scales = dim == 3 ? empty({G, nb, kb}, ScalarType::Float, index) : empty({nb, kb}, ScalarType::Float, index);
  PyObject* r = Py_BuildValue("(NN)", THPVariable_Wrap(codes), THPVariable_Wrap(scales));
  if (w->numel() == 0) return r;
  return or_raise(moe_quantize_fp8_weights((int32_t)G, (int32_t)N, (int32_t)K, dt, w->data_ptr(), static_cast<uint8_t*>(codes.data_ptr()), scales.data_ptr<float>(), s), r);
  CATCH
}

// quantize8(x, groups) -> (codes, scales)
PyObject* quantize8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  if (n != 2) OTHERWISE;
  Groups g{};
  const bool grouped = a[1] != Py_None;
  if (grouped && !groups_in(a[1], g)) OTHERWISE;
  const at::Tensor* x = tensor(a[0], 2, grouped ? g.index : -1);
  if (!x) OTHERWISE;
  const int dt = float_code(*x);
  const int64_t T = x->size(0), K = x->size(1), index = x->get_device();
  void* s;
  if (dt < 0 || K < 1 || K % 16 || !matrices_fit(1, T, K) || !pairs_fit(T, 1) || (grouped && T != g.T) || (grouped && g.k < 1) || !aligned(x->data_ptr(), 16) ||
      !here(index, &s))
    OTHERWISE;
  uint8_t* codes;
  float* scales;
  PyObject* r = make_rows8(grouped ? g.P : T, K, index, &codes, &scales);
  return or_raise(moe_quantize_fp8((int32_t)T, (int32_t)K, dt, x->data_ptr(), grouped ? (int32_t)g.k : 1, ptr<int32_t>(g.place), codes, scales, s), r);
  CATCH
}

// matmul8(x codes, x scales, w codes, w scales, groups, act, quantize, out dtype) -> tensor, or (codes, scales)
PyObject* matmul8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  if (n != 8) OTHERWISE;
  Groups g{};
  Blocks8 x, w;
  const bool grouped = a[4] != Py_None;
  if (grouped && !groups_in(a[4], g)) OTHERWISE;
  if (!blocks8_in(a[2], a[3], false, grouped ? 3 : 2, grouped ? g.index : -1, w) || !blocks8_in(a[0], a[1], true, 2, w.index, x)) OTHERWISE;
  const long act = PyLong_AsLong(a[5]), od = PyLong_AsLong(a[7]);
  const int quant = PyObject_IsTrue(a[6]);
  if (PyErr_Occurred()) return nullptr;
  const int64_t cols = act ? w.N / 2 : w.N;
  void* s;
  if ((grouped && (w.G != g.E || x.N != g.P)) || x.K != w.K || w.N < 1 || !pairs_fit(x.N, 1) || (act && w.N % 128) || (quant && !act) || !here(w.index, &s)) OTHERWISE;
  PyObject* r;
  void* out = nullptr;
  uint8_t* codes = nullptr;
  float* scales = nullptr;
  if (quant) {
    r = make_rows8(x.N, cols, w.index, &codes, &scales);
  } else {
    const at::Tensor t = empty({x.N, cols}, float_type(od), w.index);
    out = t.data_ptr();
    r = THPVariable_Wrap(t);
  }
  if (x.N == 0) return r;   // its memory has no address
  return or_raise(moe_grouped_matmul_fp8((int32_t)x.N, grouped ? (int32_t)g.E : 1, (int32_t)w.N, (int32_t)w.K, x.codes, x.scales, w.codes, w.scales,
                                         grouped ? ptr<int32_t>(g.offsets) : nullptr, (int32_t)act, (int32_t)od, out, codes, scales, s), r);
  CATCH
}

// block_end(y, groups, topk_w, residual, shared, post, gate, scale, pre, eps, z dtype) -> h, or (h, z); z alone with y None
PyObject* block_end(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  if (n != 11) OTHERWISE;
  const at::Tensor* r = tensor(a[3], 2, -1);
  if (!r) OTHERWISE;
  const int64_t T = r->size(0), N = r->size(1), index = r->get_device();
  const bool wide = N % 8 == 0, grouped = a[1] != Py_None, any = a[0] != Py_None, normed = a[8] != Py_None;
  Groups g{};
  const at::Tensor* w = nullptr;
  int yd, rd, sd, pd, qd, gd;
  const void *y, *res, *shared, *post, *pre, *gate;
  if (grouped) {
    if (!any || !groups_in(a[1], g) || g.index != index || g.T != T || g.k < 1) OTHERWISE;
    w = typed(a[2], ScalarType::Float, 2, index);
    if (!w || w->size(0) != g.T || w->size(1) != g.k) OTHERWISE;
  }
  const bool per_row = THPVariable_Check(a[6]) && THPVariable_Unpack(a[6]).dim() == 2;
  const int64_t rows[2] = {T, N}, pairs[2] = {grouped ? g.P : T, N}, width[1] = {N}, each[2] = {T, 1};
  if (N < 1 || N > 32768 || !pairs_fit(T, 1) || !floats_in(a[3], rows, index, false, &rd) || !floats_in(a[0], pairs, index, true, &yd) ||
      !floats_in(a[4], rows, index, true, &sd) || (a[4] != Py_None && sd != yd) || !floats_in(a[5], width, index, true, &pd) ||
      !floats_in(a[8], width, index, true, &qd) || !(per_row ? floats_in(a[6], each, index, true, &gd) : floats_in(a[6], width, index, true, &gd)) || gd != MOE_F32 ||
      (!any && (!normed || a[4] != Py_None || a[5] != Py_None || a[6] != Py_None)))
    OTHERWISE;
  const double scale = PyFloat_AsDouble(a[7]), eps = PyFloat_AsDouble(a[9]);
  const long zd = PyLong_AsLong(a[10]);
  if (PyErr_Occurred()) return nullptr;
  void* s;
  if (!(eps >= 1.1754944e-38 && eps <= 3e38) || !(scale >= -3.4e38 && scale <= 3.4e38) || !pointer(a[3], wide, &res) || !pointer(a[0], wide, &y) ||
      !pointer(a[4], wide, &shared) || !pointer(a[5], wide, &post) || !pointer(a[8], wide, &pre) || !pointer(a[6], wide && !per_row, &gate) || !here(index, &s))
    OTHERWISE;
  // both in one allocation up to 64 K elements; larger ones apart, so that keeping the stream does not keep what the norm made of it
  at::Tensor h, z;
  if (any && normed && T * N <= 65536) {
    const ScalarType ht = float_type(rd), zt = float_type(zd);
    const int64_t hb = (T * N * (rd == MOE_F32 ? 4 : 2) + 15) / 16 * 16;
    const at::Tensor b = room(hb + T * N * (zd == MOE_F32 ? 4 : 2), index);
    h = on(b, 0, {T, N}, ht);
    z = on(b, hb, {T, N}, zt);
  } else {
    if (any) h = empty({T, N}, float_type(rd), index);
    if (normed) z = empty({T, N}, float_type(zd), index);
  }
  PyObject* result = any && normed ? Py_BuildValue("(NN)", THPVariable_Wrap(h), THPVariable_Wrap(z)) : THPVariable_Wrap(any ? h : z);
  if (T == 0) return result;
  return or_raise(moe_combine_norm((int32_t)T, grouped ? (int32_t)g.k : 1, (int32_t)N, yd, y, ptr<int32_t>(g.place), w ? w->data_ptr<float>() : nullptr, shared, pd, post,
                                   per_row, static_cast<const float*>(gate), (float)scale, rd, res, qd, pre, (float)eps, any ? h.data_ptr() : nullptr, (int32_t)zd,
                                   normed ? z.data_ptr() : nullptr, s), result);
  CATCH
}

// views(groups) -> (offsets, tiles, order, place) of groups whose buffer holds them
PyObject* views(PyObject*, PyObject* const* a, Py_ssize_t n) {
  TRY
  Groups g{};
  if (n != 1 || !groups_in(a[0], g) || !PyLong_Check(PyTuple_GET_ITEM(a[0], 6))) OTHERWISE;
  const at::Tensor& b = THPVariable_Unpack(PyTuple_GET_ITEM(a[0], 5));
  const int64_t base = (int64_t)(uintptr_t)b.storage().data();
  auto part = [&](int64_t p, at::IntArrayRef shape) { return THPVariable_Wrap(on(b, p - base, shape, ScalarType::Int)); };
  PyObject *off = part(g.offsets, {g.E + 1}), *til = part(g.tiles, {g.E + 1}), *order = part(g.order, {g.P}), *place = part(g.place, {g.T, g.k});
  return Py_BuildValue("(NNNN)", off, til, order, place);
  CATCH
}

PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 1) OTHERWISE;
  Py_INCREF(a[0]);
  Py_XDECREF(g_raise);
  g_raise = a[0];
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init), FAST(groups_of), FAST(rows_of), FAST(route), FAST(quantize), FAST(dequantize), FAST(matmul), FAST(matmul_fp4),
                         FAST(combine), FAST(blocks8), FAST(dequantize8), FAST(quantize_weights8), FAST(quantize8), FAST(matmul8), FAST(block_end), FAST(views), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operators", "the short way from torch tensors to the operators", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operators(void) { return PyModule_Create(&module); }
