// binding.cpp -- argument checks and outputs of the trees' and pages' calls (tree.py,
// and the later half of kv.py).  They are one launch long, or few: in Python their
// checks and outputs took 6 to 15 us of the host's time on the GPU's host (the tree's
// attention 23), which is more than the launches do on the GPU; here they take 2 to 7
// (the attention 9 to 12), 1.1 of it for each result.
//
// The module knows the library by the addresses that bind() is given (it is not
// linked to it).  Every function takes its arguments in a fixed order, works on the
// tensors' device and on that device's current stream, and raises what the other
// calls of the binding raise: TypeError for a wrong type, ValueError for a wrong
// shape, layout or device, SpecError for what the library refuses.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstring>
#include <initializer_list>
#include <string>

#include "spec_kv.h"
#include "spec_tree.h"

namespace {

using at::Tensor;

struct Library {
  decltype(&spec_status_string) status_string;
  decltype(&spec_tree_mask) tree_mask;
  decltype(&spec_tree_accept) tree_accept;
  decltype(&spec_adjust) adjust;
  decltype(&spec_kv_compact) compact;
  decltype(&spec_kv_copy) copy;
  decltype(&spec_kv_resize) resize;
  decltype(&spec_kv_fork) fork;
  decltype(&spec_attend_tree_workspace_size) attend_size;
  decltype(&spec_attend_tree) attend;
} lib;
PyObject *spec_error = nullptr;

struct Raised {};  // a Python error is set

[[noreturn]] void fail(PyObject *type, const char *fmt, ...) {
  va_list args;
  va_start(args, fmt);
  PyErr_FormatV(type, fmt, args);
  va_end(args);
  throw Raised();
}

std::string text(at::IntArrayRef sizes) {
  std::string s = "[";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + "]";
}

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// A contiguous tensor of this type and shape on the device.
const void *table(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef sizes, at::Device dev) {
  const Tensor &t = tensor(o, name);
  if (t.scalar_type() != type) fail(PyExc_TypeError, "%s must be %s", name, type == at::kInt ? "int32" : "float32");
  if (t.sizes() != sizes || t.device() != dev || !t.is_contiguous())
    fail(PyExc_ValueError, "%s must be contiguous %s on %s", name, text(sizes).c_str(), dev.str().c_str());
  return t.const_data_ptr();
}
const int32_t *ints(PyObject *o, const char *name, at::IntArrayRef sizes, at::Device dev) {
  return static_cast<const int32_t *>(table(o, name, at::kInt, sizes, dev));
}
int32_t *ints_out(PyObject *o, const char *name, at::IntArrayRef sizes, at::Device dev) {
  return const_cast<int32_t *>(ints(o, name, sizes, dev));
}
// The same for what may be None.
const int32_t *ints_or_none(PyObject *o, const char *name, at::IntArrayRef sizes, at::Device dev) {
  return o == Py_None ? nullptr : ints(o, name, sizes, dev);
}
const float *floats_or_none(PyObject *o, const char *name, at::IntArrayRef sizes, at::Device dev) {
  return o == Py_None ? nullptr : static_cast<const float *>(table(o, name, at::kFloat, sizes, dev));
}

int32_t number(PyObject *o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised();
  if (x < INT32_MIN || x > INT32_MAX) fail(PyExc_OverflowError, "%lld does not fit 32 bits", x);
  return static_cast<int32_t>(x);
}
bool truth(PyObject *o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised();
  return x;
}
int32_t size32(int64_t n) {
  if (n > INT32_MAX) fail(PyExc_ValueError, "%lld elements on an axis are too many", static_cast<long long>(n));
  return static_cast<int32_t>(n);
}

// The device of a call, current while it lasts, and its stream.
struct On {
  at::Device dev;
  c10::cuda::OptionalCUDAGuard guard;
  explicit On(at::Device d) : dev(d) {
    if (!d.is_cuda()) fail(spec_error, "the tensors are on %s: this library has no CPU path", d.str().c_str());
    guard.set_index(d.index());
  }
  void *stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
  Tensor empty(at::IntArrayRef sizes, at::ScalarType type = at::kInt) const {
    return at::detail::empty_cuda(sizes, type, dev, std::nullopt);
  }
};

// f() without the interpreter's lock: it raises nothing itself.
template <class F>
void call(F f) {
  PyThreadState *thread = PyEval_SaveThread();
  const spec_status code = f();
  PyEval_RestoreThread(thread);
  if (code != SPEC_OK) fail(spec_error, "%s", lib.status_string(code));
}

int32_t *out(const Tensor &t) { return t.defined() ? static_cast<int32_t *>(t.mutable_data_ptr()) : nullptr; }

// One object for one result, a tuple for several; what is not defined is left out.
PyObject *results(std::initializer_list<Tensor> all) {
  Py_ssize_t n = 0;
  for (const Tensor &t : all) n += t.defined();
  if (n == 0) Py_RETURN_NONE;
  if (n == 1)
    for (const Tensor &t : all)
      if (t.defined()) return THPVariable_Wrap(t);
  PyObject *tuple = PyTuple_New(n);
  if (!tuple) throw Raised();
  Py_ssize_t i = 0;
  for (const Tensor &t : all)
    if (t.defined()) {
      PyObject *o = THPVariable_Wrap(t);
      if (!o) {
        Py_DECREF(tuple);
        throw Raised();
      }
      PyTuple_SET_ITEM(tuple, i++, o);
    }
  return tuple;
}

// ------------------------------------------------------------------- trees
// parents, gamma_per_row, with_status
PyObject *tree_mask(PyObject *const *a) {
  const Tensor &parents = tensor(a[0], "parents");
  if (parents.dim() != 2) fail(PyExc_ValueError, "parents must be [B, gamma_max]");
  const at::Device dev = parents.device();
  const int32_t B = size32(parents.size(0)), G = size32(parents.size(1));
  const int64_t N = static_cast<int64_t>(G) + 1;
  const int32_t *up = ints(a[0], "parents", {B, G}, dev), *gam = ints_or_none(a[1], "gamma_per_row", {B}, dev);
  const On on(dev);
  const Tensor mask = on.empty({B, N, (N + 31) / 32}), depth = on.empty({B, N}), st = truth(a[2]) ? on.empty({B}) : Tensor();
  void *const stream = on.stream();
  call([&] { return lib.tree_mask(B, G, up, gam, out(mask), out(depth), out(st), stream); });
  return results({mask, depth, st});
}

// target_tokens, draft_tokens, parents, gamma_per_row, with_status
PyObject *tree_accept(PyObject *const *a) {
  const Tensor &target = tensor(a[0], "target_tokens");
  if (target.dim() != 2 || target.size(1) < 1) fail(PyExc_ValueError, "target_tokens must be [B, gamma_max + 1]");
  const at::Device dev = target.device();
  const int32_t B = size32(target.size(0)), N = size32(target.size(1));
  const int32_t *tgt = ints(a[0], "target_tokens", {B, N}, dev), *tok = ints(a[1], "draft_tokens", {B, N - 1}, dev);
  const int32_t *up = ints(a[2], "parents", {B, N - 1}, dev), *gam = ints_or_none(a[3], "gamma_per_row", {B}, dev);
  const On on(dev);
  const Tensor acc = on.empty({B}), next = on.empty({B}), path = on.empty({B, N}), tokens = on.empty({B, N - 1});
  const Tensor st = truth(a[4]) ? on.empty({B}) : Tensor();
  void *const stream = on.stream();
  call([&] { return lib.tree_accept(B, N - 1, tgt, tok, up, gam, out(acc), out(next), out(path), out(tokens), out(st), stream); });
  return results({acc, next, path, tokens, st});
}

// logits, seq, seq_len, draft_tokens, tree_mask, prompt_len, repetition, presence, frequency, bias_ids, bias, allowed,
// gamma_per_row, out, with_status
PyObject *adjust(PyObject *const *a) {
  const Tensor &logits = tensor(a[0], "logits");
  const at::Device dev = logits.device();
  if (logits.dim() != 3 || logits.size(1) < 1 || logits.size(2) < 1)
    fail(PyExc_ValueError, "logits must be [B, gamma_max + 1, V]");
  const at::ScalarType type = logits.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) fail(PyExc_TypeError, "logits must be float32 or bfloat16");
  const int64_t B = logits.size(0), N = logits.size(1), V = logits.size(2);
  if (V > 1 && logits.stride(2) != 1) fail(PyExc_ValueError, "the vocabulary axis must be contiguous");
  Tensor to;
  if (a[13] != Py_None) {
    to = tensor(a[13], "out");
    if (to.sizes() != logits.sizes() || to.scalar_type() != type || to.device() != dev || (V > 1 && to.stride(2) != 1))
      fail(PyExc_ValueError, "out must be of the logits' shape, type and device, its vocabulary axis contiguous");
  }
  const Tensor &seq = tensor(a[1], "seq");
  if (seq.scalar_type() != at::kInt) fail(PyExc_TypeError, "seq must be int32");
  if (seq.dim() != 2 || seq.size(0) != B || seq.device() != dev || (B && seq.size(1) > 1 && seq.stride(1) != 1))
    fail(PyExc_ValueError, "seq must be [%lld, capacity] on %s with contiguous rows", static_cast<long long>(B),
         dev.str().c_str());
  if (N > 1 && a[3] == Py_None) fail(PyExc_ValueError, "draft_tokens must be given where there are drafts");
  if ((a[9] == Py_None) != (a[10] == Py_None)) fail(PyExc_ValueError, "bias_ids and bias go together");
  spec_adjust_params p = {};
  p.B = size32(B), p.gamma_max = size32(N - 1), p.V = size32(V);
  p.dtype = type == at::kFloat ? SPEC_F32 : SPEC_BF16;
  p.capacity = size32(seq.size(1));
  p.logits_row_stride = logits.stride(0), p.logits_pos_stride = logits.stride(1);
  p.seq_row_stride = B > 1 ? seq.stride(0) : seq.size(1);
  p.seq = static_cast<const int32_t *>(seq.const_data_ptr());
  p.seq_len = ints(a[2], "seq_len", {B}, dev);
  p.draft_tokens = ints_or_none(a[3], "draft_tokens", {B, N - 1}, dev);
  p.tree_mask = ints_or_none(a[4], "tree_mask", {B, N, (N + 31) / 32}, dev);
  p.prompt_len = ints_or_none(a[5], "prompt_len", {B}, dev);
  p.repetition = floats_or_none(a[6], "repetition", {B}, dev);
  p.presence = floats_or_none(a[7], "presence", {B}, dev);
  p.frequency = floats_or_none(a[8], "frequency", {B}, dev);
  if (a[10] != Py_None) {
    const Tensor &bias = tensor(a[10], "bias");
    const int64_t n = bias.dim() == 2 ? bias.size(1) : -1;
    p.bias = floats_or_none(a[10], "bias", {B, n}, dev);
    p.bias_ids = ints(a[9], "bias_ids", {B, n}, dev);
    p.n_bias = size32(n);
  }
  if (a[11] != Py_None) {
    const Tensor &w = tensor(a[11], "allowed");
    const int64_t n = (V + 31) / 32;
    if (w.scalar_type() != at::kInt) fail(PyExc_TypeError, "allowed must be int32");
    if (w.sizes() != at::IntArrayRef({B, N, n}) || w.device() != dev || (n > 1 && w.stride(2) != 1))
      fail(PyExc_ValueError, "allowed must be %s on %s with contiguous words", text({B, N, n}).c_str(), dev.str().c_str());
    p.allowed = static_cast<const int32_t *>(w.const_data_ptr());
    p.allowed_row_stride = w.stride(0), p.allowed_pos_stride = w.stride(1);
  }
  p.gamma_per_row = ints_or_none(a[12], "gamma_per_row", {B}, dev);
  const On on(dev);
  if (!to.defined()) to = on.empty({B, N, V}, type);
  p.out_row_stride = to.stride(0), p.out_pos_stride = to.stride(1);
  const Tensor st = truth(a[14]) ? on.empty({B}) : Tensor();
  void *const stream = on.stream();
  call([&] { return lib.adjust(logits.const_data_ptr(), &p, to.mutable_data_ptr(), out(st), stream); });
  return results({to, st});
}

// ------------------------------------------------------------------- pages
const spec_kv_cache *cache_of(PyObject *address) {
  void *p = PyLong_AsVoidPtr(address);
  if (!p && PyErr_Occurred()) throw Raised();
  return static_cast<const spec_kv_cache *>(p);
}

// A page table [B, max_pages] whose rows are contiguous: its row stride.
int64_t page_table(const Tensor &t, int64_t B, at::Device dev) {
  if (t.scalar_type() != at::kInt) fail(PyExc_TypeError, "page_table must be int32");
  if (t.dim() != 2 || t.device() != dev || (B >= 0 && t.size(0) != B)) fail(PyExc_ValueError, "page_table must be [B, max_pages] on %s", dev.str().c_str());
  const int64_t rows = t.size(0), wide = t.size(1);
  if ((rows && wide > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < wide))
    fail(PyExc_ValueError, "page_table rows must be contiguous and not overlap");
  return rows > 1 ? t.stride(0) : wide;
}

// the cache's address, its k_pages, page_table, kv_len, path, accepted_len, prefix_len, with_status
PyObject *compact(PyObject *const *a) {
  const at::Device dev = tensor(a[1], "k_pages").device();
  const Tensor &lens = tensor(a[3], "kv_len"), &path = tensor(a[4], "path"), &pages = tensor(a[2], "page_table");
  const int64_t B = lens.dim() == 1 ? lens.size(0) : -1, N = path.dim() == 2 ? path.size(1) : 0;
  if (B < 0) fail(PyExc_ValueError, "kv_len must be [B]");
  if (path.scalar_type() != at::kInt) fail(PyExc_TypeError, "path must be int32");
  if (N < 1) fail(PyExc_ValueError, "path must be contiguous [%lld, gamma_max + 1]", static_cast<long long>(B));
  spec_kv_batch b = {};
  b.table_row_stride = page_table(pages, B, dev);
  b.B = size32(B), b.gamma_max = size32(N - 1), b.max_pages = size32(pages.size(1));
  b.prefix_len = number(a[6]);
  b.page_table = static_cast<const int32_t *>(pages.const_data_ptr());
  b.kv_len = ints(a[3], "kv_len", {B}, dev);
  // not read, the step is past the prefix; a table without columns has no address
  b.prefix_table = b.prefix_len > 0 ? b.kv_len : nullptr;
  const int32_t *way = ints(a[4], "path", {B, N}, dev), *acc = ints(a[5], "accepted_len", {B}, dev);
  const spec_kv_cache *cache = cache_of(a[0]);
  const On on(dev);
  const Tensor st = truth(a[7]) ? on.empty({B}) : Tensor();
  void *const stream = on.stream();
  call([&] { return lib.compact(cache, &b, way, acc, out(st), stream); });
  return results({st});
}

// the cache's address, its k_pages, copies
PyObject *copy(PyObject *const *a) {
  const at::Device dev = tensor(a[1], "k_pages").device();
  const Tensor &copies = tensor(a[2], "copies");
  const int32_t n = copies.dim() == 2 ? size32(copies.size(0)) : -1;
  const int32_t *rows = ints(a[2], "copies", {n, 3}, dev);
  const spec_kv_cache *cache = cache_of(a[0]);
  const On on(dev);
  void *const stream = on.stream();
  call([&] { return lib.copy(cache, rows, n, stream); });
  Py_RETURN_NONE;
}

// refs, page_table, held, page_size, prefix_len
spec_kv_pool pool(PyObject *refs, PyObject *pages, PyObject *held, PyObject *page_size, PyObject *prefix, at::Device &dev) {
  const Tensor &r = tensor(refs, "refs"), &t = tensor(pages, "page_table");
  dev = r.device();
  spec_kv_pool p = {};
  p.refs = ints_out(refs, "refs", {r.numel()}, dev);
  p.n_pages = size32(r.numel());
  p.table_row_stride = page_table(t, -1, dev);
  p.B = size32(t.size(0)), p.max_pages = size32(t.size(1));
  p.table = static_cast<int32_t *>(t.mutable_data_ptr());
  p.held = ints_out(held, "held", {t.size(0)}, dev);
  p.page_size = number(page_size), p.prefix_len = number(prefix);
  return p;
}

// refs, page_table, held, kv_len, n_step, page_size, prefix_len, with_status
PyObject *resize(PyObject *const *a) {
  at::Device dev(at::kCPU);
  const spec_kv_pool p = pool(a[0], a[1], a[2], a[5], a[6], dev);
  const int32_t *lens = ints(a[3], "kv_len", {p.B}, dev), n = number(a[4]);
  const On on(dev);
  const Tensor st = truth(a[7]) ? on.empty({p.B}) : Tensor();
  void *const stream = on.stream();
  call([&] { return lib.resize(&p, lens, n, out(st), stream); });
  return results({st});
}

// refs, page_table, held, kv_len, src, dst, page_size, prefix_len, with_status
PyObject *fork(PyObject *const *a) {
  at::Device dev(at::kCPU);
  const spec_kv_pool p = pool(a[0], a[1], a[2], a[6], a[7], dev);
  int32_t *lens = ints_out(a[3], "kv_len", {p.B}, dev);
  const int32_t n = size32(tensor(a[4], "src").numel());
  const int32_t *src = ints(a[4], "src", {n}, dev), *dst = ints(a[5], "dst", {n}, dev);
  const On on(dev);
  const Tensor copies = on.empty({n, 3}), st = truth(a[8]) ? on.empty({n}) : Tensor();
  void *const stream = on.stream();
  call([&] { return lib.fork(&p, lens, src, dst, n, out(copies), out(st), stream); });
  return results({copies, st});
}

// --------------------------------------------------------------- attention
// the cache's address, its k_pages, q, page_table, kv_len, mask, prefix_table, prefix_len, gamma_per_row, scale,
// workspace, out, with_status
PyObject *attend_tree(PyObject *const *a) {
  const at::Device dev = tensor(a[1], "k_pages").device();
  const spec_kv_cache *cache = cache_of(a[0]);
  const Tensor &q = tensor(a[2], "q"), &pages = tensor(a[3], "page_table"), &lens = tensor(a[4], "kv_len");
  if (q.scalar_type() != at::kBFloat16) fail(PyExc_TypeError, "q must be bfloat16");
  const int64_t D = cache->head_dim;
  if (q.dim() != 4 || lens.dim() != 1 || q.size(0) != lens.size(0) || q.size(1) < 1 || q.size(3) != D)
    fail(PyExc_ValueError, "q must be [B, gamma_max + 1, n_heads, head_dim]");
  if (q.device() != dev) fail(PyExc_ValueError, "q must be on %s", dev.str().c_str());
  if (D > 1 && q.stride(3) != 1) fail(PyExc_ValueError, "the head_dim axis must be contiguous");
  const int64_t B = q.size(0), N = q.size(1);
  const int32_t Hq = size32(q.size(2));
  if (cache->n_kv_heads < 1 || cache->page_size < 1) fail(PyExc_ValueError, "the cache's pages must hold a head and a slot at least");
  if (Hq < 1 || Hq % cache->n_kv_heads) fail(PyExc_ValueError, "n_heads must be a multiple of the cache's n_kv_heads");
  spec_kv_batch b = {};
  b.table_row_stride = page_table(pages, B, dev);
  b.B = size32(B), b.gamma_max = size32(N - 1), b.max_pages = size32(pages.size(1));
  b.prefix_len = number(a[7]);
  b.page_table = static_cast<const int32_t *>(pages.const_data_ptr());
  b.kv_len = ints(a[4], "kv_len", {B}, dev);
  b.gamma_per_row = ints_or_none(a[8], "gamma_per_row", {B}, dev);
  if (b.prefix_len > 0) {
    const int64_t need = (static_cast<int64_t>(b.prefix_len) + cache->page_size - 1) / cache->page_size;
    const int64_t n = a[6] == Py_None ? -1 : tensor(a[6], "prefix_table").numel();
    if (n < need) fail(PyExc_ValueError, "prefix_table must hold the prefix's %lld page ids", static_cast<long long>(need));
    b.prefix_table = ints(a[6], "prefix_table", {n}, dev);
  }
  const int32_t *mask = ints(a[5], "mask", {B, N, (N + 31) / 32}, dev);
  const float scale = a[9] == Py_None ? static_cast<float>(std::pow(static_cast<double>(D), -0.5))
                                      : static_cast<float>(PyFloat_AsDouble(a[9]));
  if (PyErr_Occurred()) throw Raised();
  const On on(dev);
  Tensor work;
  if (PyUnicode_Check(a[10])) {
    if (PyUnicode_CompareWithASCIIString(a[10], "auto")) fail(PyExc_ValueError, "workspace must be 'auto' or a tensor");
    work = on.empty({static_cast<int64_t>(lib.attend_size(cache, &b, Hq))}, at::kByte);
  } else {
    if (a[10] == Py_None || tensor(a[10], "workspace").device() != dev || !THPVariable_Unpack(a[10]).is_contiguous())
      fail(PyExc_ValueError, "workspace must be 'auto' or a contiguous tensor on %s", dev.str().c_str());
    work = THPVariable_Unpack(a[10]);
  }
  Tensor o, lse;
  if (a[11] == Py_None) {
    o = on.empty({B, N, Hq, D}, at::kBFloat16);
    lse = on.empty({B, N, Hq}, at::kFloat);
  } else {
    const bool list = PyList_Check(a[11]);
    if (!(list || PyTuple_Check(a[11])) || PySequence_Size(a[11]) != 2) fail(PyExc_TypeError, "out must be a pair of tensors");
    o = tensor(list ? PyList_GET_ITEM(a[11], 0) : PyTuple_GET_ITEM(a[11], 0), "out");
    lse = tensor(list ? PyList_GET_ITEM(a[11], 1) : PyTuple_GET_ITEM(a[11], 1), "out");
    if (o.sizes() != q.sizes() || o.scalar_type() != at::kBFloat16 || !o.is_contiguous() ||
        lse.sizes() != at::IntArrayRef({B, N, Hq}) || lse.scalar_type() != at::kFloat || !lse.is_contiguous() ||
        o.device() != dev || lse.device() != dev)
      fail(PyExc_ValueError, "out must be contiguous bfloat16 and float32 tensors of the results' shapes");
  }
  const Tensor st = truth(a[12]) ? on.empty({B}) : Tensor();
  const int64_t strides[3] = {q.stride(0), q.stride(1), q.stride(2)};
  void *const stream = on.stream();
  call([&] {
    return lib.attend(cache, &b, mask, q.const_data_ptr(), Hq, strides, scale, o.mutable_data_ptr(),
                      static_cast<float *>(lse.mutable_data_ptr()), out(st), work.mutable_data_ptr(), work.nbytes(), stream);
  });
  return results({o, lse, st});
}

// ------------------------------------------------------------------ module
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", N, n);
    return nullptr;
  }
  if (!spec_error) {
    PyErr_SetString(PyExc_RuntimeError, "bind() comes first");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// SpecError, then the functions' addresses in the order of Library
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *f[sizeof(Library) / sizeof(void *)];
  constexpr Py_ssize_t count = sizeof(f) / sizeof(f[0]);
  if (n != count + 1) {
    PyErr_SetString(PyExc_TypeError, "SpecError and an address for each function");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < count; ++i) {
    f[i] = PyLong_AsVoidPtr(args[i + 1]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function has no address");
      return nullptr;
    }
  }
  memcpy(&lib, f, sizeof lib);
  Py_INCREF(args[0]);
  Py_XDECREF(spec_error);
  spec_error = args[0];
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"tree_mask", fast(entry<tree_mask, 3>), METH_FASTCALL, nullptr},
                         {"tree_accept", fast(entry<tree_accept, 5>), METH_FASTCALL, nullptr},
                         {"adjust", fast(entry<adjust, 15>), METH_FASTCALL, nullptr},
                         {"compact", fast(entry<compact, 8>), METH_FASTCALL, nullptr},
                         {"copy", fast(entry<copy, 3>), METH_FASTCALL, nullptr},
                         {"resize", fast(entry<resize, 8>), METH_FASTCALL, nullptr},
                         {"fork", fast(entry<fork, 9>), METH_FASTCALL, nullptr},
                         {"attend_tree", fast(entry<attend_tree, 13>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
