// Python binding of the serving operators: checks torch tensors, allocates the outputs and workspaces and calls the C ABI
// (include/fa.h).  A call costs the host 5-10 us this way, most of them launches and allocations; the same steps through
// ctypes took 17-24 us, more than the kernels of a generation step.
//
// The module has no library of its own to link: `bind` hands it the addresses of libfa.so's functions.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/full.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <initializer_list>
#include <optional>

#include "fa.h"

namespace {

using at::Tensor;

struct Functions {
  decltype(&fa_rotary) rotary;
  decltype(&fa_paged_append) paged_append;
  decltype(&fa_paged_decode) paged_decode;
  decltype(&fa_paged_decode_workspace_size) paged_decode_workspace_size;
  decltype(&fa_pages_workspace_size) pages_workspace_size;
  decltype(&fa_pages_extend) pages_extend;
  decltype(&fa_pages_fork) pages_fork;
  decltype(&fa_pages_free) pages_free;
  decltype(&fa_pages_compact) pages_compact;
  decltype(&fa_pages_copy) pages_copy;
};
Functions lib = {};
PyObject* error_class = nullptr;   // FaError(code, where)

struct Failed {
  fa_status code;
  const char* where;
};
void check(fa_status code, const char* where) {
  if (code != FA_OK) throw Failed{code, where};
}
// The library wants one sequence at least; a call on none (and, decode, on no rows) gives empty outputs and does not reach it.

struct Unlocked {                  // the interpreter may run other threads while a call allocates and launches
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// ---------------------------------------------------------------- arguments
const Tensor* optional_tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, ": expected a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, ": expected a tensor");
  return THPVariable_Unpack(o);
}
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return x;
}
int integer(PyObject* o) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  TORCH_CHECK_VALUE(x == static_cast<int>(x), "an integer is out of range");
  return static_cast<int>(x);
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw python_error();
  return x != 0;
}
void arguments(Py_ssize_t have, Py_ssize_t want) {
  TORCH_CHECK_VALUE(have == want, "expected ", want, " arguments, got ", have);
}

// ---------------------------------------------------------------- checks
int extent(int64_t x) {
  TORCH_CHECK_VALUE(x <= INT32_MAX, "a size is beyond 2^31 - 1");
  return static_cast<int>(x);
}
void int32_tensor(const Tensor& t, const char* name, int dims) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.dim() == dims &&
                        (t.numel() <= 1 || t.size(-1) <= 1 || t.stride(-1) == 1),
                    name, ": expected a ", dims, "-D int32 tensor, contiguous in its last axis");
}
// [B, heads, rows, d], or, where `packed`, [rows, heads, d]; d contiguous.
void rows_tensor(const Tensor& t, const char* name, bool four, bool packed, bool f32) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kBFloat16 || (f32 && t.scalar_type() == at::kFloat), name,
                    ": unsupported dtype ", t.scalar_type());
  TORCH_CHECK_VALUE(((four && t.dim() == 4) || (packed && t.dim() == 3)) && (t.size(-1) <= 1 || t.stride(-1) == 1), name,
                    ": expected ", four ? "[B, heads, rows, d]" : "", four && packed ? " or " : "",
                    packed ? "packed [rows, heads, d]" : "", " with contiguous d");
}
fa_strides strides(const Tensor* t) {
  if (t == nullptr) return {0, 0, 0};
  const auto s = t->strides();
  return s.size() == 4 ? fa_strides{s[0], s[1], s[2]} : fa_strides{0, s[1], s[0]};
}
int frequencies(const Tensor& f) {
  TORCH_CHECK_VALUE(f.scalar_type() == at::kDouble && f.dim() == 1 && f.is_contiguous(),
                    "freqs: expected a contiguous 1-D float64 tensor (rotary_frequencies gives one)");
  return extent(2 * f.size(0));
}
template <typename T>
T* data(const Tensor* t) {
  return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
}
template <typename T>
T* data(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// The tensors' device made current, and its current stream.
struct Place {
  c10::cuda::OptionalCUDAGuard guard;
  cudaStream_t stream;
  explicit Place(std::initializer_list<const Tensor*> tensors) {
    int device = -1;
    for (const Tensor* t : tensors) {
      if (t == nullptr) continue;
      TORCH_CHECK_VALUE(t->is_cuda(), "expected a CUDA tensor: the library reads and writes device memory only");
      const int index = t->get_device();
      TORCH_CHECK_VALUE(device < 0 || index == device, "tensors on different devices: cuda:", device, " and cuda:", index);
      device = index;
    }
    guard.set_index(static_cast<c10::DeviceIndex>(device));
    stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  }
};

Tensor new_tensor(at::IntArrayRef size, at::ScalarType type, const Tensor& like) {
  return at::empty(size, at::TensorOptions().dtype(type).device(like.device()));
}
// The caller's workspace, or a new one.
Tensor workspace_of(const Tensor* given, size_t bytes, const Tensor& like) {
  TORCH_CHECK_VALUE(given == nullptr || given->is_contiguous(), "workspace: expected a contiguous tensor");
  return given != nullptr ? *given : new_tensor({static_cast<int64_t>(bytes)}, at::kByte, like);
}

// A new output for rows like x's: in x's order of axes, d contiguous (which it would not be beside rows or heads that
// overlap, one element apart).
Tensor rows_like(const Tensor& x) {
  Tensor y = at::empty_like(x);
  return y.size(-1) <= 1 || y.stride(-1) == 1 ? y : new_tensor(x.sizes(), x.scalar_type(), x);
}

PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* t = PyTuple_New(2);
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}
PyObject* wrap_or_none(std::optional<Tensor> t) {
  if (t) return wrap(std::move(*t));
  Py_RETURN_NONE;
}

// ---------------------------------------------------------------- rotary positions
// rotary(q, k, freqs, positions, interleaved, magnitude, out, inverse)
PyObject* rotary(PyObject* const* args, Py_ssize_t n) {
  arguments(n, 8);
  const Tensor& q = tensor(args[0], "q");
  const Tensor* k = optional_tensor(args[1], "k");
  const Tensor& freqs = tensor(args[2], "freqs");
  const Tensor* positions = optional_tensor(args[3], "positions");
  const double magnitude = number(args[5]);
  const bool inverse = truth(args[7]);
  rows_tensor(q, "q", true, true, true);
  const bool packed = q.dim() == 3;
  fa_rotary_layout L = {};
  L.rotary_dim = frequencies(freqs);
  L.B = packed ? 1 : extent(q.size(0));
  L.H = extent(q.size(1));
  L.N = extent(q.size(packed ? 0 : 2));
  L.d = extent(q.size(-1));
  L.interleaved = truth(args[4]);
  if (k != nullptr) {
    rows_tensor(*k, "k", !packed, packed, true);
    TORCH_CHECK_VALUE(k->scalar_type() == q.scalar_type(), "k: unsupported dtype ", k->scalar_type(), " beside q");
    TORCH_CHECK_VALUE(k->size(0) == q.size(0) && k->size(-1) == q.size(-1) && (packed || k->size(2) == q.size(2)),
                      "q and k: batch, rows and d must agree");
    L.H_kv = extent(k->size(1));
  }
  if (positions != nullptr) {
    const bool each = !packed && positions->dim() == 2;
    int32_tensor(*positions, "positions", each ? 2 : 1);
    TORCH_CHECK_VALUE(positions->size(-1) == L.N && (!each || positions->size(0) == L.B),
                      "positions: expected one per row ([rows] or [B, rows])");
    L.positions_batch = each ? positions->stride(0) : 0;
  }
  const Tensor *oq = nullptr, *ok = nullptr;
  if (args[6] != Py_None) {
    TORCH_CHECK_VALUE(PyTuple_Check(args[6]) && PyTuple_GET_SIZE(args[6]) == 2, "out: expected a pair (q, k)");
    oq = optional_tensor(PyTuple_GET_ITEM(args[6], 0), "out");
    ok = optional_tensor(PyTuple_GET_ITEM(args[6], 1), "out");
    auto fits = [&](const Tensor* x, const Tensor* y, const char* name) {
      TORCH_CHECK_VALUE((x == nullptr) == (y == nullptr) &&
                            (x == nullptr || (y->sizes() == x->sizes() && y->scalar_type() == x->scalar_type() &&
                                              (y->size(-1) <= 1 || y->stride(-1) == 1))),
                        "out: ", name, " must have its input's shape and dtype, d contiguous");
    };
    fits(&q, oq, "q");
    fits(k, ok, "k");
  }
  Tensor q_out;
  std::optional<Tensor> k_out;
  {
    Unlocked u;
    Place place({&q, k, &freqs, positions, oq, ok});
    q_out = oq != nullptr ? *oq : rows_like(q);
    if (k != nullptr) k_out = ok != nullptr ? *ok : rows_like(*k);
    L.q = strides(&q);
    L.k = strides(k);
    L.q_out = strides(&q_out);
    L.k_out = k_out ? strides(&*k_out) : fa_strides{0, 0, 0};
    if (L.B != 0)
      check(lib.rotary(data<void>(q), data<void>(k), data<void>(q_out), k_out ? data<void>(*k_out) : nullptr,
                       data<int32_t>(positions), data<double>(freqs), &L, static_cast<float>(magnitude), inverse,
                       q.scalar_type() == at::kBFloat16 ? FA_BF16 : FA_F32, place.stream),
            "fa_rotary");
  }
  if (oq != nullptr) {               // the caller's own tensors, not views of them
    PyObject *a = PyTuple_GET_ITEM(args[6], 0), *b = PyTuple_GET_ITEM(args[6], 1);
    Py_INCREF(a);
    Py_INCREF(b);
    return pair(a, b);
  }
  return pair(wrap(std::move(q_out)), wrap_or_none(std::move(k_out)));
}

// ---------------------------------------------------------------- the paged cache
void cache(const Tensor& kp, const Tensor& vp, fa_paged_layout* L) {
  rows_tensor(kp, "k_pages", true, false, false);
  rows_tensor(vp, "v_pages", true, false, false);
  TORCH_CHECK_VALUE(kp.sizes() == vp.sizes(), "k_pages and v_pages: one shape [pages, H_kv, page_size, d]");
  L->num_pages = extent(kp.size(0));
  L->H_kv = extent(kp.size(1));
  L->page_size = extent(kp.size(2));
  L->d = extent(kp.size(3));
  L->k_pages = strides(&kp);
  L->v_pages = strides(&vp);
}
void table(const Tensor& page_table, const Tensor& seq_lens) {
  int32_tensor(page_table, "page_table", 2);
  int32_tensor(seq_lens, "seq_lens", 1);
  TORCH_CHECK_VALUE(page_table.size(0) == seq_lens.size(0), "page_table, seq_lens and the batch must agree");
}
void table(const Tensor& page_table, const Tensor& seq_lens, int64_t batch, fa_paged_layout* L) {
  table(page_table, seq_lens);
  TORCH_CHECK_VALUE(batch == seq_lens.size(0), "page_table, seq_lens and the batch must agree");
  L->B = extent(batch);
  L->max_pages = extent(page_table.size(1));
  L->table_stride = page_table.stride(0);
}

// paged_append(k, v, k_pages, v_pages, page_table, seq_lens, q, freqs, interleaved, magnitude, cu_seqlens, out, tokens, status)
PyObject* paged_append(PyObject* const* args, Py_ssize_t n) {
  arguments(n, 14);
  const Tensor &k = tensor(args[0], "k"), &v = tensor(args[1], "v");
  const Tensor &kp = tensor(args[2], "k_pages"), &vp = tensor(args[3], "v_pages");
  const Tensor &pt = tensor(args[4], "page_table"), &lens = tensor(args[5], "seq_lens");
  const Tensor *q = optional_tensor(args[6], "q"), *freqs = optional_tensor(args[7], "freqs");
  const double magnitude = number(args[9]);
  const Tensor *cu = optional_tensor(args[10], "cu_seqlens"), *out = optional_tensor(args[11], "out");
  const Tensor *counts = optional_tensor(args[12], "tokens"), *status = optional_tensor(args[13], "status");
  const bool packed = cu != nullptr;
  fa_paged_layout L = {};
  cache(kp, vp, &L);
  for (const Tensor* t : {&k, &v}) {
    rows_tensor(*t, t == &k ? "k" : "v", !packed, packed, false);
    TORCH_CHECK_VALUE(t->size(1) == L.H_kv && t->size(-1) == L.d && t->sizes() == k.sizes(),
                      "k and v: heads and d as in the cache, one shape");
  }
  if (packed) {
    int32_tensor(*cu, "cu_seqlens", 1);
    TORCH_CHECK_VALUE(cu->size(0) >= 1, "cu_seqlens: expected B + 1 offsets");
  }
  table(pt, lens, packed ? cu->size(0) - 1 : k.size(0), &L);
  for (const Tensor* t : {counts, status}) {
    if (t == nullptr) continue;
    int32_tensor(*t, t == counts ? "tokens" : "status", 1);
    TORCH_CHECK_VALUE(t->size(0) == L.B, t == counts ? "tokens" : "status", ": expected one per sequence of the batch");
  }
  L.N = packed ? 0 : extent(k.size(2));
  L.total = packed ? extent(k.size(0)) : 0;
  if (q != nullptr) {
    rows_tensor(*q, "q", !packed, packed, false);
    TORCH_CHECK_VALUE(q->size(0) == k.size(0) && q->size(-1) == L.d && (packed || q->size(2) == k.size(2)),
                      "q and k: batch, rows and d must agree");
    L.H = extent(q->size(1));
  }
  L.rotary_dim = freqs == nullptr ? 0 : frequencies(*freqs);
  L.interleaved = truth(args[8]);
  TORCH_CHECK_VALUE(out == nullptr || (q != nullptr && out->sizes() == q->sizes() && out->scalar_type() == q->scalar_type() &&
                                       (out->size(-1) <= 1 || out->stride(-1) == 1)),
                    "out: must have q's shape and dtype, d contiguous");
  std::optional<Tensor> o;
  {
    Unlocked u;
    Place place({&k, &v, &kp, &vp, &pt, &lens, q, freqs, cu, out, counts, status});
    if (out != nullptr) o = *out;
    else if (q != nullptr) o = rows_like(*q);
    L.q = strides(q);
    L.o = o ? strides(&*o) : fa_strides{0, 0, 0};
    L.k = strides(&k);
    L.v = strides(&v);
    L.cu_seqlens = data<int32_t>(cu);
    L.tokens = data<int32_t>(counts);
    L.status = data<int32_t>(status);
    if (L.B != 0 || L.total != 0)
      check(lib.paged_append(data<void>(q), data<void>(k), data<void>(v), o ? data<void>(*o) : nullptr, data<void>(kp),
                             data<void>(vp), data<int32_t>(pt), data<int32_t>(lens), data<double>(freqs), &L,
                             static_cast<float>(magnitude), place.stream),
            "fa_paged_append");
  }
  if (out != nullptr) {
    Py_INCREF(args[11]);
    return args[11];
  }
  return wrap_or_none(std::move(o));
}

// paged_decode(q, k_pages, v_pages, page_table, seq_lens, causal, scale, workspace)
PyObject* paged_decode(PyObject* const* args, Py_ssize_t n) {
  arguments(n, 8);
  const Tensor &q = tensor(args[0], "q"), &kp = tensor(args[1], "k_pages"), &vp = tensor(args[2], "v_pages");
  const Tensor &pt = tensor(args[3], "page_table"), &lens = tensor(args[4], "seq_lens");
  const bool causal = truth(args[5]);
  const Tensor* given = optional_tensor(args[7], "workspace");
  fa_paged_layout L = {};
  cache(kp, vp, &L);
  rows_tensor(q, "q", true, false, false);
  TORCH_CHECK_VALUE(q.size(3) == L.d, "q and the cache: d must agree");
  table(pt, lens, q.size(0), &L);
  const double scale = args[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(L.d)) : number(args[6]);
  L.H = extent(q.size(1));
  L.N = extent(q.size(2));
  Tensor o, lse;
  {
    Unlocked u;
    Place place({&q, &kp, &vp, &pt, &lens, given});
    o = rows_like(q);
    lse = new_tensor({L.B, L.H, L.N}, at::kFloat, q);
    L.q = strides(&q);
    L.o = strides(&o);
    if (L.B != 0 && L.N != 0) {
      const Tensor ws = workspace_of(given, lib.paged_decode_workspace_size(&L), q);
      check(lib.paged_decode(data<void>(q), data<void>(kp), data<void>(vp), data<int32_t>(pt), data<int32_t>(lens),
                             data<void>(o), data<float>(lse), &L, static_cast<float>(scale), causal, data<void>(ws),
                             ws.nbytes(), place.stream),
            "fa_paged_decode");
    }
  }
  return pair(wrap(std::move(o)), wrap(std::move(lse)));
}

// ---------------------------------------------------------------- bookkeeping of pages
fa_pages_layout pages_state(const Tensor& pt, const Tensor& lens, const Tensor& refs, int page_size) {
  table(pt, lens);
  int32_tensor(refs, "refcounts", 1);
  fa_pages_layout L;
  L.num_seqs = extent(pt.size(0));
  L.num_pages = extent(refs.size(0));
  L.page_size = page_size;
  L.max_pages = extent(pt.size(1));
  L.table_stride = pt.stride(0);
  return L;
}
int requests(const Tensor& a, const char* name_a, const Tensor& b, const char* name_b) {
  int32_tensor(a, name_a, 1);
  int32_tensor(b, name_b, 1);
  TORCH_CHECK_VALUE(a.size(0) == b.size(0), name_a, " and ", name_b, ": one length");
  return extent(a.size(0));
}

// pages_extend(page_table, seq_lens, refcounts, page_size, seqs, tokens, workspace)
PyObject* pages_extend(PyObject* const* args, Py_ssize_t n) {
  arguments(n, 7);
  const Tensor &pt = tensor(args[0], "page_table"), &lens = tensor(args[1], "seq_lens"), &refs = tensor(args[2], "refcounts");
  const Tensor &seqs = tensor(args[4], "seqs"), &tokens = tensor(args[5], "tokens");
  const Tensor* given = optional_tensor(args[6], "workspace");
  const fa_pages_layout L = pages_state(pt, lens, refs, integer(args[3]));
  const int count = requests(seqs, "seqs", tokens, "tokens");
  Tensor status;
  {
    Unlocked u;
    Place place({&pt, &lens, &refs, &seqs, &tokens, given});
    status = new_tensor({count}, at::kInt, seqs);
    if (L.num_seqs != 0 || count != 0) {
      const Tensor ws = workspace_of(given, lib.pages_workspace_size(&L, count), seqs);
      check(lib.pages_extend(data<int32_t>(pt), data<int32_t>(lens), data<int32_t>(refs), &L, data<int32_t>(seqs),
                             data<int32_t>(tokens), count, data<int32_t>(status), data<void>(ws), ws.nbytes(), place.stream),
            "fa_pages_extend");
    }
  }
  return wrap(std::move(status));
}

// pages_fork(page_table, seq_lens, refcounts, page_size, src, dst, workspace)
PyObject* pages_fork(PyObject* const* args, Py_ssize_t n) {
  arguments(n, 7);
  const Tensor &pt = tensor(args[0], "page_table"), &lens = tensor(args[1], "seq_lens"), &refs = tensor(args[2], "refcounts");
  const Tensor &src = tensor(args[4], "src"), &dst = tensor(args[5], "dst");
  const Tensor* given = optional_tensor(args[6], "workspace");
  const fa_pages_layout L = pages_state(pt, lens, refs, integer(args[3]));
  const int count = requests(src, "src", dst, "dst");
  Tensor copies, status;
  {
    Unlocked u;
    Place place({&pt, &lens, &refs, &src, &dst, given});
    copies = new_tensor({count, 3}, at::kInt, src);
    status = new_tensor({count}, at::kInt, src);
    if (L.num_seqs != 0 || count != 0) {
      const Tensor ws = workspace_of(given, lib.pages_workspace_size(&L, count), src);
      check(lib.pages_fork(data<int32_t>(pt), data<int32_t>(lens), data<int32_t>(refs), &L, data<int32_t>(src),
                           data<int32_t>(dst), count, data<int32_t>(copies), data<int32_t>(status), data<void>(ws),
                           ws.nbytes(), place.stream),
            "fa_pages_fork");
    }
  }
  return pair(wrap(std::move(copies)), wrap(std::move(status)));
}

// pages_free(page_table, seq_lens, refcounts, page_size, seqs)
PyObject* pages_free(PyObject* const* args, Py_ssize_t n) {
  arguments(n, 5);
  const Tensor &pt = tensor(args[0], "page_table"), &lens = tensor(args[1], "seq_lens"), &refs = tensor(args[2], "refcounts");
  const Tensor& seqs = tensor(args[4], "seqs");
  const fa_pages_layout L = pages_state(pt, lens, refs, integer(args[3]));
  int32_tensor(seqs, "seqs", 1);
  {
    Unlocked u;
    Place place({&pt, &lens, &refs, &seqs});
    if (L.num_seqs != 0 || seqs.size(0) != 0)
      check(lib.pages_free(data<int32_t>(pt), data<int32_t>(lens), data<int32_t>(refs), &L, data<int32_t>(seqs),
                           extent(seqs.size(0)), place.stream),
            "fa_pages_free");
  }
  Py_RETURN_NONE;
}

// pages_compact(page_table, seq_lens, refcounts, page_size, workspace)
PyObject* pages_compact(PyObject* const* args, Py_ssize_t n) {
  arguments(n, 5);
  const Tensor &pt = tensor(args[0], "page_table"), &lens = tensor(args[1], "seq_lens"), &refs = tensor(args[2], "refcounts");
  const Tensor* given = optional_tensor(args[4], "workspace");
  const fa_pages_layout L = pages_state(pt, lens, refs, integer(args[3]));
  Tensor copies;
  {
    Unlocked u;
    Place place({&pt, &lens, &refs, given});
    if (L.num_seqs == 0) {
      copies = at::full({L.num_pages / 2, 3}, -1, refs.options());
    } else {
      copies = new_tensor({L.num_pages / 2, 3}, at::kInt, refs);
      const Tensor ws = workspace_of(given, lib.pages_workspace_size(&L, 0), refs);
      check(lib.pages_compact(data<int32_t>(pt), data<int32_t>(lens), data<int32_t>(refs), &L, data<int32_t>(copies),
                              data<void>(ws), ws.nbytes(), place.stream),
            "fa_pages_compact");
    }
  }
  return wrap(std::move(copies));
}

// pages_copy(k_pages, v_pages, copies)
PyObject* pages_copy(PyObject* const* args, Py_ssize_t n) {
  arguments(n, 3);
  const Tensor &kp = tensor(args[0], "k_pages"), &vp = tensor(args[1], "v_pages"), &copies = tensor(args[2], "copies");
  fa_paged_layout L = {};
  cache(kp, vp, &L);
  int32_tensor(copies, "copies", 2);
  TORCH_CHECK_VALUE(copies.size(1) == 3 && copies.is_contiguous(), "copies: expected a contiguous [n, 3] tensor");
  L.B = 1;
  {
    Unlocked u;
    Place place({&kp, &vp, &copies});
    check(lib.pages_copy(data<void>(kp), data<void>(vp), data<int32_t>(copies), extent(copies.size(0)), &L, place.stream),
          "fa_pages_copy");
  }
  Py_RETURN_NONE;
}

// ---------------------------------------------------------------- module
// bind(error class, ten addresses in the order of Functions)
PyObject* bind(PyObject* const* args, Py_ssize_t n) {
  constexpr int count = sizeof(Functions) / sizeof(void*);
  arguments(n, 1 + count);
  void* at[count];
  for (int i = 0; i < count; ++i) {
    at[i] = PyLong_AsVoidPtr(args[1 + i]);
    if (at[i] == nullptr) throw python_error();
  }
  static_assert(sizeof(at) == sizeof(Functions), "one address per function");
  std::memcpy(&lib, at, sizeof(at));
  Py_INCREF(args[0]);
  Py_XDECREF(error_class);
  error_class = args[0];
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Failed& f) {
    if (PyObject* e = PyObject_CallFunction(error_class, "is", static_cast<int>(f.code), f.where)) {
      PyErr_SetObject(error_class, e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<bind>("bind"),
                         method<rotary>("rotary"),
                         method<paged_append>("paged_append"),
                         method<paged_decode>("paged_decode"),
                         method<pages_extend>("pages_extend"),
                         method<pages_fork>("pages_fork"),
                         method<pages_free>("pages_free"),
                         method<pages_compact>("pages_compact"),
                         method<pages_copy>("pages_copy"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&module); }
