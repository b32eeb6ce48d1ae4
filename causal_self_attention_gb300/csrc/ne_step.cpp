// ne_step.cpp -- the calls of a generation step from Python: checks of the arguments,
// outputs, the library's entry point, in one native call (the module `ne_step`, which
// ne_attn.py goes through).
//
// What it is for: these calls' kernels take 2 to 20 us, and marshalling them in Python took
// as long or longer (64 rows of norms: 1.5 us of kernel, 15 us of call; 6 to 9 us this way, by
// the host's state, two outputs' allocation among them).
//
// The regular call is made here: plain tensors on the current device, its current stream,
// the library's own workspace.  Anything else -- an argument of another type or shape,
// another device, no rows -- returns None before anything is done, and ne_attn.py goes on
// with it: that is where what is wrong is said.  What the library refuses comes back as its
// status.
#include <Python.h>

#include <climits>
#include <initializer_list>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ne_attn.h"

namespace {
using at::Tensor;
constexpr at::ScalarType kBf16 = at::kBFloat16, kE4m3 = at::kFloat8_e4m3fn, kI32 = at::kInt,
                         kU8 = at::kByte, kF32 = at::kFloat;
constexpr int kDim = 64;

// The library's entry points, given by bind().
struct {
  decltype(&ne_qk_norm_rope_fwd) norm_fwd;
  decltype(&ne_qk_norm_rope_bwd) norm_bwd;
  decltype(&ne_kv_reserve) reserve;
  decltype(&ne_kv_release) release;
  decltype(&ne_kv_append) append;
  decltype(&ne_kv_read) read;
  decltype(&ne_attn_decode_paged) decode;
} lib;

bool as_int(PyObject* o, int& v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long x = PyLong_AsLongAndOverflow(o, &over);
  if (over || x < INT_MIN || x > INT_MAX) return false;
  v = static_cast<int>(x);
  return true;
}
bool as_float(PyObject* o, float& v) {
  int i;
  if (PyFloat_CheckExact(o))
    v = static_cast<float>(PyFloat_AS_DOUBLE(o));
  else if (as_int(o, i))
    v = static_cast<float>(i);
  else
    return false;
  return true;
}

// The tensors of a call, which are on one device.
class Call {
 public:
  // A dense contiguous tensor of a type, with the sizes given (-1: any); nullptr if not.
  const Tensor* get(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> sizes) {
    const Tensor* t = dense(o, type);
    return t && t->is_contiguous() && has(*t, sizes) ? t : nullptr;
  }
  // The same where it may be None: false if it is neither.
  bool maybe(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> sizes,
             const Tensor*& t) {
    t = nullptr;
    return o == Py_None || (t = get(o, type, sizes)) != nullptr;
  }
  // Rows [n, heads, 64] bf16 whose heads are contiguous, `row` elements apart.
  const Tensor* rows(PyObject* o, int64_t& row) {
    const Tensor* t = dense(o, kBf16);
    if (!t || !has(*t, {-1, -1, kDim}) || t->stride(2) != 1) return nullptr;
    if (t->size(1) > 1 && t->stride(1) != kDim) return nullptr;
    row = t->size(0) > 1 ? t->stride(0) : kDim * t->size(1);
    return t;
  }
  // Whether the call's device is the current one (which stays as it is).
  bool current() const { return dev_ >= 0 && c10::cuda::current_device() == dev_; }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev_).stream(); }

 private:
  const Tensor* dense(PyObject* o, at::ScalarType type) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || t.scalar_type() != type || !t.has_storage())
      return nullptr;  // (a tensor that stands for others has no storage)
    if (dev_ < 0) dev_ = t.get_device();
    return t.get_device() == dev_ ? &t : nullptr;
  }
  static bool has(const Tensor& t, std::initializer_list<int64_t> sizes) {
    if (t.dim() != static_cast<int64_t>(sizes.size())) return false;
    int i = 0;
    for (const int64_t want : sizes) {
      const int64_t s = t.size(i++);
      if (s > INT_MAX || (want >= 0 && s != want)) return false;
    }
    return true;
  }
  int dev_ = -1;
};

Tensor output(const Tensor* given, at::IntArrayRef sizes, at::ScalarType type, const Tensor& like) {
  return given ? *given : at::empty(sizes, like.options().dtype(type));
}
void* at_(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
int len(const Tensor* t, int dim) { return static_cast<int>(t->size(dim)); }

// The tensors as a tuple, or the library's status.
PyObject* result(ne_status rc, std::initializer_list<Tensor> out) {
  if (rc != NE_OK) return PyLong_FromLong(rc);
  PyObject* all = PyTuple_New(static_cast<Py_ssize_t>(out.size()));
  if (!all) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : out) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(all);
      return nullptr;
    }
    PyTuple_SET_ITEM(all, i++, o);
  }
  return all;
}

// Calls the library without the interpreter's lock, as ctypes does (and has it again
// whichever way the call ends).  The arguments come by value: addresses, sizes and the stream
// are read under the lock, where the checks were made, and another thread that gives a tensor
// other memory meanwhile changes nothing of this call.
template <typename... Wanted, typename... Given>
ne_status unlocked(ne_status (*call)(Wanted...), Given... given) {
  static_assert(sizeof...(Wanted) == sizeof...(Given), "");
  struct Lock {
    PyThreadState* state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return call(given...);
}

// What the norms' two directions share.
struct Norm {
  Call c;
  const Tensor *q, *k, *qw, *kw, *pos;
  int64_t q_row, k_row;
  int n, H, Hkv, max_seqlen;
  float eps, base;

  // a: q, k, q_weight, k_weight, positions, max_seqlen, eps, rope_base
  bool parse(PyObject* const* a) {
    if (!(q = c.rows(a[0], q_row)) || !(k = c.rows(a[1], k_row)) || q->size(0) != k->size(0) ||
        q->size(0) == 0)
      return false;
    n = len(q, 0);
    H = len(q, 1);
    Hkv = len(k, 1);
    return (qw = c.get(a[2], kBf16, {kDim})) && (kw = c.get(a[3], kBf16, {kDim})) &&
           c.maybe(a[4], kI32, {n}, pos) && as_int(a[5], max_seqlen) && as_float(a[6], eps) &&
           as_float(a[7], base) && (pos || base == 0.f);
  }
};

// q, k, q_weight, k_weight, positions, max_seqlen, eps, rope_base, qr, kr
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Norm m;
  const Tensor *gq, *gk;
  if (n != 10 || !m.parse(a) || !m.c.maybe(a[8], kBf16, {m.n, m.H, kDim}, gq) ||
      !m.c.maybe(a[9], kBf16, {m.n, m.Hkv, kDim}, gk) || !m.c.current())
    Py_RETURN_NONE;
  const Tensor qr = output(gq, m.q->sizes(), kBf16, *m.q), kr = output(gk, m.k->sizes(), kBf16, *m.k);
  const ne_status rc = unlocked(lib.norm_fwd, static_cast<const ne_bf16*>(at_(m.q)),
      static_cast<const ne_bf16*>(at_(m.k)), m.q_row, m.k_row,
      static_cast<const ne_bf16*>(at_(m.qw)), static_cast<const ne_bf16*>(at_(m.kw)),
      static_cast<const int*>(at_(m.pos)), m.n, m.H, m.Hkv, kDim, m.max_seqlen, m.eps, m.base,
      static_cast<ne_bf16*>(at_(&qr)), static_cast<ne_bf16*>(at_(&kr)), m.c.stream());
  return result(rc, {qr, kr});
  END_HANDLE_TH_ERRORS
}

// dqr, dkr, q, k, q_weight, k_weight, positions, max_seqlen, eps, rope_base, dq, dk,
// dq_weight, dk_weight
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Norm m;
  if (n != 14 || !m.parse(a + 2)) Py_RETURN_NONE;
  const Tensor *dqr = m.c.get(a[0], kBf16, {m.n, m.H, kDim}), *dkr = m.c.get(a[1], kBf16, {m.n, m.Hkv, kDim});
  const Tensor *gq = nullptr, *gk = nullptr, *gqw, *gkw;
  int64_t dq_row = kDim * m.H, dk_row = kDim * m.Hkv;
  if (!dqr || !dkr || !m.c.maybe(a[12], kF32, {kDim}, gqw) || !m.c.maybe(a[13], kF32, {kDim}, gkw) ||
      !m.c.current())
    Py_RETURN_NONE;
  if (a[10] != Py_None && (!(gq = m.c.rows(a[10], dq_row)) || gq->sizes() != m.q->sizes())) Py_RETURN_NONE;
  if (a[11] != Py_None && (!(gk = m.c.rows(a[11], dk_row)) || gk->sizes() != m.k->sizes())) Py_RETURN_NONE;
  const Tensor dq = output(gq, m.q->sizes(), kBf16, *m.q), dk = output(gk, m.k->sizes(), kBf16, *m.k);
  const Tensor dqw = output(gqw, {kDim}, kF32, *m.q), dkw = output(gkw, {kDim}, kF32, *m.q);
  const ne_status rc = unlocked(lib.norm_bwd, static_cast<const ne_bf16*>(at_(dqr)),
      static_cast<const ne_bf16*>(at_(dkr)), static_cast<const ne_bf16*>(at_(m.q)),
      static_cast<const ne_bf16*>(at_(m.k)), m.q_row, m.k_row,
      static_cast<const ne_bf16*>(at_(m.qw)), static_cast<const ne_bf16*>(at_(m.kw)),
      static_cast<const int*>(at_(m.pos)), m.n, m.H, m.Hkv, kDim, m.max_seqlen, m.eps, m.base,
      static_cast<ne_bf16*>(at_(&dq)), static_cast<ne_bf16*>(at_(&dk)), dq_row, dk_row,
      static_cast<float*>(at_(&dqw)), static_cast<float*>(at_(&dkw)), nullptr, 0, m.c.stream());
  return result(rc, {dq, dk, dqw, dkw});
  END_HANDLE_TH_ERRORS
}

// What reserve and release share.
struct Pages {
  Call c;
  const Tensor *lens, *table, *free, *n_free;
  int nseq;

  // a: seq_lens, block_table, free_pages, n_free
  bool parse(PyObject* const* a) {
    if (!(lens = c.get(a[0], kI32, {-1}))) return false;
    nseq = len(lens, 0);
    return (table = c.get(a[1], kI32, {nseq, -1})) && (free = c.get(a[2], kI32, {-1})) &&
           (n_free = c.get(a[3], kI32, {1}));
  }
};

// new_lens, seq_lens, block_table, free_pages, n_free, n_tot, page_size, max_seqlen, cu_seqlens,
// start_pos, positions, slots, seq_lens_out, n_free_out
PyObject* reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Pages p;
  int n_tot, page_size, max_seqlen;
  const Tensor *g[4], *lens_out, *n_free_out;
  if (n != 14 || !p.parse(a + 1)) Py_RETURN_NONE;
  const Tensor* more = p.c.get(a[0], kI32, {p.nseq});
  if (!more || !as_int(a[5], n_tot) || n_tot < 0 || !as_int(a[6], page_size) || !as_int(a[7], max_seqlen) ||
      !p.c.maybe(a[8], kI32, {p.nseq + 1LL}, g[0]) || !p.c.maybe(a[9], kI32, {p.nseq}, g[1]) ||
      !p.c.maybe(a[10], kI32, {n_tot}, g[2]) || !p.c.maybe(a[11], kI32, {n_tot}, g[3]) ||
      !p.c.maybe(a[12], kI32, {p.nseq}, lens_out) || !p.c.maybe(a[13], kI32, {1}, n_free_out) ||
      !p.c.current())
    Py_RETURN_NONE;
  const Tensor cu = output(g[0], {p.nseq + 1LL}, kI32, *more), start = output(g[1], {p.nseq}, kI32, *more);
  const Tensor pos = output(g[2], {n_tot}, kI32, *more), slots = output(g[3], {n_tot}, kI32, *more);
  const ne_status rc = unlocked(lib.reserve, static_cast<const int*>(at_(more)),
      static_cast<const int*>(at_(p.lens)), p.nseq, static_cast<int*>(at_(p.table)),
      len(p.table, 1), static_cast<const int*>(at_(p.free)), static_cast<const int*>(at_(p.n_free)),
      len(p.free, 0), page_size, max_seqlen, n_tot, static_cast<int*>(at_(&cu)),
      static_cast<int*>(at_(&start)), n_tot ? static_cast<int*>(at_(&pos)) : nullptr,
      n_tot ? static_cast<int*>(at_(&slots)) : nullptr,
      static_cast<int*>(at_(lens_out ? lens_out : p.lens)),
      static_cast<int*>(at_(n_free_out ? n_free_out : p.n_free)), p.c.stream());
  return result(rc, {cu, start, pos, slots});
  END_HANDLE_TH_ERRORS
}

// finished, seq_lens, block_table, free_pages, n_free, page_size, max_seqlen.  The status.
PyObject* release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Pages p;
  int page_size, max_seqlen;
  if (n != 7 || !p.parse(a + 1)) Py_RETURN_NONE;
  const Tensor* done = p.c.get(a[0], at::kBool, {p.nseq});
  if (!done) done = p.c.get(a[0], kU8, {p.nseq});
  if (!done || !as_int(a[5], page_size) || !as_int(a[6], max_seqlen) || !p.c.current()) Py_RETURN_NONE;
  return PyLong_FromLong(unlocked(lib.release, static_cast<const uint8_t*>(at_(done)),
      static_cast<int*>(at_(p.lens)), p.nseq, static_cast<int*>(at_(p.table)), len(p.table, 1),
      static_cast<int*>(at_(p.free)), static_cast<int*>(at_(p.n_free)), len(p.free, 0), page_size,
      max_seqlen, p.c.stream()));
  END_HANDLE_TH_ERRORS
}

// A paged cache.
struct Cache {
  const Tensor *k, *v, *ks, *vs, *table;
  int type, Hkv;

  // a: k_pages, v_pages, block_table; k_scale, v_scale
  bool parse(Call& c, PyObject* const* a, PyObject* k_scale, PyObject* v_scale, int nseq) {
    ks = vs = nullptr;
    if ((k = c.get(a[0], kBf16, {-1, -1, -1, kDim})))
      type = NE_KV_BF16;
    else if ((k = c.get(a[0], kE4m3, {-1, -1, -1, kDim})))
      type = NE_KV_E4M3;
    else if ((k = c.get(a[0], kU8, {-1, -1, -1, kDim / 2})))
      type = NE_KV_E2M1;
    else
      return false;
    v = c.get(a[1], k->scalar_type(), {k->size(0), k->size(1), k->size(2), k->size(3)});
    table = c.get(a[2], kI32, {nseq, -1});
    Hkv = len(k, 1);
    if (!v || !table) return false;
    if (type == NE_KV_BF16) return k_scale == Py_None && v_scale == Py_None;
    auto scale = [&](PyObject* o) {
      return type == NE_KV_E4M3 ? c.get(o, kU8, {k->size(0), k->size(1), k->size(2)})
                                : c.get(o, kU8, {k->size(0), k->size(1), k->size(2), 2});
    };
    return (ks = scale(k_scale)) && (vs = scale(v_scale));
  }
  const uint8_t* scale(const Tensor* t) const { return static_cast<const uint8_t*>(at_(t)); }
};

// k, v, cu_seqlens, start_pos, k_pages, v_pages, block_table, max_seqlen, k_scale, v_scale,
// rope_base.  The status.
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  Cache s;
  int max_seqlen;
  float base;
  if (n != 11) Py_RETURN_NONE;
  const Tensor *k = c.get(a[0], kBf16, {-1, -1, kDim}), *start = c.get(a[3], kI32, {-1});
  if (!k || !start || k->size(0) == 0) Py_RETURN_NONE;
  const Tensor *v = c.get(a[1], kBf16, {k->size(0), k->size(1), kDim}),
               *cu = c.get(a[2], kI32, {start->size(0) + 1});
  if (!v || !cu || !s.parse(c, a + 4, a[8], a[9], len(start, 0)) || s.Hkv != k->size(1) ||
      !as_int(a[7], max_seqlen) || !as_float(a[10], base) || !c.current())
    Py_RETURN_NONE;
  return PyLong_FromLong(unlocked(lib.append, static_cast<const ne_bf16*>(at_(k)),
      static_cast<const ne_bf16*>(at_(v)), static_cast<const int*>(at_(cu)),
      static_cast<const int*>(at_(start)), len(start, 0), len(k, 0), s.Hkv, kDim, base, s.type,
      at_(s.k), at_(s.v), static_cast<uint8_t*>(at_(s.ks)), static_cast<uint8_t*>(at_(s.vs)),
      static_cast<const int*>(at_(s.table)), len(s.table, 1), len(s.k, 0), len(s.k, 2), max_seqlen,
      c.stream()));
  END_HANDLE_TH_ERRORS
}

// k_pages, v_pages, block_table, cu_seqlens, start_pos, n_tot, k_scale, v_scale, max_seqlen, k, v
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  Cache s;
  int n_tot, max_seqlen = 0;
  if (n != 11) Py_RETURN_NONE;
  const Tensor* start = c.get(a[4], kI32, {-1});
  if (!start || !s.parse(c, a, a[6], a[7], len(start, 0)) || !as_int(a[5], n_tot) || n_tot <= 0)
    Py_RETURN_NONE;
  const Tensor *cu = c.get(a[3], kI32, {start->size(0) + 1}), *gk, *gv;
  if (a[8] == Py_None) {  // the table's reach
    const int64_t reach = s.table->size(1) * s.k->size(2);
    max_seqlen = static_cast<int>(reach < 65535 * 128 ? reach : 65535 * 128);
  } else if (!as_int(a[8], max_seqlen)) {
    Py_RETURN_NONE;
  }
  if (!cu || !c.maybe(a[9], kBf16, {n_tot, s.Hkv, kDim}, gk) ||
      !c.maybe(a[10], kBf16, {n_tot, s.Hkv, kDim}, gv) || !c.current())
    Py_RETURN_NONE;
  const Tensor k = output(gk, {n_tot, s.Hkv, kDim}, kBf16, *start),
               v = output(gv, {n_tot, s.Hkv, kDim}, kBf16, *start);
  const ne_status rc = unlocked(lib.read, s.type, at_(s.k), at_(s.v), s.scale(s.ks), s.scale(s.vs),
      static_cast<const int*>(at_(s.table)), len(s.table, 1), len(s.k, 0), len(s.k, 2), max_seqlen,
      static_cast<const int*>(at_(cu)), static_cast<const int*>(at_(start)), len(start, 0), n_tot,
      s.Hkv, kDim, static_cast<ne_bf16*>(at_(&k)), static_cast<ne_bf16*>(at_(&v)), c.stream());
  return result(rc, {k, v});
  END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, block_table, seq_lens, max_seqlen, k_scale, v_scale, rope_base, scale, out,
// lse
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Call c;
  Cache s;
  int max_seqlen;
  float base, scale = 0.125f;
  const Tensor *go, *gl;
  if (n != 12) Py_RETURN_NONE;
  const Tensor* q = c.get(a[0], kBf16, {-1, -1, kDim});
  if (!q) Py_RETURN_NONE;
  const int B = len(q, 0), H = len(q, 1);
  const Tensor* lens = c.get(a[4], kI32, {B});
  if (!lens || !s.parse(c, a + 1, a[6], a[7], B) || s.Hkv == 0 || H % s.Hkv != 0 ||
      !as_int(a[5], max_seqlen) || !as_float(a[8], base) ||
      (a[9] != Py_None && !as_float(a[9], scale)) || !c.maybe(a[10], kBf16, {B, H, kDim}, go) ||
      !c.maybe(a[11], kF32, {B, H}, gl) || !c.current())
    Py_RETURN_NONE;
  const Tensor out = output(go, q->sizes(), kBf16, *q), lse = output(gl, {B, H}, kF32, *q);
  const ne_status rc = unlocked(lib.decode, static_cast<const ne_bf16*>(at_(q)), s.type, at_(s.k),
      at_(s.v), s.scale(s.ks), s.scale(s.vs), static_cast<const int*>(at_(s.table)),
      len(s.table, 1), len(s.k, 0), len(s.k, 2), max_seqlen, static_cast<const int*>(at_(lens)), B,
      H, s.Hkv, kDim, base, scale, static_cast<ne_bf16*>(at_(&out)), static_cast<float*>(at_(&lse)),
      nullptr, 0, c.stream());
  return result(rc, {out, lse});
  END_HANDLE_TH_ERRORS
}

// The addresses of the library's entry points, in the order of `lib`.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind: 7 addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  lib.norm_fwd = reinterpret_cast<decltype(lib.norm_fwd)>(at[0]);
  lib.norm_bwd = reinterpret_cast<decltype(lib.norm_bwd)>(at[1]);
  lib.reserve = reinterpret_cast<decltype(lib.reserve)>(at[2]);
  lib.release = reinterpret_cast<decltype(lib.release)>(at[3]);
  lib.append = reinterpret_cast<decltype(lib.append)>(at[4]);
  lib.read = reinterpret_cast<decltype(lib.read)>(at[5]);
  lib.decode = reinterpret_cast<decltype(lib.decode)>(at[6]);
  Py_RETURN_NONE;
}

#define NE_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {NE_METHOD(bind),    NE_METHOD(norm_fwd), NE_METHOD(norm_bwd),
                         NE_METHOD(reserve), NE_METHOD(release),  NE_METHOD(append),
                         NE_METHOD(read),    NE_METHOD(decode),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ne_step", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};
}  // namespace

PyMODINIT_FUNC PyInit_ne_step() { return PyModule_Create(&module); }
