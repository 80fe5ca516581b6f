// The Python calls around the attention (norms with rotation, rotated writes,
// verification, the 4-bit cache) as the usual program makes them: tensors on the
// current device and its current stream.  One call here checks the arguments, makes the
// results and enters the library, which from Python, attribute by attribute, takes
// longer than most of the kernels: a rotation of 104 rows 17 us, here 5 (of them 3.3 on the
// GPU), a verification 23 and 9, a 4-bit write and read 25 and 8, attention over the 4-bit cache 26 and 10.
//
// A call that is not plain -- something that does not fit, another device -- is
// answered by None before anything was made or launched; the Python wrapper then
// does the call or names what is wrong with it.  So a check here may refuse too
// much, never too little.  A number is the library's error.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <array>
#include <cstdint>
#include <initializer_list>

#include "../../include/jgdpa.h"

namespace {

using at::Tensor;

#define JG_FUNCTIONS(X)                \
  X(jgdpa_norm_rotate_workspace_bytes) \
  X(jgdpa_norm_rotate)                 \
  X(jgdpa_norm_rotate_bwd)             \
  X(jgdpa_cache_append_rotated)        \
  X(jgdpa_verify)                      \
  X(jgdpa_cache4_append)               \
  X(jgdpa_cache4_read)                 \
  X(jgdpa_cache4_fwd_workspace_bytes)  \
  X(jgdpa_cache4_fwd)

struct Library {
#define JG_MEMBER(f) decltype(&::f) f = nullptr;
  JG_FUNCTIONS(JG_MEMBER)
#undef JG_MEMBER
};
Library lib;

// A call's arguments; ok turns false at the first that is not plain.
struct Call {
  bool ok = true;
  int device = -1;

  const Tensor* optional(PyObject* o) {
    if (o == Py_None || !ok) return nullptr;
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.unsafeGetTensorImpl()->is_python_dispatch()) {
      ok = false;
      return nullptr;
    }
    const int at = static_cast<int>(t.get_device());
    if (device < 0) device = at;
    ok = at == device;
    return ok ? &t : nullptr;
  }
  const Tensor* required(PyObject* o) {
    const Tensor* t = optional(o);
    ok = ok && t != nullptr;
    return t;
  }
  void need(bool x) { ok = ok && x; }
  // (with the last argument read) on the current device, with the library at hand
  bool plain() { return ok && device >= 0 && lib.jgdpa_cache4_fwd != nullptr && device == c10::cuda::current_device(); }

  void is(const Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (ok && t != nullptr)
      ok = t->scalar_type() == type && t->sizes() == at::IntArrayRef(shape) && t->is_contiguous();
  }
  // a vector; its length
  int64_t vector(const Tensor* t, at::ScalarType type) {
    if (!ok || t == nullptr) return 0;
    ok = t->scalar_type() == type && t->dim() == 1 && t->is_contiguous();
    return ok ? t->size(0) : 0;
  }
  // [rows][heads][d] bf16; the stride of a row
  int64_t rows(const Tensor* t, int64_t n, int64_t heads, int64_t d) {
    if (!ok || t == nullptr) return 0;
    ok = t->scalar_type() == at::kBFloat16 && t->dim() == 3 && t->size(0) == n && t->size(1) == heads && t->size(2) == d && heads > 0;
    if (!ok) return 0;
    if (t->numel() != 0 && (t->stride(2) != 1 || (heads > 1 && t->stride(1) != d))) ok = false;
    if (n <= 1) return heads * d;
    const int64_t stride = t->stride(0);
    need(stride >= heads * d && stride % 8 == 0);
    return stride;
  }
  // a cache's pages, contiguous inside; the stride of a page
  int64_t pages(const Tensor* t, at::ScalarType type, std::array<int64_t, 4> shape, int64_t align) {
    if (!ok || t == nullptr) return 0;
    ok = t->scalar_type() == type && t->sizes() == at::IntArrayRef(shape);
    if (!ok) return 0;
    const int64_t size = shape[1] * shape[2] * shape[3];
    ok = size > 0 && (shape[3] == 1 || t->stride(3) == 1) && (shape[2] == 1 || t->stride(2) == shape[3]) &&
         (shape[1] == 1 || t->stride(1) == shape[2] * shape[3]);
    if (shape[0] <= 1) return size;
    const int64_t stride = t->stride(0);
    need(stride >= size && stride % align == 0);
    return stride;
  }
  int32_t small(int64_t x) {
    need(x >= INT32_MIN && x <= INT32_MAX);
    return static_cast<int32_t>(x);
  }
  int32_t whole(PyObject* o) {
    if (!ok || !PyLong_CheckExact(o)) {
      ok = false;
      return 0;
    }
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &over);
    need(over == 0);
    return small(x);
  }
  float real(PyObject* o) {
    if (!ok || !PyFloat_CheckExact(o)) {
      ok = false;
      return 0.f;
    }
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
  }
  int truth(PyObject* o) {
    need(o == Py_True || o == Py_False);
    return o == Py_True ? 1 : 0;
  }
};

template <typename T = void>
T* at(const Tensor* t) {
  return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
}
const int32_t* ints(const Tensor* t) { return at<const int32_t>(t); }
const float* floats(const Tensor* t) { return at<const float>(t); }
size_t bytes(const Tensor* t) { return t == nullptr ? 0 : static_cast<size_t>(t->numel()); }
Tensor empty(at::IntArrayRef shape, const Tensor& like, at::ScalarType type) {
  return at::empty(shape, like.options().dtype(type).requires_grad(false));
}
jgdpa_stream_t stream_of(const Call& c) {
  return reinterpret_cast<jgdpa_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream());
}
// A result: the caller's own object, or a new one.
struct Result {
  PyObject* given;
  Tensor made;
  const Tensor* t;
  Result(PyObject* o, const Tensor* have, at::IntArrayRef shape, const Tensor& like, at::ScalarType type) : given(o), t(have) {
    if (have == nullptr) {
      made = empty(shape, like, type);
      t = &made;
    }
  }
  PyObject* object() const {
    if (made.defined()) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
  }
};
PyObject* none() { Py_RETURN_NONE; }
PyObject* pack(std::initializer_list<PyObject*> items) {  // (takes the references)
  PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  bool ok = tuple != nullptr;
  for (PyObject* o : items) {
    ok = ok && o != nullptr;
    if (tuple != nullptr) PyTuple_SET_ITEM(tuple, i++, o);
    else Py_XDECREF(o);
  }
  if (ok) return tuple;
  Py_XDECREF(tuple);
  return nullptr;
}
#define JG_ENTER(rc, call)           \
  jgdpa_status rc;                   \
  Py_BEGIN_ALLOW_THREADS rc = call;  \
  Py_END_ALLOW_THREADS if (rc != JGDPA_OK) return PyLong_FromLong(rc)

struct Rotation {
  const Tensor* freq;
  int32_t pairs;
  int interleaved, norm;
  float eps = 0.f;
};
Rotation rotation(Call& c, PyObject* freq, PyObject* eps, PyObject* interleaved, int64_t d) {
  Rotation r;
  r.freq = c.required(freq);
  r.interleaved = c.truth(interleaved);
  r.norm = eps != Py_None;
  if (r.norm) r.eps = c.real(eps);
  const int64_t n = c.vector(r.freq, at::kFloat);
  c.need((d == 32 || d == 64 || d == 128) && n >= 1 && n <= d / 2 && (r.interleaved || n % 8 == 0));
  r.pairs = static_cast<int32_t>(c.ok ? n : 0);
  return r;
}

// Queries or keys of the packed calls.
struct Side {
  const Tensor *x = nullptr, *off = nullptr, *pos = nullptr, *w = nullptr;
  int64_t stride = 8, rows = 0;
  int32_t heads = 0;
};
Side side(Call& c, PyObject* x, PyObject* off, PyObject* pos, PyObject* w, int64_t d) {
  Side s;
  s.x = c.required(x);
  c.need(c.ok && s.x->dim() == 3);
  if (!c.ok) return s;
  s.rows = s.x->size(0);
  s.heads = c.small(s.x->size(1));
  s.stride = c.rows(s.x, s.rows, s.heads, d);
  if (pos == Py_None) {
    s.off = c.required(off);
    c.need(c.vector(s.off, at::kInt) >= 1);
  } else {
    s.pos = c.required(pos);
    c.is(s.pos, at::kInt, {s.rows});
  }
  s.w = c.optional(w);
  c.is(s.w, at::kFloat, {d});
  return s;
}
int32_t batch_of(Call& c, const Side& q, const Side& k) {
  const int64_t a = q.off == nullptr ? -1 : q.off->size(0) - 1, b = k.off == nullptr ? -1 : k.off->size(0) - 1;
  c.need(a < 0 || b < 0 || a == b);
  return c.small(a >= 0 ? a : b >= 0 ? b : 0);
}

PyObject* norm_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14) return none();
  PyObject *eps = a[7], *q_out = a[11], *k_out = a[12];
  Call c;
  const Tensor* x = c.required(a[0]);
  const int64_t d = c.ok && x->dim() == 3 ? x->size(2) : 0;
  const Rotation r = rotation(c, a[4], eps, a[8], d);
  if (!c.ok) return none();
  const Side q = side(c, a[0], a[2], a[9], a[5], d);
  Side k;
  const bool both = a[1] != Py_None;
  if (both) k = side(c, a[1], a[3], a[10], a[6], d);
  else c.need(a[6] == Py_None && k_out == Py_None);
  c.need(r.norm || (q.w == nullptr && k.w == nullptr));
  const Tensor *qo = c.optional(q_out), *ko = c.optional(k_out), *ws = c.optional(a[13]);
  int64_t qos = q.heads * d, kos = k.heads * d;
  if (qo != nullptr) qos = c.rows(qo, q.rows, q.heads, d);
  if (ko != nullptr) kos = c.rows(ko, k.rows, k.heads, d);
  c.vector(ws, at::kByte);
  if (!c.ok) return none();
  const int32_t batch = batch_of(c, q, k);
  if (!c.plain()) return none();
  const Result out_q(q_out, qo, q.x->sizes(), *q.x, at::kBFloat16);
  const Result out_k(k_out, both ? ko : q.x, both ? k.x->sizes() : q.x->sizes(), *q.x, at::kBFloat16);
  const jgdpa_stream_t stream = stream_of(c);
  JG_ENTER(rc, lib.jgdpa_norm_rotate(at(q.x), q.stride, at(out_q.t), qos, q.rows, q.heads, ints(q.off), ints(q.pos), floats(q.w),
                                     at(k.x), k.stride, both ? at(out_k.t) : nullptr, kos, k.rows, k.heads, ints(k.off),
                                     ints(k.pos), floats(k.w), batch, static_cast<int32_t>(d), floats(r.freq), r.pairs,
                                     r.interleaved, r.norm, r.eps, at(ws), bytes(ws), stream));
  return pack({out_q.object(), both ? out_k.object() : none()});
  END_HANDLE_TH_ERRORS
}

PyObject* norm_rotate_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 18) return none();
  // dq_out dk_out q k q_offsets kv_offsets inv_freq q_weight k_weight eps interleaved q_positions k_positions dq dk dqw dkw workspace
  PyObject* eps = a[9];
  Call c;
  const Tensor* x = c.required(a[0]);
  const int64_t d = c.ok && x->dim() == 3 ? x->size(2) : 0;
  const Rotation r = rotation(c, a[6], eps, a[10], d);
  if (!c.ok) return none();
  const Side q = side(c, a[0], a[4], a[11], a[7], d);
  Side k;
  const bool both = a[1] != Py_None;
  if (both) k = side(c, a[1], a[5], a[12], a[8], d);
  else c.need(a[3] == Py_None && a[8] == Py_None && a[14] == Py_None && a[16] == Py_None);
  const Tensor *qx = nullptr, *kx = nullptr;
  int64_t qs = q.stride, ks = k.stride, dqs = q.heads * d, dks = k.heads * d;
  if (r.norm) {
    qx = c.required(a[2]);
    qs = c.rows(qx, q.rows, q.heads, d);
    if (both) {
      kx = c.required(a[3]);
      ks = c.rows(kx, k.rows, k.heads, d);
    }
  }
  const Tensor *dq = c.optional(a[13]), *dk = c.optional(a[14]), *dqw = c.optional(a[15]), *dkw = c.optional(a[16]), *ws = c.optional(a[17]);
  if (dq != nullptr) dqs = c.rows(dq, q.rows, q.heads, d);
  if (dk != nullptr) dks = c.rows(dk, k.rows, k.heads, d);
  c.is(dqw, at::kFloat, {d});
  c.is(dkw, at::kFloat, {d});
  c.need(r.norm || (q.w == nullptr && k.w == nullptr && dqw == nullptr && dkw == nullptr));
  c.vector(ws, at::kByte);
  if (!c.ok) return none();
  const int32_t batch = batch_of(c, q, k);
  if (!c.plain()) return none();
  const Result out_q(a[13], dq, q.x->sizes(), *q.x, at::kBFloat16);
  const Result out_k(a[14], both ? dk : q.x, both ? k.x->sizes() : q.x->sizes(), *q.x, at::kBFloat16);
  const bool qw = dqw != nullptr || q.w != nullptr, kw = dkw != nullptr || k.w != nullptr;
  const Result out_qw(a[15], qw ? dqw : q.x, {d}, *q.x, at::kFloat), out_kw(a[16], kw ? dkw : q.x, {d}, *q.x, at::kFloat);
  Tensor own;
  if (ws == nullptr && (qw || kw)) {
    own = empty({static_cast<int64_t>(std::max<size_t>(256, lib.jgdpa_norm_rotate_workspace_bytes(static_cast<int32_t>(d), 1)))}, *q.x, at::kByte);
    ws = &own;
  }
  const jgdpa_stream_t stream = stream_of(c);
  JG_ENTER(rc, lib.jgdpa_norm_rotate_bwd(
                   at(q.x), q.stride, at(qx), qs, at(out_q.t), dqs, q.rows, q.heads, ints(q.off), ints(q.pos), floats(q.w),
                   qw ? at<float>(out_qw.t) : nullptr, at(k.x), k.stride, at(kx), ks, both ? at(out_k.t) : nullptr, dks, k.rows,
                   k.heads, ints(k.off), ints(k.pos), floats(k.w), kw ? at<float>(out_kw.t) : nullptr, batch,
                   static_cast<int32_t>(d), floats(r.freq), r.pairs, r.interleaved, r.norm, r.eps, at(ws), bytes(ws), stream));
  return pack({out_q.object(), both ? out_k.object() : none(), qw ? out_qw.object() : none(), kw ? out_kw.object() : none()});
  END_HANDLE_TH_ERRORS
}

PyObject* cache_append_rotated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 16) return none();
  // q k_new v_new slots k_cache v_cache q_offsets kv_lens inv_freq q_weight k_weight eps interleaved depths q_out workspace
  Call c;
  const Tensor *kc = c.required(a[4]), *vc = c.required(a[5]), *kn = c.required(a[1]), *vn = c.required(a[2]);
  c.need(c.ok && kc->dim() == 4 && kn->dim() == 3);
  if (!c.ok) return none();
  const std::array<int64_t, 4> shape = {kc->size(0), kc->size(1), kc->size(2), kc->size(3)};
  const int64_t heads = shape[2], d = shape[3], rows = kn->size(0);
  const int64_t kps = c.pages(kc, at::kBFloat16, shape, 8), vps = c.pages(vc, at::kBFloat16, shape, 8);
  const int64_t ks = c.rows(kn, rows, heads, d), vs = c.rows(vn, rows, heads, d);
  const Rotation r = rotation(c, a[8], a[11], a[12], d);
  const Tensor *slots = c.required(a[3]), *off = c.required(a[6]), *lens = c.required(a[7]), *depths = c.optional(a[13]);
  c.is(slots, at::kInt, {rows});
  const int64_t batch = c.vector(lens, at::kInt);
  c.is(off, at::kInt, {batch + 1});
  c.is(depths, at::kInt, {rows});
  const Tensor *q = c.optional(a[0]), *qw = c.optional(a[9]), *kw = c.optional(a[10]), *qo = c.optional(a[14]), *ws = c.optional(a[15]);
  c.is(qw, at::kFloat, {d});
  c.is(kw, at::kFloat, {d});
  c.vector(ws, at::kByte);
  int64_t q_heads = 0, qs = 0, qos = 0;
  if (q != nullptr) {
    c.need(q->dim() == 3);
    if (!c.ok) return none();
    q_heads = q->size(1);
    qs = c.rows(q, rows, q_heads, d);
    qos = q_heads * d;
    if (qo != nullptr) qos = c.rows(qo, rows, q_heads, d);
  }
  c.need((q != nullptr || (qo == nullptr && qw == nullptr)) && (r.norm || (qw == nullptr && kw == nullptr)));
  const int32_t n_rows = c.small(rows), n_pages = c.small(shape[0]), page = c.small(shape[1]), n_batch = c.small(batch);
  c.small(heads);
  c.small(q_heads);
  if (!c.plain()) return none();
  const Result out(a[14], q != nullptr ? qo : kn, q != nullptr ? q->sizes() : kn->sizes(), *kn, at::kBFloat16);
  const jgdpa_stream_t stream = stream_of(c);
  JG_ENTER(rc, lib.jgdpa_cache_append_rotated(
                   at(q), qs, q != nullptr ? at(out.t) : nullptr, qos, static_cast<int32_t>(q_heads), at(kn), at(vn), ks, vs, ints(slots),
                   n_rows, at(kc), at(vc), kps, vps, n_pages, page, static_cast<int32_t>(heads), static_cast<int32_t>(d), ints(off),
                   ints(lens), ints(depths), n_batch, floats(qw), floats(kw), floats(r.freq), r.pairs, r.interleaved, r.norm, r.eps,
                   at(ws), bytes(ws), stream));
  Py_INCREF(a[4]);
  Py_INCREF(a[5]);
  return pack({q != nullptr ? out.object() : none(), a[4], a[5]});
  END_HANDLE_TH_ERRORS
}

// Rows of probabilities; their stride.
int64_t probs(Call& c, const Tensor* t, int64_t rows, int64_t vocab) {
  if (!c.ok || t == nullptr) return vocab;
  c.need((t->scalar_type() == at::kFloat || t->scalar_type() == at::kBFloat16) && t->dim() == 2 && t->size(0) == rows &&
         t->size(1) == vocab && (vocab <= 1 || t->stride(1) == 1));
  if (!c.ok || rows <= 1) return vocab;
  c.need(t->stride(0) >= vocab);
  return t->stride(0);
}

PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) return none();
  // target_probs tokens q_offsets uniforms draft_probs parents kv_lens slots workspace
  Call c;
  const Tensor *p = c.required(a[0]), *tokens = c.required(a[1]), *off = c.required(a[2]), *u = c.required(a[3]);
  c.need(c.ok && p->dim() == 2);
  if (!c.ok) return none();
  const int64_t total = p->size(0), vocab = p->size(1), batch = c.vector(off, at::kInt) - 1;
  const Tensor *q = c.optional(a[4]), *parents = c.optional(a[5]), *lens = c.optional(a[6]), *slots = c.optional(a[7]), *ws = c.optional(a[8]);
  const int64_t ps = probs(c, p, total, vocab), ds = probs(c, q, total, vocab);
  c.need(batch >= 0 && vocab > 0 && (q == nullptr || parents == nullptr));
  c.is(tokens, at::kInt, {total});
  c.is(u, at::kFloat, {total});
  c.is(parents, at::kInt, {total});
  c.is(lens, at::kInt, {batch});
  c.is(slots, at::kInt, {total});
  c.vector(ws, at::kByte);
  const int32_t n_batch = c.small(batch), n_total = c.small(total), n_vocab = c.small(vocab);
  if (!c.plain()) return none();
  Tensor accepted = empty({batch}, *off, at::kInt), next = empty({batch}, *off, at::kInt), places = empty({total}, *off, at::kInt), keep_lens, keep_slots;
  if (lens != nullptr) keep_lens = empty({batch}, *off, at::kInt);
  if (slots != nullptr) keep_slots = empty({total}, *off, at::kInt);
  const jgdpa_stream_t stream = stream_of(c);
  JG_ENTER(rc, lib.jgdpa_verify(at(p), ps, p->scalar_type() == at::kBFloat16, at(q), ds, q != nullptr && q->scalar_type() == at::kBFloat16,
                                ints(tokens), ints(parents), floats(u), ints(off), n_batch, n_total, n_vocab, ints(lens), ints(slots),
                                at<int32_t>(&accepted), at<int32_t>(&next), at<int32_t>(&places),
                                lens != nullptr ? at<int32_t>(&keep_lens) : nullptr,
                                slots != nullptr ? at<int32_t>(&keep_slots) : nullptr, at(ws), bytes(ws), stream));
  return pack({THPVariable_Wrap(accepted), THPVariable_Wrap(next), THPVariable_Wrap(places),
               lens != nullptr ? THPVariable_Wrap(keep_lens) : none(), slots != nullptr ? THPVariable_Wrap(keep_slots) : none()});
  END_HANDLE_TH_ERRORS
}

// A cache held in 4 bits: codes and scales of keys, then of values.
struct Cache4 {
  const Tensor* t[4];
  int64_t stride[4];
  int32_t pages, page, heads;
  int64_t d;
};
Cache4 cache4(Call& c, PyObject* const* a) {
  Cache4 x{};
  for (int i = 0; i < 4; ++i) x.t[i] = c.required(a[i]);
  c.need(c.ok && x.t[0]->dim() == 4);
  if (!c.ok) return x;
  const at::IntArrayRef s = x.t[0]->sizes();
  const std::array<int64_t, 4> codes = {s[0], s[1], s[2], s[3]}, scales = {s[0], s[1], s[2], 2};
  for (int i = 0; i < 4; ++i) x.stride[i] = i % 2 == 0 ? c.pages(x.t[i], at::kByte, codes, 16) : c.pages(x.t[i], at::kBFloat16, scales, 8);
  x.pages = c.small(s[0]);
  x.heads = c.small(s[1]);
  x.page = c.small(s[2]);
  x.d = 2 * s[3];
  c.need(x.d <= 128);
  return x;
}

PyObject* cache4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) return none();
  // k_new v_new slots k_codes k_scales v_codes v_scales
  Call c;
  const Cache4 x = cache4(c, a + 3);
  const Tensor *k = c.required(a[0]), *v = c.required(a[1]), *slots = c.required(a[2]);
  const int64_t rows = c.vector(slots, at::kInt);
  const int64_t ks = c.rows(k, rows, x.heads, x.d), vs = c.rows(v, rows, x.heads, x.d);
  const int32_t n_rows = c.small(rows);
  if (!c.plain()) return none();
  const jgdpa_stream_t stream = stream_of(c);
  JG_ENTER(rc, lib.jgdpa_cache4_append(at(k), at(v), ks, vs, ints(slots), n_rows, at(x.t[0]), at(x.t[1]), at(x.t[2]), at(x.t[3]), x.stride[0],
                                       x.stride[1], x.stride[2], x.stride[3], x.pages, x.page, x.heads, static_cast<int32_t>(x.d), stream));
  for (int i = 3; i < 7; ++i) Py_INCREF(a[i]);
  return pack({a[3], a[4], a[5], a[6]});
  END_HANDLE_TH_ERRORS
}

PyObject* cache4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) return none();
  // k_codes k_scales v_codes v_scales slots k_out v_out
  Call c;
  const Cache4 x = cache4(c, a);
  const Tensor *slots = c.required(a[4]), *ko = c.optional(a[5]), *vo = c.optional(a[6]);
  const int64_t rows = c.vector(slots, at::kInt);
  int64_t ks = x.heads * x.d, vs = ks;
  if (ko != nullptr) ks = c.rows(ko, rows, x.heads, x.d);
  if (vo != nullptr) vs = c.rows(vo, rows, x.heads, x.d);
  const int32_t n_rows = c.small(rows);
  if (!c.plain()) return none();
  const Result k(a[5], ko, {rows, x.heads, x.d}, *x.t[0], at::kBFloat16), v(a[6], vo, {rows, x.heads, x.d}, *x.t[0], at::kBFloat16);
  const jgdpa_stream_t stream = stream_of(c);
  JG_ENTER(rc, lib.jgdpa_cache4_read(at(x.t[0]), at(x.t[1]), at(x.t[2]), at(x.t[3]), x.stride[0], x.stride[1], x.stride[2], x.stride[3], x.pages,
                                     x.page, x.heads, static_cast<int32_t>(x.d), ints(slots), n_rows, at(k.t), at(v.t), ks, vs, stream));
  return pack({k.object(), v.object()});
  END_HANDLE_TH_ERRORS
}

PyObject* cache4_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 18) return none();
  // q k_codes k_scales v_codes v_scales block_table q_offsets kv_lens act scale max_q bias_table window tree_mask depths out lse workspace
  Call c;
  const Cache4 x = cache4(c, a + 1);
  const Tensor *q = c.required(a[0]), *table = c.required(a[5]), *off = c.required(a[6]), *lens = c.required(a[7]);
  const int32_t act = c.whole(a[8]), max_q = c.whole(a[10]), window = c.whole(a[12]);
  const float scale = c.real(a[9]);
  c.need(c.ok && q->dim() == 3 && table->dim() == 2);
  if (!c.ok) return none();
  const bool softmax = act == JGDPA_ACT_SOFTMAX;
  const int64_t total = q->size(0), heads = q->size(1), batch = c.vector(lens, at::kInt), width = table->size(1);
  const int64_t qs = c.rows(q, total, heads, x.d);
  c.is(off, at::kInt, {batch + 1});
  c.is(table, at::kInt, {batch, width});
  const Tensor *bias = c.optional(a[11]), *mask = c.optional(a[13]), *depths = c.optional(a[14]), *out = c.optional(a[15]), *lse = c.optional(a[16]),
               *ws = c.optional(a[17]);
  int64_t bias_len = 0, words = 0;
  if (bias != nullptr) {
    c.need(bias->dim() == 2 && bias->size(1) > 0);
    if (!c.ok) return none();
    c.is(bias, at::kFloat, {heads, bias_len = bias->size(1)});
  }
  if (mask != nullptr) {
    c.need(mask->dim() == 2 && mask->size(1) > 0);
    if (!c.ok) return none();
    c.is(mask, at::kInt, {total, words = mask->size(1)});
  }
  c.is(depths, at::kInt, {total});
  c.is(out, at::kBFloat16, {total, heads, x.d});
  c.need(lse == nullptr || softmax);
  c.is(lse, at::kFloat, {heads, total});
  c.vector(ws, at::kByte);
  const int32_t n_width = c.small(width), n_batch = c.small(batch), n_heads = c.small(heads), n_bias = c.small(bias_len), n_words = c.small(words);
  if (!c.plain()) return none();
  const int32_t d = static_cast<int32_t>(x.d);
  const Result o(a[15], out, q->sizes(), *q, at::kBFloat16);
  const Result l(a[16], softmax ? lse : q, {heads, total}, *q, at::kFloat);
  Tensor own;
  if (ws == nullptr) {
    own = empty({static_cast<int64_t>(std::max<size_t>(256, lib.jgdpa_cache4_fwd_workspace_bytes(d)))}, *q, at::kByte);
    ws = &own;
  }
  const jgdpa_stream_t stream = stream_of(c);
  JG_ENTER(rc, lib.jgdpa_cache4_fwd(at(q), qs, at(x.t[0]), at(x.t[1]), at(x.t[2]), at(x.t[3]), x.stride[0], x.stride[1], x.stride[2], x.stride[3],
                                    x.pages, x.page, ints(table), n_width, ints(off), ints(lens), n_batch, total, max_q, n_heads, x.heads, d,
                                    static_cast<jgdpa_act>(act), scale, floats(bias), n_bias, window, ints(mask), n_words, ints(depths), at(o.t),
                                    softmax ? at<float>(l.t) : nullptr, at(ws), bytes(ws), stream));
  return pack({o.object(), softmax ? l.object() : none()});
  END_HANDLE_TH_ERRORS
}

// The library's functions, as {name: address}.
PyObject* use(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 1 || !PyDict_Check(a[0])) return none();
  Library got;
#define JG_TAKE(f)                                                              \
  {                                                                             \
    PyObject* o = PyDict_GetItemString(a[0], #f);                               \
    if (o == nullptr) return none();                                            \
    got.f = reinterpret_cast<decltype(got.f)>(PyLong_AsVoidPtr(o));             \
    if (got.f == nullptr) return PyErr_Occurred() != nullptr ? nullptr : none(); \
  }
  JG_FUNCTIONS(JG_TAKE)
#undef JG_TAKE
  lib = got;
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

#define JG_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {JG_METHOD(use),          JG_METHOD(norm_rotate), JG_METHOD(norm_rotate_bwd), JG_METHOD(cache_append_rotated),
                         JG_METHOD(verify),       JG_METHOD(cache4_append), JG_METHOD(cache4_read),   JG_METHOD(cache4_fwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
