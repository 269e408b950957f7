// torch_call.cpp -- the native half of binding.py for the entry points of a
// serving step: takes torch tensors, checks their types, shapes and strides
// (the C ABI cannot see them) and calls the C entry point of the same name.
//
// A step makes these calls for every layer, and each passes ten to twenty
// tensors whose checks cost 0.2 us apiece from Python, besides 0.1 us per
// argument in ctypes and 0.06 us for each pointer that the library looks up
// (which the tensors spare it): 10.4, 12.5 and 15.5 us a call for the tables,
// the append and the shared-prefix decode that way, 3.1, 3.2 and 5.0 this way,
// of which the launches take 1.5 each.  (The decode behind 513 shared rows; its
// plan looks at more numbers of shares the longer they are: 6.1 behind 32,768.)  The functions return the C entry
// point's status; what is wrong with a tensor raises TypeError or ValueError.
// No exception crosses the C interfaces on either side.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "gqa_attn.h"

namespace {

using at::Tensor;

// A Python exception is set: unwinds to the function's boundary.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw Raised();
}

// The tensor of an argument; nullptr for None where that is allowed.
const Tensor* tensor(PyObject* o, bool none = false) {
  if (none && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, none ? "a tensor or None is needed" : "a tensor is needed");
  return &THPVariable_Unpack(o);
}

// Address of a dense tensor.
void* dense(const Tensor* t) {
  if (t == nullptr) return nullptr;
  if (!t->is_contiguous()) raise(PyExc_ValueError, "tensors passed to libgqa_attn must be contiguous");
  return t->data_ptr();
}

// Address of a dense int32 tensor of n entries.
int32_t* ints(const Tensor* t, int64_t n) {
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != at::kInt) raise(PyExc_TypeError, "lengths, tables, positions and slots are int32");
  if (t->numel() != n || !t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "a contiguous int32 tensor of %lld entries is needed, got %lld entries%s",
                 (long long)n, (long long)t->numel(), t->is_contiguous() ? "" : ", not contiguous");
    throw Raised();
  }
  return static_cast<int32_t*>(t->data_ptr());
}

bool shaped(const Tensor* t, std::initializer_list<int64_t> shape) {
  return t->sizes() == at::IntArrayRef(shape.begin(), shape.size());
}

void rank(const Tensor* t, int64_t n, const char* text) {
  if (t->dim() != n) raise(PyExc_ValueError, text);
}

int dtype_code(const Tensor* t) {
  if (t->scalar_type() == at::kFloat) return GQA_F32;
  if (t->scalar_type() == at::kBFloat16) return GQA_BF16;
  raise(PyExc_TypeError, "unsupported dtype: float32 or bfloat16");
}

void one_dtype(const Tensor* first, std::initializer_list<const Tensor*> others) {
  for (const Tensor* t : others)
    if (t != nullptr && t->scalar_type() != first->scalar_type())
      raise(PyExc_TypeError, "the tensors of a call have one dtype");
}

// A size for the C ABI's int.
int size(int64_t n) {
  if (n < INT32_MIN || n > INT32_MAX) raise(PyExc_ValueError, "a size does not fit 32 bits");
  return int(n);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return float(v);
}

// A stream handle, or (None) the current stream of the current device.
void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  return reinterpret_cast<void*>(static_cast<uintptr_t>(integer(o)));
}

// Around a library call: no lookup of pointers that are known to be the current
// device's, as all of them are where the tensors say so.  (Otherwise the
// library looks them up, and refuses the call with its own error.)
class Pointers {
 public:
  Pointers(std::initializer_list<const Tensor*> all) {
    const auto device = c10::cuda::current_device();
    for (const Tensor* t : all)
      if (t != nullptr && !(t->is_cuda() && t->get_device() == device)) return;
    before_ = gqa_attn_set_pointer_checks(0);
  }
  ~Pointers() {
    if (before_ > 0) gqa_attn_set_pointer_checks(before_);
  }
  Pointers(const Pointers&) = delete;

 private:
  int before_ = 0;
};

struct Workspace {
  const Tensor* t;
  void* p;
  size_t bytes;
  explicit Workspace(PyObject* o) {
    t = tensor(o);
    p = dense(t);
    bytes = size_t(t->numel()) * t->element_size();
  }
};

// [T, H, D] with dense heads; the tokens may be further apart.
const void* heads(const Tensor* t, int64_t T, int64_t H, int64_t D, int64_t* stride) {
  if (!shaped(t, {T, H, D})) raise(PyExc_ValueError, "q is [T, Hq, D], k and v are [T, Hkv, D]");
  if (t->stride(2) != 1 || (t->stride(1) != D && H > 1))
    raise(PyExc_ValueError, "the heads of a token must be contiguous");
  *stride = T > 1 ? t->stride(0) : H * D;
  return t->data_ptr();
}

int step_tables(PyObject* const* a) {
  const Tensor *prior = tensor(a[0]), *fresh = tensor(a[1]), *table = tensor(a[2], true), *stack = tensor(a[3], true),
               *count = tensor(a[4], true), *kv = tensor(a[5]), *q_lens = tensor(a[6]), *starts = tensor(a[7]),
               *pos = tensor(a[8]), *slots = tensor(a[9]), *q_slots = tensor(a[10], true),
               *count_out = tensor(a[11], true);
  const int64_t B = prior->numel(), T = pos->numel();
  int64_t max_blocks = 0, num_blocks = 0;
  if (table != nullptr) {
    rank(table, 2, "block_table is [B, max_blocks]");
    max_blocks = table->size(1);
    num_blocks = stack == nullptr ? 0 : stack->numel();
  }
  const int32_t *p_prior = ints(prior, B), *p_new = ints(fresh, B), *p_count = ints(count, 1);
  int32_t *p_table = ints(table, B * max_blocks), *p_stack = ints(stack, num_blocks), *p_kv = ints(kv, B),
          *p_q = ints(q_lens, B), *p_starts = ints(starts, B + 1), *p_pos = ints(pos, T), *p_slots = ints(slots, T),
          *p_qs = ints(q_slots, T), *p_out = ints(count_out, 1);
  const int b = size(B), t = size(T), bs = size(integer(a[12])), nb = size(num_blocks), mb = size(max_blocks),
            rows = size(integer(a[13]));
  const Workspace ws(a[14]);
  void* const stream = stream_of(a[15]);
  const Pointers known({prior, fresh, table, stack, count, kv, q_lens, starts, pos, slots, q_slots, count_out, ws.t});
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = gqa_attn_step_tables(p_prior, p_new, p_table, p_stack, p_count, p_kv, p_q, p_starts, p_pos, p_slots, p_qs,
                            p_out, b, t, bs, nb, mb, rows, ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return rc;
}

int rope_append(PyObject* const* a) {
  const Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *wq = tensor(a[3], true),
               *wk = tensor(a[4], true), *cs = tensor(a[6], true), *pos = tensor(a[7], true), *slots = tensor(a[8]),
               *q_slots = tensor(a[9], true), *q_out = tensor(a[10]), *kc = tensor(a[11]), *vc = tensor(a[12]);
  rank(q, 3, "q is [T, Hq, D]");
  rank(k, 3, "k is [T, Hkv, D]");
  rank(q_out, 4, "q_out is [groups, Hq, q_rows, D]");
  rank(kc, 4, "k_cache and v_cache are [blocks, Hkv, block_size, D]");
  const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2), Hkv = k->size(1);
  if (q_out->size(1) != Hq || q_out->size(3) != D || kc->size(1) != Hkv || kc->size(3) != D ||
      vc->sizes() != kc->sizes())
    raise(PyExc_ValueError, "q_out is [groups, Hq, q_rows, D], k_cache and v_cache [blocks, Hkv, block_size, D]");
  one_dtype(q, {k, v, wq, wk, q_out, kc, vc});
  for (const Tensor* w : {wq, wk})
    if (w != nullptr && w->numel() != D) raise(PyExc_ValueError, "the norm weights have D entries");
  int64_t max_pos = 0, rot = 0;
  if (cs == nullptr) {
    pos = nullptr;  // nothing rotates
  } else {
    if (cs->scalar_type() != at::kFloat || pos == nullptr)
      raise(PyExc_TypeError, "cos_sin is float32 and needs positions");
    rank(cs, 2, "cos_sin is [max_pos, rot_dim]");
    max_pos = cs->size(0);
    rot = cs->size(1);
  }
  int64_t qs, ks, vs;
  const void *qp = heads(q, T, Hq, D, &qs), *kp = heads(k, T, Hkv, D, &ks), *vp = heads(v, T, Hkv, D, &vs);
  const void *pq = dense(wq), *pk = dense(wk);
  const float* pcs = static_cast<const float*>(dense(cs));
  const int32_t *ppos = ints(pos, T), *pslots = ints(slots, T), *pqs = ints(q_slots, T);
  void *po = dense(q_out), *pkc = dense(kc), *pvc = dense(vc);
  const float eps = number(a[5]);
  const int adjacent = PyObject_IsTrue(a[13]);
  if (adjacent < 0) throw Raised();
  const int t = size(T), hq = size(Hq), hkv = size(Hkv), d = size(D), r = size(rot), mp = size(max_pos),
            nb = size(kc->size(0)), bs = size(kc->size(2)), qg = size(q_out->size(0)), qr = size(q_out->size(2)),
            dt = dtype_code(q);
  const Workspace ws(a[14]);
  void* const stream = stream_of(a[15]);
  const Pointers known({q, k, v, wq, wk, cs, pos, slots, q_slots, q_out, kc, vc, ws.t});
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = gqa_attn_rope_append(qp, kp, vp, qs, ks, vs, pq, pk, eps, pcs, ppos, pslots, pqs, po, pkc, pvc, t, hq, hkv, d,
                            r, mp, adjacent, nb, bs, qg, qr, dt, ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return rc;
}

// A bound that defaults to the capacity.
int bound(PyObject* o, int64_t capacity) { return size(o == Py_None ? capacity : integer(o)); }

int decode_shared_prefix(PyObject* const* a) {
  const Tensor *q = tensor(a[0]), *kp = tensor(a[1]), *vp = tensor(a[2]), *plen = tensor(a[3], true),
               *k = tensor(a[4]), *v = tensor(a[5]), *lens = tensor(a[6], true), *o = tensor(a[7]);
  rank(q, 4, "q is [B, Hq, 1, D]");
  rank(kp, 3, "k_prefix is [Hkv, P_cap, D]");
  rank(k, 4, "k is [B, Hkv, S_cap, D]");
  const int64_t B = q->size(0), Hq = q->size(1), D = q->size(3), Hkv = kp->size(0), P = kp->size(1), S = k->size(2);
  if (q->size(2) != 1) raise(PyExc_ValueError, "decode takes one query row per request");
  if (!shaped(k, {B, Hkv, S, D}) || v->sizes() != k->sizes() || !shaped(vp, {Hkv, P, D}) || kp->size(2) != D ||
      o->sizes() != q->sizes())
    raise(PyExc_ValueError, "k_prefix and v_prefix are [Hkv, P_cap, D], k and v [B, Hkv, S_cap, D], o as q");
  one_dtype(q, {kp, vp, k, v, o});
  const void *pq = dense(q), *pkp = dense(kp), *pvp = dense(vp), *pk = dense(k), *pv = dense(v);
  const int32_t *pp = ints(plen, 1), *pl = ints(lens, B);
  void* const po = dense(o);
  const float scale = number(a[8]);
  const int b = size(B), hq = size(Hq), hkv = size(Hkv), d = size(D), p = size(P), mp = bound(a[10], P), s = size(S),
            mk = bound(a[11], S), dt = dtype_code(q);
  const Workspace ws(a[9]);
  void* const stream = stream_of(a[12]);
  const Pointers known({q, kp, vp, plen, k, v, lens, o, ws.t});
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = gqa_attn_decode_shared_prefix(pq, pkp, pvp, pp, pk, pv, pl, po, b, hq, hkv, d, p, mp, s, mk, scale, dt, ws.p,
                                     ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return rc;
}

int decode_shared_prefix_paged(PyObject* const* a) {
  const Tensor *q = tensor(a[0]), *kp = tensor(a[1]), *vp = tensor(a[2]), *ptable = tensor(a[3]),
               *plen = tensor(a[4], true), *table = tensor(a[5]), *lens = tensor(a[6]), *o = tensor(a[7]);
  rank(q, 4, "q is [B, Hq, 1, D]");
  rank(kp, 4, "k_pool is [blocks, Hkv, block_size, D]");
  rank(table, 2, "block_table is [B, max_blocks]");
  const int64_t B = q->size(0), Hq = q->size(1), D = q->size(3), n_prefix = ptable->numel(),
                max_blocks = table->size(1);
  if (q->size(2) != 1) raise(PyExc_ValueError, "decode takes one query row per request");
  if (vp->sizes() != kp->sizes() || kp->size(3) != D || o->sizes() != q->sizes())
    raise(PyExc_ValueError, "k_pool and v_pool are [blocks, Hkv, block_size, D], o as q");
  one_dtype(q, {kp, vp, o});
  const void *pq = dense(q), *pk = dense(kp), *pv = dense(vp);
  const int32_t *pt = ints(ptable, n_prefix), *pp = ints(plen, 1), *tb = ints(table, B * max_blocks),
                *pl = ints(lens, B);
  void* const po = dense(o);
  const float scale = number(a[8]);
  const int b = size(B), hq = size(Hq), hkv = size(kp->size(1)), d = size(D), bs = size(kp->size(2)),
            nb = size(kp->size(0)), np = size(n_prefix), mb = size(max_blocks), mp = size(integer(a[10])),
            mk = size(integer(a[11])), dt = dtype_code(q);
  const Workspace ws(a[9]);
  void* const stream = stream_of(a[12]);
  const Pointers known({q, kp, vp, ptable, plen, table, lens, o, ws.t});
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = gqa_attn_decode_shared_prefix_paged(pq, pk, pv, pt, pp, tb, pl, po, b, hq, hkv, d, bs, nb, np, mb, mp, mk,
                                           scale, dt, ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return rc;
}

// Attention of drafted rows; the dense (o at 7) and the paged call (8) differ in
// the cache, and in the block table before the mask.
template <bool PAGED>
int decode_tree(PyObject* const* a) {
  constexpr int T = PAGED ? 1 : 0;  // (arguments behind the block table)
  const Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *table = PAGED ? tensor(a[3]) : nullptr,
               *mask = tensor(a[3 + T], true), *q_lens = tensor(a[4 + T], true), *tree_lens = tensor(a[5 + T], true),
               *lens = tensor(a[6 + T]), *o = tensor(a[7 + T]);
  rank(q, 4, "q is [B, Hq, Tq, D]");
  rank(k, 4, PAGED ? "k_pool is [blocks, Hkv, block_size, D]" : "k is [B, Hkv, S_cap, D]");
  const int64_t B = q->size(0), Hq = q->size(1), Tq = q->size(2), D = q->size(3);
  if (v->sizes() != k->sizes() || k->size(3) != D || o->sizes() != q->sizes() || (!PAGED && k->size(0) != B))
    raise(PyExc_ValueError, PAGED ? "k_pool and v_pool are [blocks, Hkv, block_size, D], o as q"
                                  : "k and v are [B, Hkv, S_cap, D], o as q");
  one_dtype(q, {k, v, o});
  int64_t W = 0, max_blocks = 0;
  if (mask != nullptr) {
    rank(mask, 3, "tree_mask is [B, Tq, words]");
    W = mask->size(2);
    if (!shaped(mask, {B, Tq, W})) raise(PyExc_ValueError, "tree_mask is [B, Tq, words]");
  }
  if (PAGED) {
    rank(table, 2, "block_table is [B, max_blocks]");
    max_blocks = table->size(1);
  }
  const void *pq = dense(q), *pk = dense(k), *pv = dense(v);
  const int32_t *pt = ints(table, B * max_blocks), *pm = ints(mask, B * Tq * W), *pql = ints(q_lens, B),
                *ptl = ints(tree_lens, B), *pl = ints(lens, B);
  void* const po = dense(o);
  const float scale = number(a[8 + T]);
  const int b = size(B), hq = size(Hq), hkv = size(k->size(1)), d = size(D), tq = size(Tq), w = size(W),
            rows = size(k->size(2)), nb = size(k->size(0)), mb = size(max_blocks),
            mk = bound(a[10 + T], PAGED ? max_blocks * k->size(2) : k->size(2)), dt = dtype_code(q);
  const Workspace ws(a[9 + T]);
  void* const stream = stream_of(a[11 + T]);
  const Pointers known({q, k, v, table, mask, q_lens, tree_lens, lens, o, ws.t});
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = PAGED ? gqa_attn_decode_tree_paged(pq, pk, pv, pt, pm, pql, ptl, pl, po, b, hq, hkv, d, tq, w, rows, nb, mb, mk,
                                          scale, dt, ws.p, ws.bytes, stream)
             : gqa_attn_decode_tree(pq, pk, pv, pm, pql, ptl, pl, po, b, hq, hkv, d, tq, w, rows, mk, scale, dt, ws.p,
                                    ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return rc;
}

int tree_tables(PyObject* const* a) {
  const Tensor *parents = tensor(a[0]), *tree_lens = tensor(a[1]), *q_lens = tensor(a[2], true),
               *kv = tensor(a[3], true), *starts = tensor(a[4], true), *mask = tensor(a[5]),
               *pos = tensor(a[6], true);
  rank(parents, 2, "parents is [B, N]");
  rank(mask, 3, "tree_mask is [B, Tq, words]");
  const int64_t B = parents->size(0), N = parents->size(1), Tq = mask->size(1), W = mask->size(2),
                T = pos == nullptr ? 0 : pos->numel();
  if (mask->size(0) != B) raise(PyExc_ValueError, "tree_mask is [B, Tq, words]");
  const int32_t *pp = ints(parents, B * N), *pn = ints(tree_lens, B), *pq = ints(q_lens, B), *pk = ints(kv, B),
                *ps = ints(starts, B + 1);
  int32_t *pm = ints(mask, B * Tq * W), *ppos = ints(pos, T);
  const int b = size(B), n = size(N), tq = size(Tq), w = size(W), t = size(T);
  const Workspace ws(a[7]);
  void* const stream = stream_of(a[8]);
  const Pointers known({parents, tree_lens, q_lens, kv, starts, mask, pos, ws.t});
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = gqa_attn_tree_tables(pp, pn, pq, pk, ps, pm, ppos, b, n, tq, w, t, ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return rc;
}

// K and V of one layer [blocks, Hkv, block_size, D], or of several, stacked.
struct Layers {
  int n, blocks, hkv, block_size, d, dtype;
  void *k, *v;
  Layers(const Tensor* kc, const Tensor* vc) {
    const int64_t r = kc->dim();
    if ((r != 4 && r != 5) || vc->sizes() != kc->sizes())
      raise(PyExc_ValueError, "k_cache and v_cache are [blocks, Hkv, block_size, D] or [layers, blocks, ...]");
    one_dtype(kc, {vc});
    n = r == 5 ? size(kc->size(0)) : 1;
    blocks = size(kc->size(r - 4));
    hkv = size(kc->size(r - 3));
    block_size = size(kc->size(r - 2));
    d = size(kc->size(r - 1));
    dtype = dtype_code(kc);
    k = dense(kc);
    v = dense(vc);
  }
};

int compact_rows(PyObject* const* a) {
  const Tensor *path = tensor(a[0]), *keep = tensor(a[1]), *tree_lens = tensor(a[2]), *lens = tensor(a[3]),
               *table = tensor(a[4], true), *kc = tensor(a[5]), *vc = tensor(a[6]), *out = tensor(a[7]);
  rank(path, 2, "path is [B, P]");
  const int64_t B = path->size(0), P = path->size(1);
  int64_t max_blocks = 0;
  if (table != nullptr) {
    rank(table, 2, "block_table is [B, max_blocks]");
    max_blocks = table->size(1);
  }
  const Layers c(kc, vc);
  const int32_t *pp = ints(path, B * P), *pk = ints(keep, B), *pn = ints(tree_lens, B), *pl = ints(lens, B),
                *pt = ints(table, B * max_blocks);
  int32_t* const po = ints(out, B);
  const int b = size(B), w = size(P), mb = size(max_blocks);
  const Workspace ws(a[8]);
  void* const stream = stream_of(a[9]);
  const Pointers known({path, keep, tree_lens, lens, table, kc, vc, out, ws.t});
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = gqa_attn_compact_rows(pp, pk, pn, pl, pt, c.k, c.v, po, c.n, b, w, c.hkv, c.d, c.block_size, c.blocks, mb,
                             c.dtype, ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return rc;
}

int fork_tables(PyObject* const* a) {
  const Tensor *src = tensor(a[0]), *keep = tensor(a[1], true), *held = tensor(a[2]), *table = tensor(a[3]),
               *shared = tensor(a[4]), *stack = tensor(a[5]), *count = tensor(a[6]), *table_out = tensor(a[7]),
               *kv = tensor(a[8]), *shared_out = tensor(a[9]), *stack_out = tensor(a[10]), *count_out = tensor(a[11]),
               *csrc = tensor(a[12]), *cdst = tensor(a[13]), *crows = tensor(a[14]);
  rank(table, 2, "block_table is [B_in, max_blocks]");
  rank(table_out, 2, "block_table_out is [B, max_blocks]");
  const int64_t B = src->numel(), B_in = held->numel(), mb = table->size(1), nb = stack->numel();
  if (table_out->size(1) != mb) raise(PyExc_ValueError, "both block tables have max_blocks columns");
  const int32_t *ps = ints(src, B), *pk = ints(keep, B), *ph = ints(held, B_in), *pt = ints(table, B_in * mb),
                *psh = ints(shared, nb), *pst = ints(stack, nb), *pc = ints(count, 1);
  int32_t *pto = ints(table_out, B * mb), *pkv = ints(kv, B), *psho = ints(shared_out, nb), *psto = ints(stack_out, nb),
          *pco = ints(count_out, 1), *pcs = ints(csrc, B), *pcd = ints(cdst, B), *pcr = ints(crows, B);
  const int bi = size(B_in), b = size(B), m = size(mb), n = size(nb), bs = size(integer(a[15]));
  const Workspace ws(a[16]);
  void* const stream = stream_of(a[17]);
  const Pointers known({src, keep, held, table, shared, stack, count, table_out, kv, shared_out, stack_out, count_out,
                        csrc, cdst, crows, ws.t});
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = gqa_attn_fork_tables(ps, pk, ph, pt, psh, pst, pc, pto, pkv, psho, psto, pco, pcs, pcd, pcr, bi, b, m, bs, n,
                            ws.p, ws.bytes, stream);
  Py_END_ALLOW_THREADS
  return rc;
}

int copy_blocks(PyObject* const* a) {
  const Tensor *src = tensor(a[0]), *dst = tensor(a[1]), *rows = tensor(a[2], true), *kc = tensor(a[3]),
               *vc = tensor(a[4]);
  const int64_t n = src->numel();
  const Layers c(kc, vc);
  const int32_t *ps = ints(src, n), *pd = ints(dst, n), *pr = ints(rows, n);
  const int m = size(n);
  const Workspace ws(a[5]);
  void* const stream = stream_of(a[6]);
  const Pointers known({src, dst, rows, kc, vc, ws.t});
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = gqa_attn_copy_blocks(ps, pd, pr, c.k, c.v, c.n, m, c.hkv, c.d, c.block_size, c.blocks, c.dtype, ws.p, ws.bytes,
                            stream);
  Py_END_ALLOW_THREADS
  return rc;
}

template <int (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", N, n);
  try {
    return PyLong_FromLong(F(args));
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {  // (from torch)
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <int (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<step_tables, 16>("step_tables"), method<rope_append, 16>("rope_append"),
                         method<decode_shared_prefix, 13>("decode_shared_prefix"),
                         method<decode_shared_prefix_paged, 13>("decode_shared_prefix_paged"),
                         method<decode_tree<false>, 12>("decode_tree"),
                         method<decode_tree<true>, 13>("decode_tree_paged"), method<tree_tables, 9>("tree_tables"),
                         method<compact_rows, 10>("compact_rows"), method<fork_tables, 18>("fork_tables"),
                         method<copy_blocks, 7>("copy_blocks"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_call", "Native calls of libgqa_attn on torch tensors.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_call() {
  PyObject* m = PyModule_Create(&module);
  // (binding.py uses the module with the torch it was built for alone)
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", GQA_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
