// The way from PyTorch's tensors to the C entries of the operators around the
// KL, natively: some of their kernels take 3 to 6 us, and reading types, sizes,
// strides and addresses and making the outputs took more in Python. A call, from
// ops.py's way to this one: norm and rotation of 256 tokens 20.5 -> 5.9 us, their
// gradients (4,099 tokens) 33.3 -> 11.1, an append of 64 tokens 11.1 -> 3.5, one
// token's attention 21.1 -> 8.9.
//
// Each call here takes the arguments that are as the documentation wants them,
// and returns None, with nothing launched, for all others: another kind of
// tensor, outputs that the caller made, another current device, nothing to do,
// any refusal of the C entry or exception on the way. ops.py then makes the call
// itself and says what is wrong with it. So no refusal is worded here, and none
// is left out: whatever passes here passes there. A launch that failed is another
// matter: a kernel of the call may run already, and some calls change their arguments
// in place, so the status is returned, for ops.py to raise, and nothing made again.
#include <Python.h>
#include <dlfcn.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <utility>

#include "streamkl.h"

namespace {

// The entries of one build of the library.
struct Entries {
  decltype(&streamkl_qk_norm_rope_fwd) rope_fwd;
  decltype(&streamkl_qk_norm_rope_bwd) rope_bwd;
  decltype(&streamkl_qk_norm_rope_bwd_workspace_size) rope_bwd_size;
  decltype(&streamkl_paged_append) append;
  decltype(&streamkl_paged_attn) attn;
  decltype(&streamkl_paged_attn_workspace_size) attn_size;
  decltype(&streamkl_paged_tree_attn) tree;
  decltype(&streamkl_paged_tree_attn_workspace_size) tree_size;
  decltype(&streamkl_paged_compact) compact;
  decltype(&streamkl_paged_copy) copy;
  decltype(&streamkl_paged_fork) fork;
  decltype(&streamkl_paged_resize) resize;
};

// An argument that is not for here.
struct Other {};

void want(bool good) {
  if (!good) throw Other{};
}

// A call's arguments as they are read one after the other.
struct Args {
  PyObject* const* at;
  PyObject* next() { return *at++; }

  const Entries& entries() {
    void* p = PyCapsule_GetPointer(next(), nullptr);
    want(p != nullptr);
    return *static_cast<const Entries*>(p);
  }
  // a plain tensor on the GPU; nullptr for None, where that may be
  const at::Tensor* tensor(bool may_be_none = false) {
    PyObject* o = next();
    if (o == Py_None) {
      want(may_be_none);
      return nullptr;
    }
    want(THPVariable_CheckExact(o));
    const at::Tensor& t = THPVariable_Unpack(o);
    want(t.is_cuda() && t.layout() == at::kStrided);
    return &t;
  }
  int integer() {
    PyObject* o = next();
    want(PyLong_CheckExact(o));
    int over = 0;
    const long v = PyLong_AsLongAndOverflow(o, &over);
    want(!over && v >= INT_MIN && v <= INT_MAX);
    return static_cast<int>(v);
  }
  int integer_or(int none) {
    if (*at != Py_None) return integer();
    ++at;
    return none;
  }
  float real() {
    PyObject* o = next();
    want(PyFloat_CheckExact(o));
    const double v = PyFloat_AS_DOUBLE(o);
    want(std::fabs(v) < 1e38);  // (as a float, too)
    return static_cast<float>(v);
  }
  int flag() {
    PyObject* o = next();
    want(PyBool_Check(o));
    return o == Py_True;
  }
};

int fits(int64_t n) {
  want(n >= 0 && n <= INT_MAX);
  return static_cast<int>(n);
}

int type_of(at::ScalarType t) {
  if (t == at::kBFloat16) return STREAMKL_BF16;
  if (t == at::kHalf) return STREAMKL_FP16;
  want(t == at::kFloat);
  return STREAMKL_FP32;
}

// What every tensor of a call has to share; the device has to be the current one.
struct Home {
  at::Device device;
  at::ScalarType type;
  explicit Home(const at::Tensor& t) : device(t.device()), type(t.scalar_type()) {
    want(c10::cuda::current_device() == device.index());
  }
  void rows(const at::Tensor& t, int dim) const {  // of contiguous elements
    want(t.dim() == dim && t.scalar_type() == type && t.device() == device && t.stride(dim - 1) == 1);
  }
  void list(const at::Tensor& t, int64_t n, at::ScalarType ty) const {  // a contiguous vector
    want(t.dim() == 1 && t.size(0) == n && t.scalar_type() == ty && t.device() == device && t.is_contiguous());
  }
  float* weight(const at::Tensor* t, int64_t d) const {
    if (t == nullptr) return nullptr;
    list(*t, d, at::kFloat);
    return static_cast<float*>(t->data_ptr());
  }
  // (past the dispatcher: 0.5 us an output)
  at::Tensor make(at::IntArrayRef sizes, at::ScalarType ty) const {
    return at::Tensor(at::detail::empty_cuda(sizes, ty, device, std::nullopt));
  }
  // the status word, made here unless given
  int* status(const at::Tensor* given, at::Tensor* made) const {
    if (given == nullptr) {
      *made = at::zeros({1}, at::TensorOptions().dtype(at::kInt).device(device));
      return static_cast<int*>(made->data_ptr());
    }
    want(given->scalar_type() == at::kInt && given->device() == device && given->numel() >= 1);
    return static_cast<int*>(given->data_ptr());
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
};

// A launch that failed.
struct Failed {
  streamkl_status status;
};

// The launch, other threads running meanwhile; throws unless it went well.
template <typename F, typename A>
void launch(F entry, const A& args, const Home& home) {
  void* stream = home.stream();
  PyThreadState* state = PyEval_SaveThread();
  const streamkl_status st = entry(&args, stream);
  PyEval_RestoreThread(state);
  if (st == STREAMKL_ERR_CUDA) throw Failed{st};
  want(st == STREAMKL_OK);
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Failed& failed) {
    PyErr_Clear();
    return PyLong_FromLong(failed.status);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// A tuple of tensors, None for the undefined ones.
template <typename... T>
PyObject* tuple(const T&... t) {
  const at::Tensor* all[] = {&t...};
  PyObject* out = PyTuple_New(sizeof...(t));
  want(out != nullptr);
  for (size_t i = 0; i < sizeof...(t); ++i) {
    PyObject* o = Py_None;
    if (all[i]->defined())
      o = THPVariable_Wrap(*all[i]);
    else
      Py_INCREF(o);
    want(o != nullptr);
    PyTuple_SET_ITEM(out, i, o);
  }
  return out;
}

// Queries or keys of a norm + rotation call: [B, N, H, d], or packed
// [total, H, d] with positions.
struct Side {
  const at::Tensor* x;
  int B = 1, N = 0, H = 0, d = 0, repeat;
  bool packed;
  streamkl_rows in{};
  const int* positions = nullptr;
  long long pos_stride = 0;
  float* weight = nullptr;

  Side(const Home& home, const at::Tensor* t, bool packed_, const at::Tensor* pos, const at::Tensor* w, int repeat_)
      : x(t), repeat(repeat_), packed(packed_) {
    if (t == nullptr) return;
    const int o = packed ? 0 : 1;
    home.rows(*t, 3 + o);
    if (!packed) B = fits(t->size(0));
    N = fits(t->size(o));
    H = fits(t->size(o + 1));
    d = fits(t->size(o + 2));
    in = {t->data_ptr(), {packed ? 0 : t->stride(0), t->stride(o), t->stride(o + 1)}};
    want(B > 0 && N > 0 && H > 0 && (pos != nullptr || !packed));
    if (pos != nullptr) {
      want(pos->scalar_type() == at::kInt && pos->device() == home.device);
      if (pos->dim() == 2) {
        want(!packed && pos->size(0) == B && pos->size(1) == N && pos->stride(0) >= 0 && (N == 1 || pos->stride(1) == 1));
        pos_stride = pos->stride(0);
      } else {
        want(pos->dim() == 1 && pos->size(0) == N && (N == 1 || pos->stride(0) == 1));
      }
      positions = static_cast<const int*>(pos->data_ptr());
    }
    weight = home.weight(w, d);
  }
  // heads before the tokens unless packed
  at::Tensor make_outer(const Home& home, streamkl_rows* r) const {
    if (x == nullptr) return {};
    const long long heads = static_cast<long long>(H) * repeat;
    at::Tensor y = packed ? home.make({N, heads, d}, home.type) : home.make({B, heads, N, d}, home.type);
    *r = {y.data_ptr(), {packed ? 0 : heads * N * d, packed ? heads * d : d, packed ? d : static_cast<long long>(N) * d}};
    return y;
  }
  void outer(const Home& home, const at::Tensor* g, streamkl_rows* r) const {
    if (x == nullptr) return;
    want(g != nullptr);
    home.rows(*g, packed ? 3 : 4);
    const long long heads = static_cast<long long>(H) * repeat;
    if (packed) {
      want(g->size(0) == N && g->size(1) == heads && g->size(2) == d);
      *r = {g->data_ptr(), {0, g->stride(0), g->stride(1)}};
    } else {
      want(g->size(0) == B && g->size(1) == heads && g->size(2) == N && g->size(3) == d);
      *r = {g->data_ptr(), {g->stride(0), g->stride(2), g->stride(1)}};
    }
  }
  at::Tensor make_grad(const Home& home, streamkl_rows* r) const {
    if (x == nullptr) return {};
    at::Tensor y = home.make(x->sizes(), home.type);
    const long long h = d, t = h * H;
    *r = {y.data_ptr(), {packed ? 0 : t * N, t, h}};
    return y;
  }
};

void tables(const Home& home, const at::Tensor* cos, const at::Tensor* sin, int* len, int* rot) {
  for (const at::Tensor* t : {cos, sin})
    want(t->dim() == 2 && t->scalar_type() == at::kFloat && t->device() == home.device && t->is_contiguous());
  want(cos->sizes() == sin->sizes());
  *len = fits(cos->size(0));
  *rot = fits(2 * cos->size(1));
}

struct RopeCall {
  const at::Tensor *q, *k, *dq, *dk, *cos, *sin, *qpos, *kpos, *wq, *wk, *status;
  float eps;
  int interleaved, repeat;
};

// Checks and fields that both directions share.
streamkl_rope_args rope_args(const RopeCall& c, const Home& home, const Side& q, const Side& k) {
  want(c.q == nullptr || c.k == nullptr || (q.B == k.B && q.d == k.d));
  const Side& x = c.q != nullptr ? q : k;
  streamkl_rope_args u{};
  u.struct_size = sizeof(u);
  u.q = q.in, u.k = k.in;
  u.cos = static_cast<const float*>(c.cos->data_ptr()), u.sin = static_cast<const float*>(c.sin->data_ptr());
  tables(home, c.cos, c.sin, &u.table_len, &u.rot);
  u.q_positions = q.positions, u.q_pos_stride = q.pos_stride;
  u.k_positions = k.positions, u.k_pos_stride = k.pos_stride;
  u.q_weight = q.weight, u.k_weight = k.weight;
  u.dtype = type_of(home.type);
  u.B = x.B, u.NQ = q.N, u.NK = k.N, u.HQ = q.H, u.HK = k.H, u.d = x.d;
  u.interleaved = c.interleaved, u.k_repeat = c.repeat, u.eps = c.eps;
  return u;
}

// The tensor that a call goes by, and the keys' positions.
const at::Tensor& rope_lead(RopeCall* c) {
  const at::Tensor* x = c->q != nullptr ? c->q : c->k;
  want(x != nullptr && (x->dim() == 3 || x->dim() == 4) && c->repeat >= 1);
  if (c->kpos == nullptr && c->qpos != nullptr && c->k != nullptr) {
    want(c->q == nullptr || c->q->dim() != c->k->dim() || c->q->size(-3) == c->k->size(-3));
    c->kpos = c->qpos;
  }
  return *x;
}

// rope_fwd(entries, q, k, cos, sin, positions, k_positions, q_weight, k_weight, eps, interleaved, k_repeat, dev_status)
PyObject* rope_fwd(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n == 13);
    Args a{argv};
    const Entries& lib = a.entries();
    RopeCall c{};
    c.q = a.tensor(true), c.k = a.tensor(true), c.cos = a.tensor(), c.sin = a.tensor();
    c.qpos = a.tensor(true), c.kpos = a.tensor(true), c.wq = a.tensor(true), c.wk = a.tensor(true);
    c.eps = a.real(), c.interleaved = a.flag(), c.repeat = a.integer(), c.status = a.tensor(true);
    const at::Tensor& x = rope_lead(&c);
    const Home home(x);
    const Side q(home, c.q, x.dim() == 3, c.qpos, c.wq, 1), k(home, c.k, x.dim() == 3, c.kpos, c.wk, c.repeat);
    streamkl_rope_args u = rope_args(c, home, q, k);
    const at::Tensor yq = q.make_outer(home, &u.q_out), yk = k.make_outer(home, &u.k_out);
    at::Tensor word;
    u.dev_status = home.status(c.status, &word);
    launch(lib.rope_fwd, u, home);
    return tuple(yq, yk);
  });
}

// rope_bwd(entries, q, k, dq_out, dk_out, cos, sin, positions, k_positions, q_weight, k_weight, eps, interleaved,
//          k_repeat, workspace, dev_status)
PyObject* rope_bwd(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n == 16);
    Args a{argv};
    const Entries& lib = a.entries();
    RopeCall c{};
    c.q = a.tensor(true), c.k = a.tensor(true), c.dq = a.tensor(true), c.dk = a.tensor(true);
    c.cos = a.tensor(), c.sin = a.tensor();
    c.qpos = a.tensor(true), c.kpos = a.tensor(true), c.wq = a.tensor(true), c.wk = a.tensor(true);
    c.eps = a.real(), c.interleaved = a.flag(), c.repeat = a.integer();
    const at::Tensor* given = a.tensor(true);
    c.status = a.tensor(true);
    const at::Tensor& x = rope_lead(&c);
    const Home home(x);
    const Side q(home, c.q, x.dim() == 3, c.qpos, c.wq, 1), k(home, c.k, x.dim() == 3, c.kpos, c.wk, c.repeat);
    streamkl_rope_args u = rope_args(c, home, q, k);
    q.outer(home, c.dq, &u.q_out);
    k.outer(home, c.dk, &u.k_out);
    const at::Tensor dq = q.make_grad(home, &u.dq), dk = k.make_grad(home, &u.dk);
    at::Tensor dwq, dwk, word, space;
    if (q.weight != nullptr) u.dq_weight = static_cast<float*>((dwq = home.make({u.d}, at::kFloat)).data_ptr());
    if (k.weight != nullptr) u.dk_weight = static_cast<float*>((dwk = home.make({u.d}, at::kFloat)).data_ptr());
    if (dwq.defined() || dwk.defined()) {
      u.ws_bytes = lib.rope_bwd_size(u.B, u.NQ, u.NK, u.HQ, u.HK, u.d);
      if (given != nullptr) {
        want(given->device() == home.device && given->is_contiguous() && given->nbytes() >= u.ws_bytes);
        u.workspace = given->data_ptr();
      } else {
        u.workspace = (space = home.make({static_cast<int64_t>(u.ws_bytes)}, at::kByte)).data_ptr();
      }
    }
    u.dev_status = home.status(c.status, &word);
    launch(lib.rope_bwd, u, home);
    return tuple(dq, dk, dwq, dwk);
  });
}

// The fields of the paged cache, in the struct of either call; the sequences
// and their heads as the caches have them.
template <typename U>
void cache_args(U* u, const Home& home, const at::Tensor& kc, const at::Tensor& vc, const at::Tensor& table,
                const at::Tensor& lens, const at::Tensor* cu, int total, int d) {
  want(home.type == at::kBFloat16 || home.type == at::kHalf);
  home.rows(kc, 4);
  home.rows(vc, 4);
  want(kc.sizes() == vc.sizes() && kc.size(3) == d);
  want(table.scalar_type() == at::kInt && table.device() == home.device && table.dim() == 2);
  want(table.size(1) <= 1 || table.stride(1) == 1);
  u->struct_size = sizeof(*u);
  u->k_cache = {kc.data_ptr(), {kc.stride(0), kc.stride(1), kc.stride(2)}};
  u->v_cache = {vc.data_ptr(), {vc.stride(0), vc.stride(1), vc.stride(2)}};
  u->block_table = static_cast<const int*>(table.data_ptr());
  u->table_stride = table.stride(0);
  u->B = fits(table.size(0));
  home.list(lens, u->B, at::kInt);
  u->kv_lens = static_cast<const int*>(lens.data_ptr());
  if (cu != nullptr) {
    home.list(*cu, static_cast<int64_t>(u->B) + 1, at::kInt);
    u->cu_seqlens = static_cast<const int*>(cu->data_ptr());
  } else {
    want(total == u->B);
  }
  u->dtype = type_of(home.type);
  u->T = total;
  u->d = d;
  u->num_pages = fits(kc.size(0)), u->HK = fits(kc.size(1)), u->page_size = fits(kc.size(2));
  u->max_pages = fits(table.size(1));
  want(total > 0 && u->B > 0 && u->HK > 0);
}

// append(entries, k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens, cos, sin, k_weight, eps, interleaved,
//        dev_status); True when done
PyObject* append(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n == 14);
    Args a{argv};
    const Entries& lib = a.entries();
    const at::Tensor *k = a.tensor(), *v = a.tensor(), *kc = a.tensor(), *vc = a.tensor(), *table = a.tensor(),
                     *lens = a.tensor(), *cu = a.tensor(true), *cos = a.tensor(true), *sin = a.tensor(true),
                     *w = a.tensor(true);
    streamkl_append_args u{};
    u.eps = a.real(), u.interleaved = a.flag();
    const at::Tensor* status = a.tensor(true);
    const Home home(*kc);
    home.rows(*k, 3);
    home.rows(*v, 3);
    want(k->sizes() == v->sizes() && (cos == nullptr) == (sin == nullptr));
    cache_args(&u, home, *kc, *vc, *table, *lens, cu, fits(k->size(0)), fits(k->size(2)));
    want(k->size(1) == u.HK);
    u.k = {k->data_ptr(), {0, k->stride(0), k->stride(1)}};
    u.v = {v->data_ptr(), {0, v->stride(0), v->stride(1)}};
    if (cos != nullptr) {
      tables(home, cos, sin, &u.table_len, &u.rot);
      u.cos = static_cast<const float*>(cos->data_ptr()), u.sin = static_cast<const float*>(sin->data_ptr());
    }
    u.k_weight = home.weight(w, u.d);
    at::Tensor word;
    u.dev_status = home.status(status, &word);
    launch(lib.append, u, home);
    Py_RETURN_TRUE;
  });
}

// The attention over the cache, of drafted tokens (`tree`) or not.
PyObject* attn_call(Args a, bool tree) {
  const Entries& lib = a.entries();
  const at::Tensor *q = a.tensor(), *kc = a.tensor(), *vc = a.tensor(), *table = a.tensor(), *lens = a.tensor();
  const at::Tensor* mask = tree ? a.tensor() : nullptr;
  const at::Tensor* cu = a.tensor(true);
  streamkl_paged_tree_attn_args t{};
  streamkl_paged_attn_args& u = t.attn;
  u.max_seqlen_q = a.integer_or(INT_MIN), u.max_kv_len = a.integer_or(INT_MIN);
  const bool scaled = *a.at != Py_None;
  if (scaled)
    u.scale = a.real();
  else
    a.next();
  if (!tree) u.causal = a.flag(), u.num_splits = a.integer();
  const at::Tensor *given = a.tensor(true), *status = a.tensor(true);
  const Home home(*kc);
  home.rows(*q, 3);
  cache_args(&u, home, *kc, *vc, *table, *lens, cu, fits(q->size(0)), fits(q->size(2)));
  u.HQ = fits(q->size(1));
  want(u.HQ > 0 && u.HQ % u.HK == 0 && u.num_splits >= 0);
  if (!scaled) u.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(u.d)));
  if (u.max_seqlen_q == INT_MIN) {
    u.max_seqlen_q = cu != nullptr ? u.T : 1;
    if (tree && mask->dim() == 2) u.max_seqlen_q = static_cast<int>(std::min<int64_t>(u.max_seqlen_q, 32 * mask->size(1)));
  }
  if (u.max_kv_len == INT_MIN) u.max_kv_len = fits(static_cast<int64_t>(u.page_size) * u.max_pages);
  if (tree) {
    want(mask->dim() == 2 && mask->scalar_type() == at::kInt && mask->device() == home.device);
    want(mask->size(0) == u.T && mask->size(1) > 0 && mask->stride(1) == 1);
    t.struct_size = sizeof(t);
    t.mask = static_cast<const int*>(mask->data_ptr());
    t.mask_stride = mask->stride(0);
    t.mask_words = fits(mask->size(1));
  }
  u.q = {q->data_ptr(), {0, q->stride(0), q->stride(1)}};
  const at::Tensor o = home.make(q->sizes(), home.type), lse = home.make({u.T, u.HQ}, at::kFloat);
  u.out = {o.data_ptr(), {0, static_cast<long long>(u.HQ) * u.d, u.d}};
  u.lse = static_cast<float*>(lse.data_ptr());
  at::Tensor word, space;
  if (given != nullptr) {
    want(given->device() == home.device && given->is_contiguous());
    u.workspace = given->data_ptr(), u.ws_bytes = given->nbytes();
  } else {
    u.ws_bytes = tree ? lib.tree_size(u.B, u.T, u.HQ, u.HK, u.d, u.max_seqlen_q, u.max_kv_len)
                      : lib.attn_size(u.B, u.T, u.HQ, u.HK, u.d, u.max_seqlen_q, u.max_kv_len, u.num_splits);
    u.workspace = (space = home.make({static_cast<int64_t>(u.ws_bytes)}, at::kByte)).data_ptr();
  }
  u.dev_status = home.status(status, &word);
  if (tree)
    launch(lib.tree, t, home);
  else
    launch(lib.attn, u, home);
  return tuple(o, lse);
}

// attn(entries, q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, max_seqlen_q, max_kv_len, scale, causal,
//      num_splits, workspace, dev_status)
PyObject* attn(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n == 14);
    return attn_call(Args{argv}, false);
  });
}

// tree_attn(entries, q, k_cache, v_cache, block_table, kv_lens, tree_mask, cu_seqlens, max_seqlen_q, max_kv_len, scale,
//           workspace, dev_status)
PyObject* tree_attn(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n == 13);
    return attn_call(Args{argv}, true);
  });
}

// compact(entries, k_cache, v_cache, block_table, kv_lens, cu_seqlens, kept, num_kept, dev_status); True when done
PyObject* compact(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n == 9);
    Args a{argv};
    const Entries& lib = a.entries();
    const at::Tensor *kc = a.tensor(), *vc = a.tensor(), *table = a.tensor(), *lens = a.tensor(), *cu = a.tensor(),
                     *kept = a.tensor(), *count = a.tensor(), *status = a.tensor(true);
    const Home home(*kc);
    want(kc->dim() == 4);
    struct : streamkl_compact_args {  // (with the field of the calls that take tokens)
      int T;
    } u{};
    cache_args(&u, home, *kc, *vc, *table, *lens, cu, 1, fits(kc->size(3)));
    want(kept->dim() == 2 && kept->scalar_type() == at::kInt && kept->device() == home.device);
    want(kept->size(0) == u.B && kept->size(1) > 0 && kept->stride(1) == 1);
    home.list(*count, u.B, at::kInt);
    u.kept = static_cast<const int*>(kept->data_ptr());
    u.kept_stride = kept->stride(0);
    u.max_kept = fits(kept->size(1));
    u.num_kept = static_cast<const int*>(count->data_ptr());
    at::Tensor word;
    u.dev_status = home.status(status, &word);
    streamkl_compact_args args = u;
    args.struct_size = sizeof(args);
    launch(lib.compact, args, home);
    Py_RETURN_TRUE;
  });
}

// copy(entries, k_cache, v_cache, pairs, dev_status); True when done
PyObject* copy(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n == 5);
    Args a{argv};
    const Entries& lib = a.entries();
    const at::Tensor *kc = a.tensor(), *vc = a.tensor(), *pairs = a.tensor(), *status = a.tensor(true);
    const Home home(*kc);
    home.rows(*kc, 4);
    home.rows(*vc, 4);
    want(kc->sizes() == vc->sizes() && (home.type == at::kBFloat16 || home.type == at::kHalf));
    want(pairs->dim() == 2 && pairs->size(1) == 2 && pairs->scalar_type() == at::kInt && pairs->device() == home.device &&
         pairs->is_contiguous());
    streamkl_page_copy_args u{};
    u.struct_size = sizeof(u);
    u.k_cache = {kc->data_ptr(), {kc->stride(0), kc->stride(1), kc->stride(2)}};
    u.v_cache = {vc->data_ptr(), {vc->stride(0), vc->stride(1), vc->stride(2)}};
    u.pairs = static_cast<const int*>(pairs->data_ptr());
    u.dtype = type_of(home.type);
    u.n = fits(pairs->size(0)), u.HK = fits(kc->size(1)), u.d = fits(kc->size(3));
    u.page_size = fits(kc->size(2)), u.num_pages = fits(kc->size(0));
    want(u.n > 0 && u.HK > 0);
    at::Tensor word;
    u.dev_status = home.status(status, &word);
    launch(lib.copy, u, home);
    Py_RETURN_TRUE;
  });
}

// The fields that fork and resize share.
template <typename U>
void table_args(U* u, const Home& home, const at::Tensor& refs, const at::Tensor& table, const at::Tensor& lens) {
  want(home.type == at::kInt && refs.dim() == 1 && table.dim() == 2 && table.stride(1) == 1);
  home.list(refs, refs.size(0), at::kInt);
  u->struct_size = sizeof(*u);
  u->page_refs = static_cast<int*>(refs.data_ptr());
  u->block_table = static_cast<int*>(table.data_ptr());
  u->table_stride = table.stride(0);
  u->B = fits(table.size(0));
  home.list(lens, u->B, at::kInt);
  u->kv_lens = static_cast<int*>(lens.data_ptr());
  u->num_pages = fits(refs.size(0)), u->max_pages = fits(table.size(1));
  want(u->B > 0);
}

// fork(entries, page_refs, block_table, kv_lens, source, dev_status); True when done
PyObject* fork(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n == 6);
    Args a{argv};
    const Entries& lib = a.entries();
    const at::Tensor *refs = a.tensor(), *table = a.tensor(), *lens = a.tensor(), *source = a.tensor(),
                     *status = a.tensor(true);
    const Home home(*table);
    streamkl_fork_args u{};
    table_args(&u, home, *refs, *table, *lens);
    home.list(*source, u.B, at::kInt);
    u.source = static_cast<const int*>(source->data_ptr());
    at::Tensor word;
    u.dev_status = home.status(status, &word);
    launch(lib.fork, u, home);
    Py_RETURN_TRUE;
  });
}

// resize(entries, page_refs, block_table, kv_lens, new_lens, page_size, dev_status, step_lens)
PyObject* resize(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n == 8);
    Args a{argv};
    const Entries& lib = a.entries();
    const at::Tensor *refs = a.tensor(), *table = a.tensor(), *lens = a.tensor(), *to = a.tensor();
    streamkl_resize_args u{};
    u.page_size = a.integer();
    const at::Tensor *status = a.tensor(true), *step = a.tensor(true);
    const Home home(*table);
    table_args(&u, home, *refs, *table, *lens);
    home.list(*to, u.B, at::kInt);
    if (step != nullptr) {
      home.list(*step, u.B, at::kInt);
      u.step_lens = static_cast<int*>(step->data_ptr());
    }
    u.new_lens = static_cast<const int*>(to->data_ptr());
    const at::Tensor copies = home.make({u.B, 2}, at::kInt);
    u.copies = static_cast<int*>(copies.data_ptr());
    at::Tensor word;
    u.dev_status = home.status(status, &word);
    // (made before the launch: nothing may fail behind it)
    struct Owned {
      PyObject* o;
      ~Owned() { Py_XDECREF(o); }
    } out{THPVariable_Wrap(copies)};
    want(out.o != nullptr);
    launch(lib.resize, u, home);
    return std::exchange(out.o, nullptr);
  });
}

// entries(path): those of a library that is loaded already.
PyObject* entries(PyObject*, PyObject* path) {
  const char* name = PyUnicode_AsUTF8(path);
  if (name == nullptr) return nullptr;
  void* lib = dlopen(name, RTLD_NOW | RTLD_NOLOAD);
  if (lib == nullptr) return PyErr_Format(PyExc_OSError, "%s is not loaded", name);
  auto* e = new Entries{};  // (for good, like the library)
  auto find = [&](auto* to, const char* symbol) {
    *to = reinterpret_cast<std::remove_pointer_t<decltype(to)>>(dlsym(lib, symbol));
    return *to != nullptr;
  };
  if (!(find(&e->rope_fwd, "streamkl_qk_norm_rope_fwd") && find(&e->rope_bwd, "streamkl_qk_norm_rope_bwd") &&
        find(&e->rope_bwd_size, "streamkl_qk_norm_rope_bwd_workspace_size") && find(&e->append, "streamkl_paged_append") &&
        find(&e->attn, "streamkl_paged_attn") && find(&e->attn_size, "streamkl_paged_attn_workspace_size") &&
        find(&e->tree, "streamkl_paged_tree_attn") &&
        find(&e->tree_size, "streamkl_paged_tree_attn_workspace_size") && find(&e->compact, "streamkl_paged_compact") &&
        find(&e->copy, "streamkl_paged_copy") && find(&e->fork, "streamkl_paged_fork") &&
        find(&e->resize, "streamkl_paged_resize"))) {
    delete e;
    return PyErr_Format(PyExc_OSError, "%s lacks an entry", name);
  }
  return PyCapsule_New(e, nullptr, nullptr);
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef kMethods[] = {{"entries", entries, METH_O, nullptr},
                          {"rope_fwd", FAST(rope_fwd), nullptr},
                          {"rope_bwd", FAST(rope_bwd), nullptr},
                          {"append", FAST(append), nullptr},
                          {"attn", FAST(attn), nullptr},
                          {"tree_attn", FAST(tree_attn), nullptr},
                          {"compact", FAST(compact), nullptr},
                          {"copy", FAST(copy), nullptr},
                          {"fork", FAST(fork), nullptr},
                          {"resize", FAST(resize), nullptr},
                          {nullptr, nullptr, 0, nullptr}};
#undef FAST
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
