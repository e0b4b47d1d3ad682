// The short way of the Python binding's step calls: arguments that are all as the
// library wants them (contiguous tensors of the right types on the current
// device, nothing to be allocated) are read from the tensors themselves and
// passed on.  Reading them through Python costs a call twice what launching its
// kernel does.  For any other arguments a function returns None without having
// done anything, and the caller looks at them one by one.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "qlin.h"

namespace {

struct Other {};  // arguments that are not for this way

// Arguments in order; each of the functions below takes the next one.
struct Args {
  PyObject* const* at;
  PyObject* const* end;
  int device = -1;

  PyObject* next() {
    if (at == end) throw Other();
    return *at++;
  }
  int64_t integer() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw Other();
    return v;
  }
  void* address() { return reinterpret_cast<void*>(static_cast<uintptr_t>(integer())); }
  double number() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw Other();
    return v;
  }
  // a contiguous tensor of the call's device, or none
  const at::Tensor* tensor() {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o)) throw Other();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous()) throw Other();
    return &t;
  }
  const at::Tensor* tensor(at::ScalarType type) {
    const at::Tensor* t = tensor();
    if (t && t->scalar_type() != type) throw Other();
    return t;
  }
  template <typename V>
  V* values(at::ScalarType type, int64_t n) {
    const at::Tensor* t = tensor(type);
    if (t && t->numel() != n) throw Other();
    return t ? static_cast<V*>(t->data_ptr()) : nullptr;
  }
  float* floats(int64_t n) { return values<float>(at::kFloat, n); }
  int32_t* ints(int64_t n) { return values<int32_t>(at::kInt, n); }
};

void want(bool ok) {
  if (!ok) throw Other();
}
template <typename V = void>
V* data(const at::Tensor* t) {
  return t ? static_cast<V*>(t->data_ptr()) : nullptr;
}
int code_of(const at::Tensor* t) {
  switch (t->scalar_type()) {
    case at::kBFloat16: return QLIN_BF16;
    case at::kHalf: return QLIN_F16;
    case at::kFloat: return QLIN_F32;
    default: throw Other();
  }
}
// [n, heads * width] or [n, heads, D]: elements of a row
int64_t row_of(const at::Tensor* t, int64_t n) {
  want((t->dim() == 2 || t->dim() == 3) && n > 0 && t->size(0) == n);
  return t->numel() / n;
}
size_t bytes_of(const at::Tensor* t) {
  if (!t) return 0;
  want(t->element_size() == 1);
  return (size_t)t->numel();
}

// A call of the library, its arguments formed before, while other threads run: a
// launch waits where the stream's queue is full.  (What the arguments name is held
// by the caller's frame.)
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename... P, typename... A>
qlin_status unlocked(qlin_status (*call)(P...), A... a) {
  const Unlocked other_threads_run;
  return call(a...);
}

template <typename F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, F&& f) {
  try {
    Args a{args, args + n};
    const qlin_status st = f(a);
    return PyLong_FromLong(st);
  } catch (const Other&) {
  } catch (...) {  // what a tensor refuses
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// device, cache, step, rows, width, cache heads, cache dtype, q, k, v, q_gamma, k_gamma, eps, turns, pairs, q_out, ws, flags,
// stream, position, axis
PyObject* kv_append(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded(args, nargs, [](Args& a) {
    a.device = (int)a.integer();
    const auto* cache = static_cast<const qlin_kv_cache*>(a.address());
    const auto* step = static_cast<const qlin_kv_step*>(a.address());
    const int64_t n = a.integer(), D = a.integer(), heads = a.integer(), dtype = a.integer();
    const at::Tensor *q = a.tensor(), *k = a.tensor(), *v = a.tensor();
    const float *q_gamma = a.floats(D), *k_gamma = a.floats(D);
    const float eps = (float)a.number();
    const at::Tensor* turns = a.tensor(at::kLong);
    const int pairs = a.integer() != 0;
    const at::Tensor *q_out = a.tensor(), *ws = a.tensor();
    const unsigned flags = (unsigned)a.integer();
    void* stream = a.address();
    const at::Tensor* position = a.tensor(at::kInt);
    PyObject* axis = a.next();
    want((k == nullptr) == (v == nullptr) && (q || k) && (q == nullptr) == (q_out == nullptr));
    const int src = code_of(q ? q : k);
    int64_t Hq = 0;
    if (q) {
      Hq = row_of(q, n) / D;
      want(Hq > 0 && q->numel() == n * Hq * D && code_of(q_out) == dtype && row_of(q_out, n) == Hq * D);
    }
    if (k) want(code_of(k) == src && code_of(v) == src && row_of(k, n) == heads * D && row_of(v, n) == heads * D);
    const int64_t nt = turns ? turns->numel() : 0;
    const auto* turn = nt ? data<const uint64_t>(turns) : nullptr;
    if (!position) {
      want(axis == Py_None);
      return unlocked(qlin_kv_append, cache, step, (int)Hq, src, data(q), Hq * D, data(k), heads * D, data(v), heads * D,
                      q_gamma, k_gamma, eps, turn, (int)nt, pairs, data(q_out), Hq * D, data(ws), bytes_of(ws), flags, stream);
    }
    want((position->dim() == 1 || position->dim() == 2) && position->size(0) == n);
    const int64_t axes = position->dim() == 2 ? position->size(1) : 1;
    const uint8_t* axis_of = nullptr;
    if (axis != Py_None) {
      want(PyBytes_CheckExact(axis) && PyBytes_GET_SIZE(axis) == nt && axes <= QLIN_MAX_AXES);
      axis_of = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(axis));
    }
    want(axes <= QLIN_MAX_AXES);
    return unlocked(qlin_kv_append_at, cache, step, (int)Hq, src, data(q), Hq * D, data(k), heads * D, data(v), heads * D,
                    q_gamma, k_gamma, eps, turn, (int)nt, pairs, data<const int32_t>(position), axes, (int)axes, axis_of,
                    data(q_out), Hq * D, data(ws), bytes_of(ws), flags, stream);
  });
}

// [B, heads, room], whole
float* scores_of(const at::Tensor* t, int64_t B, int64_t heads, int64_t room) {
  want(t->dim() == 3 && t->size(0) == B && t->size(1) == heads && t->size(2) == room);
  return data<float>(t);
}
int32_t* positions_of(const at::Tensor* t, int64_t B, int64_t heads, int64_t room) {
  if (!t) return nullptr;
  want(t->dim() == 3 && t->size(0) == B && t->size(1) == heads && t->size(2) == room);
  return data<int32_t>(t);
}
int64_t room_of(const at::Tensor* t) {
  want(t && t->dim() == 3);
  return t->size(2);
}

// device, cache, step, B, T, width, cache heads, cache dtype, q, stats, score, keep, n_keep, decay, scale, score_out,
// position_out, at, ws, flags, stream
PyObject* kv_weigh(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded(args, nargs, [](Args& a) {
    a.device = (int)a.integer();
    const auto* cache = static_cast<const qlin_kv_cache*>(a.address());
    const auto* step = static_cast<const qlin_kv_step*>(a.address());
    const int64_t B = a.integer(), T = a.integer(), D = a.integer(), heads = a.integer(), dtype = a.integer(), n = B * T;
    const at::Tensor *q = a.tensor(), *stats = a.tensor(at::kFloat), *score = a.tensor(at::kFloat);
    want(q && stats && score);
    const int64_t Hq = row_of(q, n) / D, room = room_of(score);
    want(code_of(q) == dtype && Hq > 0 && q->numel() == n * Hq * D && stats->dim() == 3 && stats->size(0) == n &&
         stats->size(1) == Hq && stats->size(2) == 2);
    const at::Tensor* keep = a.tensor(at::kInt);
    if (keep) want(keep->dim() == 2 && keep->size(0) == B && keep->size(1) == T);
    const int32_t* n_keep = a.ints(B);
    const float decay = (float)a.number(), scale = (float)a.number();
    const at::Tensor *score_out = a.tensor(at::kFloat), *position_out = a.tensor(at::kInt);
    const int32_t* at_ = a.ints(n);
    const at::Tensor* ws = a.tensor();
    const unsigned flags = (unsigned)a.integer();
    void* stream = a.address();
    return unlocked(qlin_kv_weigh, cache, step, (int)Hq, data(q), Hq * D, data<const float>(stats), scale,
                    data<const int32_t>(keep), T, n_keep, decay, scores_of(score, B, heads, room), heads * room, room,
                    scores_of(score_out ? score_out : score, B, heads, room), positions_of(position_out, B, heads, room),
                    heads * room, room, room, at_, data(ws), bytes_of(ws), flags, stream);
  });
}

// device, cache, step, B, cache heads, score, n_keep, first, since, position, score_out, position_out, len_out, ws, flags, stream
PyObject* kv_evict(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded(args, nargs, [](Args& a) {
    a.device = (int)a.integer();
    const auto* cache = static_cast<const qlin_kv_cache*>(a.address());
    const auto* step = static_cast<const qlin_kv_step*>(a.address());
    const int64_t B = a.integer(), heads = a.integer();
    const at::Tensor* score = a.tensor(at::kFloat);
    const int64_t room = room_of(score);
    const int32_t* n_keep = a.ints(B);
    const int64_t first = a.integer();
    const int32_t* since = a.ints(B);
    const at::Tensor *position = a.tensor(at::kInt), *score_out = a.tensor(at::kFloat), *position_out = a.tensor(at::kInt);
    int32_t* len_out = a.ints(B);
    const at::Tensor* ws = a.tensor();
    const unsigned flags = (unsigned)a.integer();
    void* stream = a.address();
    want(ws && n_keep && first >= 0 && first <= INT32_MAX);
    return unlocked(qlin_kv_evict, cache, step, scores_of(score, B, heads, room), positions_of(position, B, heads, room),
                    heads * room, room, scores_of(score_out ? score_out : score, B, heads, room),
                    positions_of(position_out ? position_out : position, B, heads, room), heads * room, room, room, n_keep,
                    (int)first, since, len_out, data(ws), bytes_of(ws), flags, stream);
  });
}

// device, logits, out, history, history_len, prompt_len, draft, mask, repetition, presence, frequency, bias_token, bias, allowed,
// flags, stream
PyObject* adjust_logits(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded(args, nargs, [](Args& a) {
    a.device = (int)a.integer();
    const at::Tensor *logits = a.tensor(), *out = a.tensor();
    want(logits && out && logits->dim() == 2 && out->dim() == 2 && out->scalar_type() == logits->scalar_type() &&
         out->sizes() == logits->sizes());
    const int64_t M = logits->size(0), V = logits->size(1);
    const at::Tensor *history = a.tensor(at::kInt), *history_len = a.tensor(at::kInt), *prompt_len = a.tensor(at::kInt);
    const at::Tensor *draft = a.tensor(at::kInt), *mask = a.tensor(at::kInt);
    const at::Tensor *repetition = a.tensor(at::kFloat), *presence = a.tensor(at::kFloat), *frequency = a.tensor(at::kFloat);
    const at::Tensor *token = a.tensor(at::kInt), *bias = a.tensor(at::kFloat), *allowed = a.tensor(at::kInt);
    const unsigned flags = (unsigned)a.integer();
    void* stream = a.address();
    const at::Tensor* of_sequences = nullptr;
    for (const at::Tensor* t : {history, draft, history_len, prompt_len, repetition, presence, frequency})
      if (t && !of_sequences) of_sequences = t;
    if (!of_sequences && token && token->dim() == 2) of_sequences = token;
    if (of_sequences) want(of_sequences->dim() > 0);
    const int64_t B = of_sequences ? of_sequences->size(0) : M > QLIN_MAX_SEQUENCES ? 1 : M;  // (rows that nothing tells apart)
    want(M > 0 && B > 0 && M % B == 0);
    const int64_t T = M / B;
    qlin_adjustments s = {};
    if (history) {
      want(history->dim() == 2 && history->size(0) == B && history->size(1) <= INT32_MAX);
      s.L = (int32_t)history->size(1), s.history_stride = s.L;
    }
    for (const at::Tensor* t : {history_len, prompt_len, repetition, presence, frequency}) want(!t || t->numel() == B);
    want(!draft || (draft->dim() == 2 && draft->size(0) == B && draft->size(1) == T));
    if (mask) {
      want(draft && ((mask->dim() == 1 && mask->size(0) == T) || (mask->dim() == 2 && mask->size(0) == B && mask->size(1) == T)));
      s.tree_stride = mask->dim() == 2 ? T : 0;
    }
    want((token == nullptr) == (bias == nullptr));
    if (token) {
      want(token->sizes() == bias->sizes() && (token->dim() == 1 || (token->dim() == 2 && token->size(0) == B)) &&
           token->size(-1) <= INT32_MAX);
      s.n_bias = (int32_t)token->size(-1), s.bias_stride = token->dim() == 2 ? s.n_bias : 0;
    }
    if (allowed) {
      want((allowed->dim() == 1 || (allowed->dim() == 2 && allowed->size(0) == M)) && allowed->size(-1) >= (V + 31) / 32);
      s.allowed_stride = allowed->dim() == 2 ? allowed->size(1) : 0;
    }
    s.history = data<const int32_t>(history), s.history_len = data<const int32_t>(history_len);
    s.prompt_len = data<const int32_t>(prompt_len), s.draft = data<const int32_t>(draft), s.mask = data<const int32_t>(mask);
    s.repetition = data<const float>(repetition), s.presence = data<const float>(presence);
    s.frequency = data<const float>(frequency), s.bias_token = data<const int32_t>(token), s.bias = data<const float>(bias);
    s.allowed = data<const int32_t>(allowed);
    return unlocked(qlin_adjust_logits, (int)B, (int)T, V, code_of(logits), data(logits), V, data(out), V, &s, flags, stream);
  });
}

PyMethodDef methods[] = {
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kv_append)), METH_FASTCALL, nullptr},
    {"kv_weigh", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kv_weigh)), METH_FASTCALL, nullptr},
    {"kv_evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kv_evict)), METH_FASTCALL, nullptr},
    {"adjust_logits", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(adjust_logits)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qlin_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qlin_binding() { return PyModule_Create(&module); }
