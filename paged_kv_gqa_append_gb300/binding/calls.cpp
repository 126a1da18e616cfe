// The usual form of the small calls, marshalled in C++.
//
// A call of one token costs the GPU 2 to 5 us, and checking a dozen tensors from
// Python and converting two dozen arguments through ctypes 6 to 12 us.  Each
// function here does the checks of the Python function of the same name on the
// tensors themselves and calls the library on the current stream.  It returns
// the library's status, or -1 whenever anything is not as the usual call has it
// -- a check that fails, an argument of another kind, a device that is not the
// current one, nothing to do.  The Python function then goes its own way: it
// says what is wrong, or makes the call.  So there is one place for errors, and
// this one never has to explain anything.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <limits.h>
#include <stdint.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "pkv.h"

namespace {

using at::ScalarType;
constexpr long kOther = -1;
constexpr int64_t kKvRow = PKV_NUM_KV_HEADS * PKV_HEAD_DIM, kQRow = PKV_NUM_Q_HEADS * PKV_HEAD_DIM;

// Reads arguments one after another; once one is not as expected, ok stays false.
struct Args {
  PyObject* const* at;
  int dev = -1;
  bool ok = true;

  const at::Tensor* tensor(int i, ScalarType type) {
    if (!ok || !THPVariable_Check(at[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(at[i]);
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type) return fail();
    return &t;
  }
  // the tensor whose device is the call's
  const at::Tensor* first(int i) {
    if (!THPVariable_Check(at[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(at[i]);
    if (!t.is_cuda()) return fail();
    dev = t.get_device();
    ok = dev == c10::cuda::current_device();
    return ok ? &t : nullptr;
  }
  bool none(int i) const { return at[i] == Py_None; }
  // a contiguous tensor of n elements
  void* vec(int i, ScalarType type, int64_t n) {
    const at::Tensor* t = tensor(i, type);
    if (!t || !t->is_contiguous() || t->numel() != n) return fail();
    return t->data_ptr();
  }
  void* opt(int i, ScalarType type, int64_t n) { return none(i) ? nullptr : vec(i, type, n); }
  void* error_word(int i) {
    if (none(i)) return nullptr;
    const at::Tensor* t = tensor(i, ScalarType::Int);
    if (!t || !t->is_contiguous() || t->numel() < 1) return fail();
    return t->data_ptr();
  }
  // token rows [tokens][heads][64] with contiguous heads; tokens < 0: any number, returned there
  void* rows(int i, int64_t heads, int64_t& tokens, long long& stride) {
    const at::Tensor* t = tensor(i, ScalarType::BFloat16);
    if (!t || t->dim() != 3 || t->size(1) != heads || t->size(2) != PKV_HEAD_DIM || t->stride(2) != 1 ||
        t->stride(1) != PKV_HEAD_DIM || (tokens >= 0 && t->size(0) != tokens))
      return fail();
    tokens = t->size(0);
    stride = tokens > 1 ? t->stride(0) : heads * PKV_HEAD_DIM;
    return t->data_ptr();
  }
  // block tables [>= rows][width]
  void* tables(int i, int64_t rows, int& all, int& width) {
    const at::Tensor* t = tensor(i, ScalarType::Int);
    if (!t || t->dim() != 2 || !t->is_contiguous() || t->size(0) < rows) return fail();
    all = to_int(t->size(0));
    width = to_int(t->size(1));
    return t->data_ptr();
  }
  int to_int(int64_t v) {
    if (v < 0 || v > INT_MAX) ok = false;
    return (int)v;
  }
  int integer(int i, int otherwise) {
    if (none(i)) return otherwise;
    if (!PyLong_Check(at[i])) return ok = false, 0;
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(at[i], &over);
    if (over || v < INT_MIN || v > INT_MAX) return ok = false, 0;
    return (int)v;
  }
  float number(int i) {
    if (!PyFloat_Check(at[i])) return ok = false, 0.f;
    return (float)PyFloat_AS_DOUBLE(at[i]);
  }
  // a block-scaled pool and its scales
  int bs8(int i, void*& pool, void*& scales, int& pages) {
    const at::Tensor* t = first(i);
    if (!t) return 0;
    const bool int8 = t->scalar_type() == ScalarType::Char;
    if ((!int8 && t->scalar_type() != ScalarType::Float8_e4m3fn) || t->dim() != 5 || t->size(1) != 2 ||
        t->size(2) != PKV_NUM_KV_HEADS || t->size(3) != PKV_PAGE_TOKENS || t->size(4) != PKV_HEAD_DIM ||
        !t->is_contiguous())
      return ok = false, 0;
    pool = t->data_ptr();
    pages = to_int(t->size(0));
    scales = vec(i + 1, ScalarType::Float, t->size(0) * 2 * PKV_NUM_KV_HEADS);
    return int8 ? PKV_BS8_INT8 : PKV_BS8_E4M3;
  }
  int64_t elements(int i) {
    if (!ok || !THPVariable_Check(at[i])) return ok = false, 0;
    return THPVariable_Unpack(at[i]).numel();
  }
  const int32_t* ints(void* p) const { return static_cast<const int32_t*>(p); }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
  std::nullptr_t fail() {
    ok = false;
    return nullptr;
  }
};

// q, k, v, positions, token_seq, block_tables, kv_pool, rope_cos, rope_sin, q_out, k_out, q_weight,
// k_weight, eps, interleaved, d_err, max_blocks
long norm_rope(Args& a) {
  enum { Q, K, V, POS, SEQ, BT, POOL, COS, SIN, QO, KO, QW, KW, EPS, INTER, ERR, MB };
  if (!a.first(K)) return kOther;
  int64_t T = -1;
  long long qs = 0, ks = 0, vs = 0;
  void* k = a.rows(K, PKV_NUM_KV_HEADS, T, ks);
  if (!a.ok || T < 1 || a.none(Q) != a.none(QO) || (a.none(Q) && !a.none(QW))) return kOther;
  void* q = a.none(Q) ? nullptr : a.rows(Q, PKV_NUM_Q_HEADS, T, qs);
  void* qo = a.opt(QO, ScalarType::BFloat16, T * kQRow);
  void* ko = a.opt(KO, ScalarType::BFloat16, T * kKvRow);
  void* pos = a.vec(POS, ScalarType::Int, T);
  void *v = nullptr, *bt = nullptr, *seq = nullptr, *pool = nullptr;
  int S = 0, width = 0, pages = 0;
  if (!a.none(POOL)) {
    const at::Tensor* t = a.tensor(POOL, ScalarType::BFloat16);
    if (!t || t->dim() != 5 || t->size(1) != 2 || t->size(2) != PKV_NUM_KV_HEADS || t->size(3) != PKV_PAGE_TOKENS ||
        t->size(4) != PKV_HEAD_DIM || !t->is_contiguous())
      return kOther;
    pool = t->data_ptr();
    pages = a.to_int(t->size(0));
    v = a.rows(V, PKV_NUM_KV_HEADS, T, vs);
    bt = a.tables(BT, 0, S, width);
    seq = a.opt(SEQ, ScalarType::Int, T);
  }
  const at::Tensor* cos = a.tensor(COS, ScalarType::Float);
  if (!cos || cos->dim() != 2 || !cos->is_contiguous()) return kOther;
  const int64_t max_pos = cos->size(0), pairs = cos->size(1);
  const at::Tensor* sin = a.tensor(SIN, ScalarType::Float);
  if (!sin || sin->dim() != 2 || sin->size(0) != max_pos || sin->size(1) != pairs || !sin->is_contiguous() || pairs < 1 ||
      pairs > PKV_ROPE_PAIRS)
    return kOther;
  void* w[2] = {nullptr, nullptr};
  int f32 = -1;
  for (int i = 0; i < 2; ++i) {
    if (a.none(QW + i)) continue;
    if (!THPVariable_Check(a.at[QW + i])) return kOther;
    const ScalarType type = THPVariable_Unpack(a.at[QW + i]).scalar_type();
    if (type != ScalarType::BFloat16 && type != ScalarType::Float) return kOther;
    const int is = type == ScalarType::Float;
    if (f32 >= 0 && f32 != is) return kOther;
    f32 = is;
    w[i] = a.vec(QW + i, type, PKV_HEAD_DIM);
  }
  const float eps = a.number(EPS);
  const int inter = PyObject_IsTrue(a.at[INTER]);
  void* err = a.error_word(ERR);
  const int mb = a.integer(MB, width), tokens = a.to_int(T), positions = a.to_int(max_pos);
  if (!a.ok || inter < 0) return kOther;
  return kv_append_norm_rope(q, qs, k, ks, v, vs, w[0], w[1], f32 == 1, eps, cos->data_ptr<float>(), sin->data_ptr<float>(),
                             positions, (int)pairs, inter, a.ints(pos), a.ints(seq), tokens, a.ints(bt), S, width, mb, pool,
                             pages, qo, ko, static_cast<int*>(err), a.stream());
}

// kv_pool, kv_scales, k, v, cu_new, seq_lens, block_tables, rope_cos, rope_sin, q_in, q_out, d_err, max_blocks
long append_bs8(Args& a) {
  enum { POOL, SCALES, K, V, CU, LENS, BT, COS, SIN, Q, QO, ERR, MB };
  void *pool = nullptr, *scales = nullptr;
  int pages = 0;
  const int code = a.bs8(POOL, pool, scales, pages);
  int64_t T = -1;
  long long qs = 0, ks = 0, vs = 0;
  void* k = a.rows(K, PKV_NUM_KV_HEADS, T, ks);
  void* v = a.rows(V, PKV_NUM_KV_HEADS, T, vs);
  const int64_t S = a.elements(LENS);
  if (!a.ok || T < 1 || S < 1 || a.none(COS) != a.none(SIN) || a.none(Q) != a.none(QO) || (!a.none(Q) && a.none(COS)))
    return kOther;
  void* lens = a.vec(LENS, ScalarType::Int, S);
  void* cu = a.vec(CU, ScalarType::Int, S + 1);
  int all = 0, width = 0;
  void* bt = a.tables(BT, S, all, width);
  int64_t max_pos = 0;
  void *cos = nullptr, *sin = nullptr, *q = nullptr, *qo = nullptr;
  if (!a.none(COS)) {
    const at::Tensor* t = a.tensor(COS, ScalarType::Float);
    if (!t || t->dim() != 2 || t->size(1) != PKV_ROPE_PAIRS) return kOther;
    max_pos = t->size(0);
    cos = a.vec(COS, ScalarType::Float, max_pos * PKV_ROPE_PAIRS);
    sin = a.vec(SIN, ScalarType::Float, max_pos * PKV_ROPE_PAIRS);
  }
  if (!a.none(Q)) {
    q = a.rows(Q, PKV_NUM_Q_HEADS, T, qs);
    qo = a.vec(QO, ScalarType::BFloat16, T * kQRow);
  }
  void* err = a.error_word(ERR);
  const int mb = a.integer(MB, width), tokens = a.to_int(T), seqs = a.to_int(S), positions = a.to_int(max_pos);
  if (!a.ok) return kOther;
  return kv_append_rope_bs8(k, ks, v, vs, a.ints(cu), a.ints(lens), tokens, a.ints(bt), seqs, width, mb, pool,
                            static_cast<float*>(scales), pages, code, static_cast<float*>(cos), static_cast<float*>(sin),
                            positions, q, qs, qo, static_cast<int*>(err), a.stream());
}

// kv_pool, kv_scales, page_ids, out, d_err
long read_bs8(Args& a) {
  void *pool = nullptr, *scales = nullptr;
  int pages = 0;
  const int code = a.bs8(0, pool, scales, pages);
  const int64_t n = a.elements(2);
  if (!a.ok || n < 1) return kOther;
  void* ids = a.vec(2, ScalarType::Int, n);
  void* out = a.vec(3, ScalarType::BFloat16, n * PKV_PAGE_ELEMS);
  void* err = a.error_word(4);
  const int count = a.to_int(n);
  if (!a.ok) return kOther;
  return kv_read_bs8(pool, static_cast<float*>(scales), pages, code, a.ints(ids), count, out, static_cast<int*>(err),
                     a.stream());
}

// kv_pool, kv_scales, q, block_tables, seq_lens, out, scale, workspace, max_seq_len, d_err, max_blocks
long decode_bs8(Args& a) {
  enum { POOL, SCALES, Q, BT, LENS, OUT, SCALE, WS, LONGEST, ERR, MB };
  void *pool = nullptr, *scales = nullptr;
  int pages = 0;
  const int code = a.bs8(POOL, pool, scales, pages);
  const at::Tensor* t = a.tensor(Q, ScalarType::BFloat16);
  if (!t || t->dim() < 2 || t->size(-1) != PKV_HEAD_DIM || t->size(-2) != PKV_NUM_Q_HEADS || t->numel() < 1) return kOther;
  const int64_t n = t->numel(), S = n / kQRow;
  void* q = a.vec(Q, ScalarType::BFloat16, n);
  void* out = a.vec(OUT, ScalarType::BFloat16, n);
  void* lens = a.vec(LENS, ScalarType::Int, S);
  int all = 0, width = 0;
  void* bt = a.tables(BT, S, all, width);
  const float scale = a.number(SCALE);
  const int64_t size = a.elements(WS);
  void* ws = a.vec(WS, ScalarType::Byte, size);
  void* err = a.error_word(ERR);
  const int mb = a.integer(MB, width), seqs = a.to_int(S);
  if (!a.ok || (a.none(LONGEST) && (mb < 0 || mb > INT_MAX / PKV_PAGE_TOKENS))) return kOther;
  const int longest = a.integer(LONGEST, PKV_PAGE_TOKENS * mb);
  if (!a.ok) return kOther;
  return paged_gqa_decode_bs8(q, pool, static_cast<float*>(scales), pages, code, a.ints(bt), width, mb, a.ints(lens), seqs,
                              longest, out, scale, ws, (size_t)size, static_cast<int*>(err), a.stream());
}

// logits, out, ids, history, history_lens, prompt_lens, repetition, presence, frequency, bias_ids, bias_values, allow_mask
long process_logits(Args& a) {
  enum { X, OUT, IDS, HIST, HLENS, PLENS, REP, PRES, FREQ, BIDS, BVALS, MASK };
  const at::Tensor* x = a.first(X);
  if (!x || x->dim() != 2) return kOther;
  const ScalarType type = x->scalar_type();
  const int dtype = type == ScalarType::Float ? PKV_LOGITS_F32 : type == ScalarType::BFloat16 ? PKV_LOGITS_BF16
                    : type == ScalarType::Half ? PKV_LOGITS_F16 : -1;
  const int64_t rows = x->size(0), vocab = x->size(1);
  if (dtype < 0 || rows < 1 || vocab < 2 || x->stride(1) != 1) return kOther;
  const long long stride = rows > 1 ? x->stride(0) : vocab;
  void *out = nullptr, *hist = nullptr, *hl = nullptr, *pl = nullptr, *rep = nullptr, *pres = nullptr, *freq = nullptr;
  void *bi = nullptr, *bv = nullptr, *mask = nullptr;
  long long out_stride = 0, mask_stride = 0;
  int64_t H = 0, B = 0;
  if (!a.none(OUT)) {
    const at::Tensor* t = a.tensor(OUT, ScalarType::Float);
    if (!t || t->dim() != 2 || t->size(0) != rows || t->size(1) != vocab || t->stride(1) != 1) return kOther;
    out = t->data_ptr();
    out_stride = rows > 1 ? t->stride(0) : vocab;
  }
  void* ids = a.vec(IDS, ScalarType::Int, rows);
  if (!a.none(HIST)) {
    const at::Tensor* t = a.tensor(HIST, ScalarType::Int);
    if (!t || t->dim() != 2 || t->size(0) != rows || t->size(1) < 1) return kOther;
    H = t->size(1);
    hist = a.vec(HIST, ScalarType::Int, rows * H);
    hl = a.vec(HLENS, ScalarType::Int, rows);
    pl = a.opt(PLENS, ScalarType::Int, rows);
    rep = a.opt(REP, ScalarType::Float, rows);
    pres = a.opt(PRES, ScalarType::Float, rows);
    freq = a.opt(FREQ, ScalarType::Float, rows);
  } else {
    for (int i = HLENS; i <= FREQ; ++i)
      if (!a.none(i)) return kOther;
  }
  if (a.none(BIDS) != a.none(BVALS)) return kOther;
  if (!a.none(BIDS)) {
    const at::Tensor *t = a.tensor(BIDS, ScalarType::Int), *u = a.tensor(BVALS, ScalarType::Float);
    if (!t || !u || t->dim() != 2 || t->size(0) != rows || u->dim() != 2 || u->size(0) != rows || u->size(1) != t->size(1))
      return kOther;
    B = t->size(1);
    bi = a.vec(BIDS, ScalarType::Int, rows * B);
    bv = a.vec(BVALS, ScalarType::Float, rows * B);
  }
  if (!a.none(MASK)) {
    const at::Tensor* t = a.tensor(MASK, ScalarType::Int);
    if (!t || t->dim() != 2 || t->size(0) != rows || t->size(1) < (vocab + 31) / 32) return kOther;
    mask_stride = t->size(1);
    mask = a.vec(MASK, ScalarType::Int, rows * mask_stride);
  }
  const int r = a.to_int(rows), v = a.to_int(vocab), b = a.to_int(B);
  if (!a.ok) return kOther;
  return pkv_process_logits(x->data_ptr(), dtype, r, v, stride, static_cast<float*>(out), out_stride,
                            static_cast<int32_t*>(ids), a.ints(hist), H, a.ints(hl), a.ints(pl), static_cast<float*>(rep),
                            static_cast<float*>(pres), static_cast<float*>(freq), a.ints(bi), static_cast<float*>(bv), b,
                            static_cast<const uint32_t*>(mask), mask_stride, a.stream());
}

template <long (*F)(Args&), int kArgs>
PyObject* entry(PyObject*, PyObject* const* at, Py_ssize_t n) {
  long st = kOther;
  if (n == kArgs) {
    try {
      Args a{at};
      st = F(a);
    } catch (...) {  // a tensor of a kind that has no such property: the Python checks say so
      st = kOther;
    }
    if (st < 0) PyErr_Clear();
  }
  return PyLong_FromLong(st);
}

PyMethodDef kMethods[] = {
    {"norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<norm_rope, 17>)), METH_FASTCALL, nullptr},
    {"append_bs8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<append_bs8, 13>)), METH_FASTCALL, nullptr},
    {"read_bs8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<read_bs8, 5>)), METH_FASTCALL, nullptr},
    {"decode_bs8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<decode_bs8, 11>)), METH_FASTCALL, nullptr},
    {"process_logits", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<process_logits, 12>)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", "Marshalling of the small calls (see calls.cpp).", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
