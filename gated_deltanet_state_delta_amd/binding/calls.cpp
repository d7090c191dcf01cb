// calls.cpp -- the short way from Python to the calls that a serving loop makes
// for every layer and token: attn_decode, kv_append, kv_read and rope.
//
// Such a call on one token a row runs for 3 to 6 us on the GPU; building its
// arguments in Python took 9 to 14 us.  Each function here takes the call's
// tensors as they come in the ordinary case -- on the current device, in the
// types and layouts that the kernels read in place -- checks them, fills the
// argument struct, allocates outputs and workspace through torch and calls
// libgdn.  For anything else, refusals of libgdn among it, it launches nothing and
// returns None, and the caller goes the general way in Python, which converts,
// copies or raises.  So no error text and no conversion is written twice.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/libgdn.h"

namespace {

typedef at::Tensor Tensor;

// libgdn's entry points, given by bind().
decltype(&gdn_attn_decode) g_attn;
decltype(&gdn_attn_decode_workspace_size) g_attn_workspace;
decltype(&gdn_kv_append) g_append;
decltype(&gdn_kv_read) g_read;
decltype(&gdn_rope) g_rope;

// Tensors of one call: all on the device of that index.
struct Args {
  PyObject* const* v;
  int64_t device;
  void* stream;

  // The tensor at i, or null for what is none or lies elsewhere.
  const Tensor* tensor(int i) const {
    if (!THPVariable_Check(v[i])) return nullptr;
    const Tensor& t = THPVariable_Unpack(v[i]);
    return t.is_cuda() && t.get_device() == device && t.layout() == at::kStrided ? &t : nullptr;
  }
  bool none(int i) const { return v[i] == Py_None; }
  // An optional tensor: false if it is neither None nor one of the call's.
  bool maybe(int i, const Tensor** t) const {
    *t = none(i) ? nullptr : tensor(i);
    return *t || none(i);
  }
};

int io_code(const Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? GDN_BF16 : t.scalar_type() == at::kFloat ? GDN_F32 : -1;
}
int cache_code(const Tensor& t) {
  return t.scalar_type() == at::kFloat8_e4m3fn ? GDN_E4M3 : t.scalar_type() == at::kChar ? GDN_I8 : io_code(t);
}
bool fits(int64_t n) { return n >= 0 && n <= INT32_MAX; }
bool aligned16(const Tensor& t) { return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0; }

// int32 values of one dimension, dense.
bool ints(const Tensor& t, int64_t n) {
  return t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == n && t.is_contiguous();
}

// Token and head strides of [B, T, h, d] or [tokens, h, d] whose tokens are one
// stride apart.
bool token_strides(const Tensor& t, int64_t* token, int64_t* head) {
  const int64_t n = t.dim(), h = t.size(n - 2), d = t.size(n - 1);
  if (t.is_contiguous()) {
    *token = h * d;
    *head = d;
    return true;
  }
  if (t.stride(n - 1) != 1) return false;
  if (n == 4) {
    if (t.size(1) != 1) return false;
    *token = t.size(0) > 1 ? t.stride(0) : h * d;
  } else {
    *token = t.size(0) > 1 ? t.stride(0) : h * d;
  }
  *head = h > 1 ? t.stride(n - 2) : d;
  return true;
}

// The fields that A, an argument struct, has for caches, page table, lengths and
// scales.  Strides go to ks, vs: {page, token, head}.
template <typename A>
bool cache_fields(A& a, const Tensor* kc, const Tensor* vc, const Tensor* table, const Tensor* lens, const Tensor* k_scale,
                  const Tensor* v_scale, int64_t rows, int64_t hkv, int64_t d, int64_t* ks, int64_t* vs) {
  if (!kc || !vc || !table || !lens || kc->dim() != 4 || vc->dim() != 4 || !vc->sizes().equals(kc->sizes()) ||
      vc->scalar_type() != kc->scalar_type())
    return false;
  const int64_t n = kc->size(0), page = kc->size(1);
  if (kc->size(2) != hkv || kc->size(3) != d || page < 1 || !fits(n) || !fits(page) || !fits(hkv) || !fits(d) || !fits(rows))
    return false;
  a.cache_dtype = cache_code(*kc);
  if (a.cache_dtype < 0 || (a.cache_dtype < GDN_E4M3 && a.cache_dtype != a.io_dtype)) return false;
  for (int i = 0; i < 2; ++i) {
    const Tensor& c = i ? *vc : *kc;
    int64_t* s = i ? vs : ks;
    if (c.stride(3) != 1) return false;
    // dimensions of one entry get their dense stride
    s[2] = hkv == 1 ? d : c.stride(2);
    s[1] = page == 1 ? d : c.stride(1);
    s[0] = n == 1 ? ((page - 1) * s[1] + (hkv - 1) * s[2] + d + 15) / 16 * 16 : c.stride(0);
  }
  if (table->scalar_type() != at::kInt || table->dim() != 2 || table->size(0) != rows) return false;
  const int64_t width = table->size(1), row = table->stride(0);
  if (!fits(width) || (table->stride(1) != 1 && width != 1) || (row < width && rows != 1) || !ints(*lens, rows)) return false;
  if ((k_scale != nullptr) != (v_scale != nullptr) || (k_scale != nullptr) != (a.cache_dtype >= GDN_E4M3)) return false;
  a.k_scale = a.v_scale = nullptr;
  a.k_block_scale = a.v_block_scale = nullptr;
  a.scale_block = 0;
  if (k_scale) {
    if (!v_scale->sizes().equals(k_scale->sizes()) || k_scale->scalar_type() != at::kFloat || v_scale->scalar_type() != at::kFloat ||
        !k_scale->is_contiguous() || !v_scale->is_contiguous())
      return false;
    float* k = static_cast<float*>(k_scale->data_ptr());
    float* v = static_cast<float*>(v_scale->data_ptr());
    if (k_scale->dim() == 3) {
      const int64_t blocks = k_scale->size(2);
      if (k_scale->size(0) != n || k_scale->size(1) != hkv || blocks < 1 || page % blocks != 0) return false;
      a.scale_block = static_cast<int32_t>(page / blocks);
      a.k_block_scale = k;
      a.v_block_scale = v;
    } else {
      if (k_scale->dim() != 1 || k_scale->size(0) != hkv || a.cache_dtype != GDN_E4M3) return false;
      a.k_scale = k;
      a.v_scale = v;
    }
  }
  a.k_cache = kc->data_ptr();
  a.v_cache = vc->data_ptr();
  a.n_pages = static_cast<int32_t>(n);
  a.page_size = static_cast<int32_t>(page);
  a.max_pages = static_cast<int32_t>(width);
  a.page_table = static_cast<const int32_t*>(table->data_ptr());
  a.page_table_stride = row > width ? row : width;
  a.lens = static_cast<const int32_t*>(lens->data_ptr());
  a.batch = static_cast<int32_t>(rows);
  a.hkv = static_cast<int32_t>(hkv);
  a.d = static_cast<int32_t>(d);
  return true;
}

Args args_of(PyObject* const* v, Py_ssize_t n) {  // the last two: device, stream
  return Args{v, PyLong_AsLongLong(v[n - 2]), PyLong_AsVoidPtr(v[n - 1])};
}

// Without the interpreter's lock, as ctypes and torch make such calls: an
// allocation may have to free memory and wait, a launch for room in its queue,
// and other threads go on meanwhile.  It costs nothing that shows: one token a
// row appended in 4.0 us, turned in 5.0, either way.  No Python object is touched
// inside; an exception takes the lock back.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

bool count_is(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", got, want);
  return got == want;
}

// attn_decode(q, k_cache, v_cache, page_table, lens, scale, k_scale, v_scale, device, stream) -> out
PyObject* attn_decode(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 10)) return nullptr;
  const Args in = args_of(v, n);
  const Tensor *q = in.tensor(0), *kc = in.tensor(1), *vc = in.tensor(2), *ks, *vs;
  if (!q || !kc || !in.maybe(6, &ks) || !in.maybe(7, &vs) || q->dim() != 4 || kc->dim() != 4 || !q->is_contiguous() || !aligned16(*q))
    Py_RETURN_NONE;
  gdn_attn_decode_args a = {};
  a.io_dtype = io_code(*q);
  const int64_t T = q->size(1), hq = q->size(2), d = q->size(3);
  int64_t k[3], w[3];
  if (a.io_dtype < 0 || !fits(T) || !fits(hq) ||
      !cache_fields(a, kc, vc, in.tensor(3), in.tensor(4), ks, vs, q->size(0), kc->size(2), d, k, w))
    Py_RETURN_NONE;
  a.T = static_cast<int32_t>(T);
  a.hq = static_cast<int32_t>(hq);
  const double scale = in.none(5) ? std::pow(static_cast<double>(d), -0.5) : PyFloat_AsDouble(v[5]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  a.scale = static_cast<float>(scale);
  a.q = q->data_ptr();
  a.q_stride_row = T * hq * d;
  a.q_stride_token = hq * d;
  a.q_stride_head = d;
  a.k_stride_page = k[0];
  a.k_stride_token = k[1];
  a.k_stride_head = k[2];
  a.v_stride_page = w[0];
  a.v_stride_token = w[1];
  a.v_stride_head = w[2];
  Tensor out;
  gdn_status status;
  {
    const Unlocked unlocked;
    Tensor space;
    out = at::empty(q->sizes(), q->options());
    a.out = out.data_ptr();
    const size_t need = g_attn_workspace(&a);
    if (need > 0) {
      space = at::empty({static_cast<int64_t>(need)}, q->options().dtype(at::kByte));
      a.workspace = space.data_ptr();
      a.workspace_bytes = need;
    }
    status = g_attn(&a, in.stream);
  }
  if (status != GDN_OK) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// The tokens of an append or a read: [B, T, h, d], or [tokens, h, d] with offsets.
bool token_count(const Tensor* cu, int64_t rows, int64_t dim, const Tensor& t, int64_t* total) {
  if (cu) {
    if (dim != 3 || !ints(*cu, rows + 1)) return false;
    *total = t.size(0);
  } else {
    if (dim != 4 || t.size(0) != rows) return false;
    *total = rows * t.size(1);
  }
  return true;
}

// kv_append(k, v, k_cache, v_cache, page_table, lens, cu_seqlens, k_scale, v_scale, device, stream) -> True
PyObject* kv_append(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 11)) return nullptr;
  const Args in = args_of(v, n);
  const Tensor *x = in.tensor(0), *y = in.tensor(1), *lens = in.tensor(5), *cu, *ks, *vs;
  if (!x || !y || !lens || !in.maybe(6, &cu) || !in.maybe(7, &ks) || !in.maybe(8, &vs) || lens->dim() != 1 ||
      !y->sizes().equals(x->sizes()) || y->scalar_type() != x->scalar_type())
    Py_RETURN_NONE;
  gdn_kv_append_args a = {};
  a.io_dtype = io_code(*x);
  const int64_t rows = lens->size(0), dim = x->dim();
  if (a.io_dtype < 0 || !token_count(cu, rows, dim, *x, &a.total_tokens) || !aligned16(*x) || !aligned16(*y) ||
      !token_strides(*x, &a.k_stride_token, &a.k_stride_head) || !token_strides(*y, &a.v_stride_token, &a.v_stride_head))
    Py_RETURN_NONE;
  const int64_t unit = a.io_dtype == GDN_BF16 ? 8 : 4;
  if ((a.k_stride_token | a.k_stride_head | a.v_stride_token | a.v_stride_head) % unit != 0) Py_RETURN_NONE;
  int64_t k[3], w[3];
  if (!cache_fields(a, in.tensor(2), in.tensor(3), in.tensor(4), lens, ks, vs, rows, x->size(dim - 2), x->size(dim - 1), k, w))
    Py_RETURN_NONE;
  a.k = x->data_ptr();
  a.v = y->data_ptr();
  a.cu_seqlens = cu ? static_cast<const int32_t*>(cu->data_ptr()) : nullptr;
  a.kc_stride_page = k[0];
  a.kc_stride_token = k[1];
  a.kc_stride_head = k[2];
  a.vc_stride_page = w[0];
  a.vc_stride_token = w[1];
  a.vc_stride_head = w[2];
  gdn_status status;
  {
    const Unlocked unlocked;
    status = g_append(&a, in.stream);
  }
  if (status != GDN_OK) Py_RETURN_NONE;
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// kv_read(k_cache, v_cache, page_table, lens, tokens, cu_seqlens, io code, k_scale, v_scale, device, stream) -> (k, v)
PyObject* kv_read(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 11)) return nullptr;
  const Args in = args_of(v, n);
  const Tensor *kc = in.tensor(0), *lens = in.tensor(3), *cu, *ks, *vs;
  if (!kc || !lens || !in.maybe(5, &cu) || !in.maybe(7, &ks) || !in.maybe(8, &vs) || kc->dim() != 4 || lens->dim() != 1 ||
      !PyLong_CheckExact(v[4]))
    Py_RETURN_NONE;
  gdn_kv_read_args a = {};
  a.io_dtype = static_cast<int32_t>(PyLong_AsLong(v[6]));
  const int64_t tokens = PyLong_AsLongLong(v[4]), rows = lens->size(0), hkv = kc->size(2), d = kc->size(3);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  int64_t k[3], w[3];
  if (!fits(tokens) || (cu && !ints(*cu, rows + 1)) ||
      !cache_fields(a, kc, in.tensor(1), in.tensor(2), lens, ks, vs, rows, hkv, d, k, w))
    Py_RETURN_NONE;
  a.total_tokens = cu ? tokens : rows * tokens;
  if (a.total_tokens > (int64_t(1) << 28) || rows == 0) Py_RETURN_NONE;  // before memory is taken for it; not launched
  const auto options = kc->options().dtype(a.io_dtype == GDN_BF16 ? at::kBFloat16 : at::kFloat);
  Tensor out[2];
  a.k_stride_token = a.v_stride_token = hkv * d;
  a.k_stride_head = a.v_stride_head = d;
  a.cu_seqlens = cu ? static_cast<const int32_t*>(cu->data_ptr()) : nullptr;
  a.zero_rest = 1;
  a.kc_stride_page = k[0];
  a.kc_stride_token = k[1];
  a.kc_stride_head = k[2];
  a.vc_stride_page = w[0];
  a.vc_stride_token = w[1];
  a.vc_stride_head = w[2];
  gdn_status status;
  {
    const Unlocked unlocked;
    for (Tensor& t : out) t = cu ? at::empty({tokens, hkv, d}, options) : at::empty({rows, tokens, hkv, d}, options);
    a.k = out[0].data_ptr();
    a.v = out[1].data_ptr();
    status = g_read(&a, in.stream);
  }
  if (status != GDN_OK) Py_RETURN_NONE;
  PyObject *first = THPVariable_Wrap(std::move(out[0])), *second = THPVariable_Wrap(std::move(out[1]));
  return Py_BuildValue("(NN)", first, second);
  END_HANDLE_TH_ERRORS
}

// rope(q, k, inv_freq, lens, cu_seqlens, positions, interleaved, factor, device, stream) -> (q, k)
PyObject* rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count_is(n, 10)) return nullptr;
  const Args in = args_of(v, n);
  const Tensor *q = in.tensor(0), *f = in.tensor(2), *k, *lens, *cu, *pos;
  if (!q || !f || !in.maybe(1, &k) || !in.maybe(3, &lens) || !in.maybe(4, &cu) || !in.maybe(5, &pos)) Py_RETURN_NONE;
  gdn_rope_args a = {};
  a.io_dtype = io_code(*q);
  const int64_t dim = q->dim();
  if (a.io_dtype < 0 || (dim != 3 && dim != 4) || f->dim() != 1 || f->scalar_type() != at::kDouble || !f->is_contiguous() ||
      (lens != nullptr) == (pos != nullptr) || (cu && !lens))
    Py_RETURN_NONE;
  const int64_t d = q->size(dim - 1), rot = 2 * f->size(0);
  if (rot < 2 || rot > d || !fits(d) || !fits(q->size(dim - 2)) || !token_strides(*q, &a.q_stride_token, &a.q_stride_head))
    Py_RETURN_NONE;
  const auto lead = q->sizes().slice(0, dim - 2);
  if (k && (k->dim() != dim || k->scalar_type() != q->scalar_type() || !k->sizes().slice(0, dim - 2).equals(lead) ||
            k->size(dim - 1) != d || !fits(k->size(dim - 2)) || !token_strides(*k, &a.k_stride_token, &a.k_stride_head)))
    Py_RETURN_NONE;
  a.total_tokens = dim == 4 ? lead[0] * lead[1] : lead[0];
  if (pos) {
    if (!pos->sizes().equals(lead) || !pos->is_contiguous() || (pos->scalar_type() != at::kInt && pos->scalar_type() != at::kLong))
      Py_RETURN_NONE;
    a.positions = pos->data_ptr();
    a.positions_i64 = pos->scalar_type() == at::kLong;
  } else {
    const int64_t rows = lens->dim() == 1 ? lens->size(0) : -1;
    if (rows < 1 || !fits(rows) || !ints(*lens, rows) || (cu ? dim != 3 || !ints(*cu, rows + 1) : dim != 4 || lead[0] != rows))
      Py_RETURN_NONE;
    a.batch = static_cast<int32_t>(rows);
    a.lens = static_cast<const int32_t*>(lens->data_ptr());
    a.cu_seqlens = cu ? static_cast<const int32_t*>(cu->data_ptr()) : nullptr;
  }
  const int interleaved = PyObject_IsTrue(v[6]);
  a.factor = static_cast<float>(PyFloat_AsDouble(v[7]));
  if (interleaved < 0 || PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  a.interleaved = interleaved;
  a.hq = static_cast<int32_t>(q->size(dim - 2));
  a.hkv = k ? static_cast<int32_t>(k->size(dim - 2)) : 0;
  a.d = static_cast<int32_t>(d);
  a.rot = static_cast<int32_t>(rot);
  a.inv_freq = static_cast<const double*>(f->data_ptr());
  a.q = q->data_ptr();
  a.qo_stride_token = a.hq * d;
  a.qo_stride_head = d;
  if (k) {
    a.k = k->data_ptr();
    a.ko_stride_token = a.hkv * d;
    a.ko_stride_head = d;
  }
  a.zero_rest = 1;
  Tensor qo, ko;
  gdn_status status;
  {
    const Unlocked unlocked;
    qo = at::empty(q->sizes(), q->options());
    a.q_out = qo.data_ptr();
    if (k) {
      ko = at::empty(k->sizes(), k->options());
      a.k_out = ko.data_ptr();
    }
    status = g_rope(&a, in.stream);
  }
  if (status != GDN_OK) Py_RETURN_NONE;
  PyObject* first = THPVariable_Wrap(std::move(qo));
  if (!k) return Py_BuildValue("(NO)", first, Py_None);
  PyObject* second = THPVariable_Wrap(std::move(ko));
  return Py_BuildValue("(NN)", first, second);
  END_HANDLE_TH_ERRORS
}

// bind(header_digest, attn_decode, attn_decode_workspace_size, kv_append, kv_read, rope): libgdn's entry
// points, as addresses.  The structs that they take are laid out by the header, so one of another header is refused.
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!count_is(n, 6)) return nullptr;
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(v[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no address");
      return nullptr;
    }
  }
  const char* digest = reinterpret_cast<decltype(&gdn_header_digest)>(p[0])();
  if (!digest || std::strcmp(digest, GDN_HEADER_DIGEST) != 0) {
    PyErr_SetString(PyExc_RuntimeError, "_calls.so and libgdn.so were built from different headers; build both again");
    return nullptr;
  }
  g_attn = reinterpret_cast<decltype(g_attn)>(p[1]);
  g_attn_workspace = reinterpret_cast<decltype(g_attn_workspace)>(p[2]);
  g_append = reinterpret_cast<decltype(g_append)>(p[3]);
  g_read = reinterpret_cast<decltype(g_read)>(p[4]);
  g_rope = reinterpret_cast<decltype(g_rope)>(p[5]);
  Py_RETURN_NONE;
}

#define GDN_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDN_METHOD(attn_decode), GDN_METHOD(kv_append), GDN_METHOD(kv_read), GDN_METHOD(rope), GDN_METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
