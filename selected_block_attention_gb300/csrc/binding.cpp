// Python entry points of the paged-cache calls, the rotary calls and the block-sparse gradients
// (module _paged): tensors in, argument checks, outputs allocated, one call of the C ABI.
//
// A decode step makes the paged calls once per layer on batches whose kernels take a few
// microseconds, so the host's share counts: reading a dozen tensors' properties, packing
// and allocating from Python took 17 to 25 us a call, from here 5 to 9; likewise the others on
// short rows.  The other entry points'
// kernels run long enough for their ctypes binding.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../include/sba.h"

namespace {

struct Error {
  PyObject* type;
  std::string text;
};
[[noreturn]] void value_error(const std::string& text) { throw Error{PyExc_ValueError, text}; }
[[noreturn]] void type_error(const std::string& text) { throw Error{PyExc_TypeError, text}; }
struct Raised {};  // a Python error is set already

PyObject* g_error = nullptr;  // SBAError

// ------------------------------------------------------------------ arguments
// Names in order; the first `required` must be given, those from `positional` on only by
// keyword.
struct Signature {
  const char* function;
  std::initializer_list<const char*> list;
  int required, positional;
  PyObject* names[32];
  int n = 0;
  Signature(const char* f, int req, int pos, std::initializer_list<const char*> l)
      : function(f), list(l), required(req), positional(pos) {
    for (const char* s : l) names[n++] = PyUnicode_InternFromString(s);
  }
  void read(PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames, PyObject** out) const {
    for (int i = 0; i < n; ++i) out[i] = nullptr;
    if (nargs > positional)
      type_error(std::string(function) + "() takes at most " + std::to_string(positional) + " positional arguments");
    for (Py_ssize_t i = 0; i < nargs; ++i) out[i] = args[i];
    const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t k = 0; k < nk; ++k) {
      PyObject* name = PyTuple_GET_ITEM(kwnames, k);
      int at = -1;
      for (int i = 0; i < n && at < 0; ++i)
        if (names[i] == name) at = i;
      for (int i = 0; i < n && at < 0; ++i)
        if (PyUnicode_Compare(names[i], name) == 0) at = i;
      if (at < 0 || out[at] != nullptr) {
        const char* s = PyUnicode_AsUTF8(name);
        type_error(std::string(function) + "() got " + (at < 0 ? "an unexpected" : "a second") + " argument '" +
                   (s ? s : "?") + "'");
      }
      out[at] = args[nargs + k];
    }
    for (int i = 0; i < required; ++i)
      if (out[i] == nullptr)
        type_error(std::string(function) + "() misses the argument '" + PyUnicode_AsUTF8(names[i]) + "'");
    for (int i = required; i < n; ++i)
      if (out[i] == Py_None) out[i] = nullptr;
  }
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor* optional(PyObject* o, const char* name) { return o ? &tensor(o, name) : nullptr; }
double real(PyObject* o, double absent) {
  if (!o) return absent;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
int whole(PyObject* o, int absent) {
  if (!o) return absent;
  PyObject* i = PyNumber_Index(o);
  if (!i) throw Raised{};
  const long long v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v > INT32_MAX || v < INT32_MIN) value_error("an integer argument is out of range");
  return static_cast<int>(v);
}
bool truth(PyObject* o, bool absent) {
  if (!o) return absent;
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}
int size32(int64_t v, const char* name) {
  if (v > INT32_MAX) value_error(std::string(name) + " is too large");
  return static_cast<int>(v);
}

// Address of a contiguous CUDA tensor on device `index`; null for an absent one.
void* at_of(const at::Tensor* t, const char* name, int index, at::ScalarType type, at::IntArrayRef shape,
            const char* whose = "the cache's") {
  if (!t) return nullptr;
  if (t->scalar_type() != type) type_error(std::string(name) + " must be " + c10::toString(type));
  if (!t->is_cuda() || t->get_device() != index || t->sizes() != shape || !t->is_contiguous()) {
    std::string s;
    for (int64_t d : shape) s += (s.empty() ? "" : ", ") + std::to_string(d);
    value_error(std::string(name) + " must be a contiguous tensor of shape [" + s + "] on " + whose + " device");
  }
  return t->data_ptr();
}

struct Cache {
  sba_paged_cache c;
  int index;
};
// Objects in the order k_pages, v_pages, page_table, seq_lens, k_scales, v_scales, cu_seqlens.
Cache cache_of(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo, PyObject* kso, PyObject* vso, PyObject* cuo) {
  const at::Tensor &k = tensor(ko, "k_pages"), &v = tensor(vo, "v_pages");
  const at::Tensor &table = tensor(to, "page_table"), &lens = tensor(lo, "seq_lens");
  if (!k.is_cuda() || !v.is_cuda()) value_error("libsba works on CUDA tensors only (no CPU path)");
  Cache r{};
  r.index = static_cast<int>(k.get_device());
  const auto type = k.scalar_type();
  if ((type != at::kFloat8_e4m3fn && type != at::kBFloat16) || v.scalar_type() != type)
    type_error("k_pages and v_pages must both be float8_e4m3fn or both bfloat16");
  if (k.dim() != 4 || v.sizes() != k.sizes() || v.get_device() != r.index)
    value_error("k_pages and v_pages must be [num_pages, Hkv, page_size, D] on one device");
  const int64_t pages = k.size(0), heads = k.size(1), size = k.size(2), d = k.size(3);
  for (const at::Tensor* t : {&k, &v}) {
    const auto st = t->strides();
    if (st[3] != 1 || st[2] != d || (st[1] != size * d && heads > 1) || (st[0] != k.stride(0) && pages > 1))
      value_error("k_pages, v_pages: pages must be dense and lie as far apart in both pools");
  }
  if (table.dim() != 2) value_error("page_table must be [B, width]");
  const int64_t batch = table.size(0);
  const int64_t scales[2] = {pages, heads}, rows[1] = {batch}, offsets[1] = {batch + 1};
  sba_paged_cache& c = r.c;
  c.k_pages = k.data_ptr();
  c.v_pages = v.data_ptr();
  c.k_scales = static_cast<float*>(at_of(optional(kso, "k_scales"), "k_scales", r.index, at::kFloat, scales));
  c.v_scales = static_cast<float*>(at_of(optional(vso, "v_scales"), "v_scales", r.index, at::kFloat, scales));
  c.page_table = static_cast<int32_t*>(at_of(&table, "page_table", r.index, at::kInt, table.sizes()));
  c.seq_lens = static_cast<int32_t*>(at_of(&lens, "seq_lens", r.index, at::kInt, rows));
  c.cu_seqlens = static_cast<int32_t*>(at_of(optional(cuo, "cu_seqlens"), "cu_seqlens", r.index, at::kInt, offsets));
  c.page_stride = pages > 1 ? k.stride(0) : heads * size * d;
  c.num_pages = size32(pages, "num_pages");
  c.page_size = size32(size, "page_size");
  c.Hkv = size32(heads, "Hkv");
  c.D = size32(d, "D");
  c.dtype = type == at::kBFloat16 ? SBA_BF16 : SBA_E4M3;
  c.table_width = size32(table.size(1), "page_table");
  c.B = size32(batch, "page_table");
  return r;
}

// bf16 token rows: [N, H, D] with cu_seqlens, else [B, H, D] (one token per row) or
// [B, Q, H, D].  Heads are dense inside a token, tokens equally far apart.
struct Tokens {
  void* at;
  int q, n, heads;
  long long stride;
};
Tokens tokens_of(const at::Tensor& t, const char* name, const Cache& c) {
  if (t.scalar_type() != at::kBFloat16) type_error(std::string(name) + " must be bfloat16");
  const bool packed = c.c.cu_seqlens != nullptr;
  const int64_t dim = t.dim();
  if (dim != 3 && (dim != 4 || packed))
    value_error(std::string(name) + " must be [B, H, D] or [B, Q, H, D], or [N, H, D] with cu_seqlens");
  const auto sz = t.sizes(), st = t.strides();
  const int64_t heads = sz[dim - 2], d = sz[dim - 1];
  if (!t.is_cuda() || t.get_device() != c.index || d != c.c.D || st[dim - 1] != 1 || (st[dim - 2] != d && heads > 1))
    value_error(std::string(name) + " must be on the cache's device, with its head dimension and dense heads");
  if (!packed && sz[0] != c.c.B) value_error(std::string(name) + " must have one entry per row of page_table");
  const int64_t q = dim == 4 ? sz[1] : 1, n = sz[0] * q;
  const int64_t stride = dim == 4 && q > 1 ? st[1] : st[0];
  if (dim == 4 && q > 1 && sz[0] > 1 && st[0] != q * stride)
    value_error(std::string(name) + ": tokens must lie equally far apart");
  return {t.data_ptr(), size32(q, name), size32(n, name), size32(heads, name), n > 1 ? stride : heads * d};
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int index) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)), std::nullopt);
}

// A given tensor has new values: autograd must not use the old ones that it may have saved.
void written(PyObject* given) {
  if (!given) return;
  const at::Tensor& t = THPVariable_Unpack(given);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// `fn(stream)` with the tensors' device current: the library launches on it and looks up its state
// there.
template <class Fn>
void call_on(int index, Fn fn) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  const int code = fn(reinterpret_cast<sba_stream_t>(c10::cuda::getCurrentCUDAStream(index).stream()));
  if (code == SBA_OK) return;
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", code, sba_last_error()) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, sba_last_error());
  }
  throw Raised{};
}

template <class Args>
void call(int (*fn)(const Args*, sba_stream_t), const Args& a, int index) {
  call_on(index, [&](sba_stream_t stream) { return fn(&a, stream); });
}

template <class Body>
PyObject* guarded(Body body) {
  try {
    return body();
  } catch (const Raised&) {
  } catch (const Error& e) {
    PyErr_SetString(e.type, e.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// out and lse of a call on queries q: given ones checked, absent ones made.
struct Results {
  at::Tensor out, lse;
  void* out_p;
  float* lse_p;
  PyObject* wrap() const {
    PyObject* a = THPVariable_Wrap(out);
    PyObject* b = a ? (lse.defined() ? THPVariable_Wrap(lse) : Py_NewRef(Py_None)) : nullptr;
    PyObject* t = b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    if (!t) throw Raised{};
    return t;
  }
};
Results results(const at::Tensor& q, PyObject* out, PyObject* lse, bool return_lse, int index) {
  Results r;
  const auto rows = q.sizes().slice(0, q.dim() - 1);
  r.out = out ? tensor(out, "out") : fresh(q.sizes(), at::kBFloat16, index);
  if (lse) r.lse = tensor(lse, "lse");
  else if (return_lse) r.lse = fresh(rows, at::kFloat, index);
  r.out_p = at_of(&r.out, "out", index, at::kBFloat16, q.sizes());
  r.lse_p = r.lse.defined() ? static_cast<float*>(at_of(&r.lse, "lse", index, at::kFloat, rows)) : nullptr;
  return r;
}

// ------------------------------------------------------------------ entry points
const char kAppendDoc[] =
    "paged_kv_append(k, v, k_pages, v_pages, page_table, seq_lens, *, k_scales=None, v_scales=None, "
    "cu_seqlens=None, q=None, cos=None, sin=None, interleaved=False, q_out=None)\n--\n\n"
    "Write the rows' last tokens into a paged cache.  k / v bf16 [B, Hkv, D] (one token per\n"
    "row), [B, Q, Hkv, D], or [N, Hkv, D] with cu_seqlens int32 [B + 1]; token strides may be\n"
    "those of a slice.  k_pages / v_pages [num_pages, Hkv, page_size, D] float8_e4m3fn (with\n"
    "fp32 scales [num_pages, Hkv]) or bfloat16, page_table int32 [B, width], seq_lens int32\n"
    "[B] with the new tokens counted.  cos / sin fp32 [max_pos, rot_dim / 2] turn keys (and\n"
    "q, [..., Hq, D]) by their positions.  Returns q_out (new unless given; may be q), or\n"
    "None without q.";
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  static const Signature sig("paged_kv_append", 6, 6,
                             {"k", "v", "k_pages", "v_pages", "page_table", "seq_lens", "k_scales", "v_scales",
                              "cu_seqlens", "q", "cos", "sin", "interleaved", "q_out"});
  return guarded([&]() -> PyObject* {
    PyObject* o[32];
    sig.read(args, nargs, kwnames, o);
    const Cache c = cache_of(o[2], o[3], o[4], o[5], o[6], o[7], o[8]);
    sba_paged_append_args a{};
    a.cache = c.c;
    const Tokens k = tokens_of(tensor(o[0], "k"), "k", c), v = tokens_of(tensor(o[1], "v"), "v", c);
    if (k.heads != c.c.Hkv || v.heads != c.c.Hkv || v.q != k.q || v.n != k.n)
      value_error("k and v must have the same tokens and the cache's heads");
    a.cache.Q = k.q;
    a.cache.N = k.n;
    a.k = k.at;
    a.v = v.at;
    a.k_stride = k.stride;
    a.v_stride = v.stride;
    at::Tensor q_out;
    if (o[9]) {
      const at::Tensor& qt = tensor(o[9], "q");
      const Tokens q = tokens_of(qt, "q", c);
      if (q.q != k.q || q.n != k.n) value_error("q must have k's tokens");
      q_out = o[13] ? tensor(o[13], "q_out") : fresh(qt.sizes(), at::kBFloat16, c.index);
      const Tokens to = tokens_of(q_out, "q_out", c);
      if (to.q != q.q || to.n != q.n || to.heads != q.heads) value_error("q_out must have q's shape");
      a.q = q.at;
      a.q_out = to.at;
      a.q_stride = q.stride;
      a.q_out_stride = to.stride;
      a.Hq = q.heads;
    } else if (o[13]) {
      value_error("q_out needs q");
    }
    if (o[10] || o[11]) {
      if (!o[10] || !o[11] || tensor(o[10], "cos").dim() != 2)
        value_error("cos and sin go together, [max_pos, rot_dim / 2]");
      const at::Tensor &cos = tensor(o[10], "cos"), &sin = tensor(o[11], "sin");
      a.cos = static_cast<float*>(at_of(&cos, "cos", c.index, at::kFloat, cos.sizes()));
      a.sin = static_cast<float*>(at_of(&sin, "sin", c.index, at::kFloat, cos.sizes()));
      a.max_pos = size32(cos.size(0), "cos");
      a.rot_dim = size32(2 * cos.size(1), "cos");
    }
    a.interleaved = truth(o[12], false);
    call(sba_paged_kv_append, a, c.index);
    if (!q_out.defined()) Py_RETURN_NONE;
    if (o[13]) return Py_NewRef(o[13]);
    return THPVariable_Wrap(q_out);
  });
}

const char kAttentionDoc[] =
    "paged_attention_fwd(q, k_pages, v_pages, page_table, seq_lens, *, k_scales=None, v_scales=None, "
    "cu_seqlens=None, softmax_scale=None, window_left=-1, window_right=-1, logits_soft_cap=None, "
    "sink_bias=None, out=None, lse=None, workspace=None, return_lse=True)\n--\n\n"
    "Attention of the rows' last tokens over a paged cache (as paged_kv_append fills it).\n"
    "q bf16 [B, Hq, D], [B, Q, Hq, D], or [N, Hq, D] with cu_seqlens; windows, soft cap and\n"
    "sink_bias as in ragged_flash_attention_fwd (window_right=0 is causal).  Returns\n"
    "(out, lse) in q's shape and [..., Hq].";
PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  static const Signature sig("paged_attention_fwd", 5, 5,
                             {"q", "k_pages", "v_pages", "page_table", "seq_lens", "k_scales", "v_scales",
                              "cu_seqlens", "softmax_scale", "window_left", "window_right", "logits_soft_cap",
                              "sink_bias", "out", "lse", "workspace", "return_lse"});
  return guarded([&]() -> PyObject* {
    PyObject* o[32];
    sig.read(args, nargs, kwnames, o);
    const Cache c = cache_of(o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
    sba_paged_attention_args a{};
    a.cache = c.c;
    const at::Tensor& qt = tensor(o[0], "q");
    const Tokens q = tokens_of(qt, "q", c);
    a.cache.Q = q.q;
    a.cache.N = q.n;
    a.q = q.at;
    a.q_stride = q.stride;
    a.Hq = q.heads;
    a.softmax_scale = static_cast<float>(real(o[8], 0.0));
    a.window_left = whole(o[9], -1);
    a.window_right = whole(o[10], -1);
    a.logits_soft_cap = static_cast<float>(real(o[11], 0.0));
    if (o[12]) {
      const at::Tensor& b = tensor(o[12], "sink_bias");
      a.sink_bias_per_head = b.dim() == 2;
      if (b.dim() != 1 && (b.dim() != 2 || b.size(0) != q.heads))
        value_error("sink_bias must be [Hq, num_sinks] or [num_sinks]");
      a.num_sinks = size32(b.size(-1), "sink_bias");
      a.sink_bias = static_cast<float*>(at_of(&b, "sink_bias", c.index, at::kFloat, b.sizes()));
      if (a.num_sinks == 0) a.sink_bias = nullptr;
    }
    const Results r = results(qt, o[13], o[14], truth(o[16], true), c.index);
    a.out = r.out_p;
    a.lse = r.lse_p;
    at::Tensor ws;
    if (o[15]) {
      ws = tensor(o[15], "workspace");
      if (!ws.is_cuda() || ws.get_device() != c.index || !ws.is_contiguous())
        value_error("workspace must be a contiguous tensor on the cache's device");
    } else {
      const size_t need = sba_paged_attention_workspace_size(c.c.B, q.n, q.heads, c.c.Hkv, c.c.D);
      ws = fresh({static_cast<int64_t>(need ? need : 16)}, at::kByte, c.index);
    }
    a.workspace = ws.data_ptr();
    a.workspace_bytes = ws.nbytes();
    call(sba_paged_attention_fwd, a, c.index);
    return r.wrap();
  });
}

const char kSelectDoc[] =
    "nsa_select_paged_fwd(q, k_pages, v_pages, page_table, seq_lens, block_indices, block_counts, "
    "block_size, *, k_scales=None, v_scales=None, causal=True, softmax_scale=None, g_slc=None, "
    "out=None, lse=None, return_lse=True)\n--\n\n"
    "Selection-branch NSA of the rows' last tokens over a paged cache: the decode form of\n"
    "nsa_select_fwd.  q bf16 [B, Hq, D] or [B, Q, Hq, D], block_indices int32\n"
    "[B, (Q,) Hkv, S], block_counts int or int32 [B, (Q,) Hkv], g_slc bf16 [B, (Q,) Hq] or\n"
    "None.  Returns (out, lse).";
PyObject* select(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  static const Signature sig("nsa_select_paged_fwd", 8, 8,
                             {"q", "k_pages", "v_pages", "page_table", "seq_lens", "block_indices", "block_counts",
                              "block_size", "k_scales", "v_scales", "causal", "softmax_scale", "g_slc", "out", "lse",
                              "return_lse"});
  return guarded([&]() -> PyObject* {
    PyObject* o[32];
    sig.read(args, nargs, kwnames, o);
    const Cache c = cache_of(o[1], o[2], o[3], o[4], o[8], o[9], nullptr);
    sba_nsa_select_paged_args a{};
    a.cache = c.c;
    const at::Tensor& qt = tensor(o[0], "q");
    const Tokens q = tokens_of(qt, "q", c);
    a.cache.Q = q.q;
    a.cache.N = q.n;
    a.q = q.at;
    a.q_stride = q.stride;
    a.Hq = q.heads;
    const at::Tensor& idx = tensor(o[5], "block_indices");
    if (idx.dim() < 1) value_error("block_indices must be [B, (Q,) Hkv, S]");
    a.S = size32(idx.size(-1), "block_indices");
    at::DimVector lead(qt.sizes().begin(), qt.sizes().end() - 2);
    lead.push_back(c.c.Hkv);
    if (THPVariable_Check(o[6])) {
      const at::Tensor& n = THPVariable_Unpack(o[6]);
      a.block_counts = static_cast<int32_t*>(at_of(&n, "block_counts", c.index, at::kInt, lead));
    } else {
      a.block_count_scalar = whole(o[6], 0);
    }
    lead.push_back(a.S);
    a.block_indices = static_cast<int32_t*>(at_of(&idx, "block_indices", c.index, at::kInt, lead));
    a.block_size = whole(o[7], 0);
    a.causal = truth(o[10], true);
    a.softmax_scale = static_cast<float>(real(o[11], 0.0));
    a.g_slc = at_of(optional(o[12], "g_slc"), "g_slc", c.index, at::kBFloat16, qt.sizes().slice(0, qt.dim() - 1));
    const Results r = results(qt, o[13], o[14], truth(o[15], true), c.index);
    a.out = r.out_p;
    a.lse = r.lse_p;
    call(sba_nsa_select_paged_fwd, a, c.index);
    return r.wrap();
  });
}

const char kGradDoc[] =
    "blocksparse_attn_bwd(q, k, v, out, lse, d_out, q_positions, q_segment_ids, kv_positions, "
    "kv_segment_ids, lower, upper, lower_full, upper_full, q_blocksize, kv_blocksize, *, causal=True, "
    "window_left=-1, window_right=-1, padding_segment_id=-1, softmax_scale=None, dq=None, dk=None, dv=None, "
    "workspace=None)\n--\n\n"
    "Gradients (dq, dk, dv) of blocksparse_attn_fwd (bf16): out and lse are the forward's\n"
    "results for the same arguments and bounds, d_out the gradient of the loss with respect\n"
    "to out.  No autograd graph is built; given outputs count as changed for graphs that saved them.";
PyObject* grad(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  static const Signature sig("blocksparse_attn_bwd", 16, 16,
                             {"q", "k", "v", "out", "lse", "d_out", "q_positions", "q_segment_ids", "kv_positions",
                              "kv_segment_ids", "lower", "upper", "lower_full", "upper_full", "q_blocksize",
                              "kv_blocksize", "causal", "window_left", "window_right", "padding_segment_id",
                              "softmax_scale", "dq", "dk", "dv", "workspace"});
  return guarded([&]() -> PyObject* {
    PyObject* o[32];
    sig.read(args, nargs, kwnames, o);
    const at::Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k");
    if (!q.is_cuda()) value_error("libsba works on CUDA tensors only (no CPU path)");
    if (q.dim() != 4 || k.dim() != 4) value_error("q must be [B, T, Hq, D], k and v [B, T, Hkv, D]");
    const int index = static_cast<int>(q.get_device());
    const int64_t B = q.size(0), T = q.size(1), Hq = q.size(2), Hkv = k.size(2), D = q.size(3);
    const int q_block = whole(o[14], 0), kv_block = whole(o[15], 0);
    const int64_t qs[4] = {B, T, Hq, D}, ks[4] = {B, T, Hkv, D}, rows[3] = {B, T, Hq}, ts[2] = {B, T};
    const int64_t bounds[3] = {B, 1, q_block > 0 ? (T + q_block - 1) / q_block : 0};
    auto at = [&](int i, const char* name, at::ScalarType type, at::IntArrayRef shape) {
      return at_of(&tensor(o[i], name), name, index, type, shape, "q's");
    };
    const void* in[6] = {at(0, "q", at::kBFloat16, qs),     at(1, "k", at::kBFloat16, ks),
                         at(2, "v", at::kBFloat16, ks),     at(3, "out", at::kBFloat16, qs),
                         at(4, "lse", at::kFloat, rows),    at(5, "d_out", at::kBFloat16, qs)};
    static const char* const kInts[8] = {"q_positions", "q_segment_ids", "kv_positions", "kv_segment_ids",
                                         "lower",       "upper",         "lower_full",   "upper_full"};
    const int32_t* ints[8];
    for (int i = 0; i < 8; ++i)
      ints[i] = static_cast<const int32_t*>(at(6 + i, kInts[i], at::kInt, i < 4 ? at::IntArrayRef(ts) : at::IntArrayRef(bounds)));
    static const char* const kMade[3] = {"dq", "dk", "dv"};
    at::Tensor made[3];
    void* to[3];
    for (int i = 0; i < 3; ++i) {
      const at::IntArrayRef shape = i == 0 ? at::IntArrayRef(qs) : at::IntArrayRef(ks);
      made[i] = o[21 + i] ? tensor(o[21 + i], kMade[i]) : fresh(shape, at::kBFloat16, index);
      to[i] = at_of(&made[i], kMade[i], index, at::kBFloat16, shape, "q's");
    }
    const int b = size32(B, "B"), t = size32(T, "T"), hq = size32(Hq, "Hq");
    at::Tensor ws;
    if (o[24]) {
      ws = tensor(o[24], "workspace");
      if (!ws.is_cuda() || ws.get_device() != index || !ws.is_contiguous())
        value_error("workspace must be a contiguous tensor on q's device");
    } else {
      const size_t need = sba_blocksparse_attn_bwd_workspace_size(b, t, hq, size32(Hkv, "Hkv"), size32(D, "D"));
      ws = fresh({static_cast<int64_t>(need ? need : 256)}, at::kByte, index);
    }
    const int causal = truth(o[16], true), left = whole(o[17], -1), right = whole(o[18], -1), pad = whole(o[19], -1);
    const float scale = static_cast<float>(real(o[20], 0.0));
    call_on(index, [&](sba_stream_t stream) {
      return sba_blocksparse_attn_bwd(in[0], in[1], in[2], in[3], static_cast<const float*>(in[4]), in[5], ints[0], ints[1],
                                      ints[2], ints[3], ints[4], ints[5], ints[6], ints[7], b, t, hq, size32(Hkv, "Hkv"),
                                      size32(D, "D"), q_block, kv_block, causal, left, right, pad, scale, to[0], to[1],
                                      to[2], ws.data_ptr(), ws.nbytes(), stream);
    });
    for (int i = 0; i < 3; ++i) written(o[21 + i]);
    PyObject* r = PyTuple_New(3);
    if (!r) throw Raised{};
    for (int i = 0; i < 3; ++i) {
      PyObject* x = o[21 + i] ? Py_NewRef(o[21 + i]) : THPVariable_Wrap(made[i]);
      if (!x) {
        Py_DECREF(r);
        throw Raised{};
      }
      PyTuple_SET_ITEM(r, i, x);
    }
    return r;
  });
}

const char kTablesDoc[] =
    "rotary_tables(length, rot_dim, *, base=10000.0, factor=1.0, original_length=0, slow=1.0, fast=32.0, "
    "amplitude=1.0, device=None, cos=None, sin=None)\n--\n\n"
    "Tables (cos, sin), fp32 [length, rot_dim / 2], of positions 0 .. length - 1, as rotary_embed\n"
    "and paged_kv_append take them.  Pair i turns by base ** (-2 i / rot_dim) radians a position;\n"
    "factor > 1 stretches them for longer contexts: all of them, or with original_length those that\n"
    "make fewer than `fast` turns over it (wholly below `slow` turns).  amplitude multiplies both.";
PyObject* tables(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  static const Signature sig("rotary_tables", 2, 2,
                             {"length", "rot_dim", "base", "factor", "original_length", "slow", "fast", "amplitude",
                              "device", "cos", "sin"});
  return guarded([&]() -> PyObject* {
    PyObject* o[32];
    sig.read(args, nargs, kwnames, o);
    const int length = whole(o[0], 0), rot = whole(o[1], 0);
    const double base = real(o[2], 10000.0), factor = real(o[3], 1.0), slow = real(o[5], 1.0), fast = real(o[6], 32.0);
    const double amplitude = real(o[7], 1.0);
    const int original = whole(o[4], 0);
    if (length < 0 || rot < 0) value_error("length and rot_dim must not be negative");
    if (!o[9] != !o[10]) value_error("cos and sin go together");
    const int64_t shape[2] = {length, rot / 2};
    at::Tensor made[2];
    void* to[2];
    int index;
    if (o[9]) {
      made[0] = tensor(o[9], "cos");
      made[1] = tensor(o[10], "sin");
      if (!made[0].is_cuda()) value_error("libsba works on CUDA tensors only (no CPU path)");
      index = static_cast<int>(made[0].get_device());
    } else {
      c10::Device device(at::kCUDA);
      if (o[8]) {
        if (THPDevice_Check(o[8])) {
          device = reinterpret_cast<THPDevice*>(o[8])->device;
        } else if (PyUnicode_Check(o[8])) {
          const char* text = PyUnicode_AsUTF8(o[8]);
          if (!text) throw Raised{};
          device = c10::Device(std::string(text));
        } else {
          type_error("device must be a torch.device or a text");
        }
      }
      if (!device.is_cuda()) value_error("libsba works on CUDA tensors only (no CPU path)");
      index = device.has_index() ? device.index() : c10::cuda::current_device();
      for (at::Tensor& t : made) t = fresh(shape, at::kFloat, index);
    }
    to[0] = at_of(&made[0], "cos", index, at::kFloat, shape, "cos's");
    to[1] = at_of(&made[1], "sin", index, at::kFloat, shape, "cos's");
    call_on(index, [&](sba_stream_t stream) {
      return sba_rotary_tables(length, rot, base, factor, original, slow, fast, amplitude, static_cast<float*>(to[0]),
                               static_cast<float*>(to[1]), stream);
    });
    written(o[9]);
    written(o[10]);
    PyObject* a = o[9] ? Py_NewRef(o[9]) : THPVariable_Wrap(made[0]);
    PyObject* b = a ? (o[10] ? Py_NewRef(o[10]) : THPVariable_Wrap(made[1])) : nullptr;
    PyObject* r = b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    if (!r) throw Raised{};
    return r;
  });
}

// Token rows [B, T, H, D] or [N, H, D], heads dense inside a token, tokens equally far apart.
struct Rows {
  void* at;
  int64_t B, T, heads, d;
  long long stride;
};
Rows rows_of(const at::Tensor& t, const char* name, const at::Tensor& like) {
  const int64_t dim = t.dim();
  if (t.scalar_type() != like.scalar_type()) type_error(std::string(name) + " must have q's dtype");
  if (dim != like.dim()) value_error(std::string(name) + " must have q's leading dimensions");
  const auto sz = t.sizes(), st = t.strides();
  for (int64_t i = 0; i < dim - 2; ++i)
    if (sz[i] != like.size(i)) value_error(std::string(name) + " must have q's leading dimensions");
  const int64_t heads = sz[dim - 2], d = sz[dim - 1];
  if (!t.is_cuda() || t.get_device() != like.get_device() || d != like.size(dim - 1) || (st[dim - 1] != 1 && d > 1) ||
      (st[dim - 2] != d && heads > 1))
    value_error(std::string(name) + " must be on q's device, with its head dimension and dense heads");
  const int64_t B = dim == 4 ? sz[0] : 1, T = sz[dim - 3], n = B * T;
  const int64_t stride = dim == 4 && T == 1 ? st[0] : st[dim - 3];
  if (dim == 4 && T > 1 && B > 1 && st[0] != T * stride) value_error(std::string(name) + ": tokens must lie equally far apart");
  return {t.data_ptr(), B, T, heads, d, n > 1 ? stride : heads * d};
}

const char kEmbedDoc[] =
    "rotary_embed(q, k, cos, sin, *, positions=None, interleaved=False, inverse=False, q_out=None, "
    "k_out=None)\n--\n\n"
    "Queries and keys rotated by their positions.  q [B, T, Hq, D] and k [B, T, Hkv, D] (or\n"
    "[N, H, D]; k may be None), bf16 or fp32, may be slices of one projection's output; cos / sin\n"
    "fp32 [max_pos, rot_dim / 2]; positions int32 [B, T] ([N]), by default those in the row (at most\n"
    "max_pos of them), a negative one leaves its token as it is.  inverse turns back: the gradient.  Returns\n"
    "(q_out, k_out), new unless given (may be q and k).  No autograd graph is built: the gradient is\n"
    "the call with inverse; given outputs count as changed for graphs that saved them.";
PyObject* embed(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  static const Signature sig("rotary_embed", 4, 4,
                             {"q", "k", "cos", "sin", "positions", "interleaved", "inverse", "q_out", "k_out"});
  return guarded([&]() -> PyObject* {
    PyObject* o[32];
    sig.read(args, nargs, kwnames, o);
    const at::Tensor& qt = tensor(o[0], "q");
    if (!qt.is_cuda()) value_error("libsba works on CUDA tensors only (no CPU path)");
    if (qt.dim() != 3 && qt.dim() != 4) value_error("q must be [B, T, Hq, D] or [N, Hq, D]");
    const auto type = qt.scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) type_error("q must be bfloat16 or float32");
    const int index = static_cast<int>(qt.get_device());
    const PyObject* none = Py_None;
    const bool with_k = o[1] != none;
    if (!with_k && o[8]) value_error("k_out needs k");
    sba_rotary_embed_args a{};
    at::Tensor out[2];
    const Rows q = rows_of(qt, "q", qt);
    out[0] = o[7] ? tensor(o[7], "q_out") : fresh(qt.sizes(), type, index);
    const Rows qo = rows_of(out[0], "q_out", qt);
    if (qo.heads != q.heads) value_error("q_out must have q's shape");
    a.q = q.at;
    a.q_out = qo.at;
    a.q_stride = q.stride;
    a.q_out_stride = qo.stride;
    a.Hq = size32(q.heads, "q");
    if (with_k) {
      const at::Tensor& kt = tensor(o[1], "k");
      const Rows k = rows_of(kt, "k", qt);
      out[1] = o[8] ? tensor(o[8], "k_out") : fresh(kt.sizes(), type, index);
      const Rows ko = rows_of(out[1], "k_out", qt);
      if (ko.heads != k.heads) value_error("k_out must have k's shape");
      a.k = k.at;
      a.k_out = ko.at;
      a.k_stride = k.stride;
      a.k_out_stride = ko.stride;
      a.Hkv = size32(k.heads, "k");
    }
    const at::Tensor &cos = tensor(o[2], "cos"), &sin = tensor(o[3], "sin");
    if (cos.dim() != 2) value_error("cos and sin must be [max_pos, rot_dim / 2]");
    a.cos = static_cast<float*>(at_of(&cos, "cos", index, at::kFloat, cos.sizes(), "q's"));
    a.sin = static_cast<float*>(at_of(&sin, "sin", index, at::kFloat, cos.sizes(), "q's"));
    a.max_pos = size32(cos.size(0), "cos");
    a.rot_dim = size32(2 * cos.size(1), "cos");
    a.positions = static_cast<int32_t*>(at_of(optional(o[4], "positions"), "positions", index, at::kInt,
                                              qt.sizes().slice(0, qt.dim() - 2), "q's"));
    a.B = size32(q.B, "q");
    a.T = size32(q.T, "q");
    a.D = size32(q.d, "q");
    a.dtype = type == at::kFloat ? SBA_F32 : SBA_BF16;
    a.interleaved = truth(o[5], false);
    a.inverse = truth(o[6], false);
    call(sba_rotary_embed, a, index);
    written(o[7]);
    written(o[8]);
    PyObject* x = o[7] ? Py_NewRef(o[7]) : THPVariable_Wrap(out[0]);
    PyObject* y = x ? (o[8] ? Py_NewRef(o[8]) : with_k ? THPVariable_Wrap(out[1]) : Py_NewRef(Py_None)) : nullptr;
    PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    if (!r) throw Raised{};
    return r;
  });
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(type);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"paged_kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)),
     METH_FASTCALL | METH_KEYWORDS, kAppendDoc},
    {"paged_attention_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)),
     METH_FASTCALL | METH_KEYWORDS, kAttentionDoc},
    {"nsa_select_paged_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(select)),
     METH_FASTCALL | METH_KEYWORDS, kSelectDoc},
    {"blocksparse_attn_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grad)),
     METH_FASTCALL | METH_KEYWORDS, kGradDoc},
    {"rotary_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tables)),
     METH_FASTCALL | METH_KEYWORDS, kTablesDoc},
    {"rotary_embed", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(embed)),
     METH_FASTCALL | METH_KEYWORDS, kEmbedDoc},
    {"set_error", set_error, METH_O, "The exception class for the library's error codes: (code, message)."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged", "Calls of libsba bound in C++: paged caches, rotary positions, block-sparse gradients.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__paged() { return PyModule_Create(&kModule); }
