// pa_calls.cpp -- the Python module _calls: the checks and the argument passing of the
// speculative-decoding calls and of those for bounded caches over torch tensors (binding.py documents
// them and raises PaError).
//
// Why not ctypes, as for the calls around it: their kernels take 2 to 15 us at serving sizes, and
// reading some ten tensors' properties and converting up to thirty arguments took 3 to 10 us of
// Python a call (rotary caching 14.4 us a call, one tree of 8 nodes 29 us; 3.0 and 14.2 in a
// captured graph).  Through this module the same checks take under a microsecond.
//
// Checks raise ValueError (TypeError for what is not a tensor or a number); the functions return
// the library's status.  Calls that are not given a workspace they need take it from torch's
// allocator, from the pool of the stream that the call goes to; no other call allocates.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <initializer_list>
#include <optional>

#include "pa.h"

namespace {

struct Bad {  // a refused argument: a ValueError, or the Python error that is set already
  const char* what;
};

using Args = PyObject* const*;

bool none(PyObject* o) { return o == Py_None; }

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "a tensor is expected");
    throw Bad{nullptr};
  }
  return THPVariable_Unpack(o);
}
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Bad{nullptr};
  return x;
}
int32_t int32(int64_t x) {
  if (x < INT32_MIN || x > INT32_MAX) throw Bad{"a size does not fit 32 bits"};
  return (int32_t)x;
}
int32_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Bad{nullptr};
  return int32(x);
}

// Other Python threads may run while the library is at work (a launch may wait for room in the
// device's queue).
struct Released {
  PyThreadState* state = PyEval_SaveThread();
  ~Released() { PyEval_RestoreThread(state); }
};

// The call's device (the current one) and stream.
struct Call {
  int dev;
  cudaStream_t stream;
  bool given;  // a stream was given: it need not be the current one
  explicit Call(PyObject* s) : dev(c10::cuda::current_device()), given(!none(s)) {
    if (!given) {
      stream = c10::cuda::getCurrentCUDAStream(dev).stream();
      return;
    }
    PyObject* h = PyObject_GetAttrString(s, "cuda_stream");
    if (!h) throw Bad{nullptr};
    stream = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Bad{nullptr};
  }
  bool here(const at::Tensor& t) const { return t.is_cuda() && t.get_device() == dev; }
  const at::Tensor& array(PyObject* o) const {
    const at::Tensor& t = tensor(o);
    if (!here(t) || !t.is_contiguous())
      throw Bad{"tensors must be contiguous and live on the current CUDA device"};
    return t;
  }
  int32_t* ints(PyObject* o, int64_t* numel = nullptr) const {
    const at::Tensor& t = array(o);
    if (t.scalar_type() != at::kInt) throw Bad{"metadata tensors must be int32"};
    if (numel) *numel = t.numel();
    return static_cast<int32_t*>(t.data_ptr());
  }
  // An optional fp32 array of the shape a (x b).
  float* floats(PyObject* o, int64_t a, int64_t b, const char* what) const {
    if (none(o)) return nullptr;
    const at::Tensor& t = array(o);
    if (t.scalar_type() != at::kFloat || t.dim() != (b < 0 ? 1 : 2) || t.size(0) != a ||
        (b >= 0 && t.size(1) != b))
      throw Bad{what};
    return static_cast<float*>(t.data_ptr());
  }
  float* head_scales(PyObject* o, int64_t heads) const {
    return floats(o, heads, -1, "per-head scales must be contiguous fp32 [num_kv_heads] tensors");
  }
};

pa_dtype dtype(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return PA_F32;
    case at::kBFloat16: return PA_BF16;
    case at::kFloat8_e4m3fn: return PA_FP8_E4M3;
    default: throw Bad{"tensors must be float32, bfloat16 or float8_e4m3fn"};
  }
}

// Both pools [num_blocks, block, kv heads, head size]; V may be missing.
struct Pools {
  void *k, *v;
  int64_t blocks;
  int32_t block, heads, dim;
  pa_dtype type;
  Pools(const Call& c, PyObject* ko, PyObject* vo, bool v_optional = false) : v(nullptr) {
    const at::Tensor& kt = c.array(ko);
    if (kt.dim() != 4) throw Bad{"pools must be [NB, b, Hkv, D]"};
    if (!v_optional || !none(vo)) {
      const at::Tensor& vt = c.array(vo);
      if (vt.sizes() != kt.sizes() || vt.scalar_type() != kt.scalar_type())
        throw Bad{"k_blocks and v_blocks must match"};
      v = vt.data_ptr();
    }
    k = kt.data_ptr();
    blocks = kt.size(0);
    block = int32(kt.size(1));
    heads = int32(kt.size(2));
    dim = int32(kt.size(3));
    type = dtype(kt);
  }
};

// A call's workspace: the tensor given, or one of `size()` bytes.
struct Workspace {
  std::optional<at::Tensor> own;
  void* ptr;
  size_t bytes;
  template <typename F>
  Workspace(const Call& c, PyObject* o, F size) {
    if (none(o)) {
      bytes = size();
      // memory of another stream's pool may still be in use by what that stream has queued
      c10::cuda::OptionalCUDAStreamGuard guard;
      if (c.given)
        guard.reset_stream(c10::cuda::getStreamFromExternal(c.stream, (c10::DeviceIndex)c.dev));
      own = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(
                                            at::kCUDA, (c10::DeviceIndex)c.dev));
      ptr = own->data_ptr();
    } else {
      const at::Tensor& t = c.array(o);
      ptr = t.data_ptr();
      bytes = t.nbytes();
    }
  }
};

// Elements between the tokens of [T, N, D] rows whose heads are contiguous.
int64_t token_stride(const at::Tensor& t) {
  if ((t.stride(2) != 1 && t.size(2) > 1) || (t.stride(1) != t.size(2) && t.size(1) > 1))
    throw Bad{"q, k, v, q_out: a token's heads must be contiguous"};
  return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

pa_status rope_and_cache(Args a) {
  const Call c(a[15]);
  if (none(a[0]) != none(a[3])) throw Bad{"give both q and q_out or neither"};
  auto rows = [&](PyObject* o) -> const at::Tensor& {
    const at::Tensor& t = tensor(o);
    if (!c.here(t) || t.dim() != 3)
      throw Bad{"q, k, v and q_out must be [T, heads, D] tensors on the current CUDA device"};
    return t;
  };
  const at::Tensor &k = rows(a[1]), &v = rows(a[2]);
  const Pools p(c, a[4], a[5]);
  if (v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
    throw Bad{"k and v must be [T, Hkv, D] of one dtype"};
  if (k.size(1) != p.heads || k.size(2) != p.dim)
    throw Bad{"kv heads / head size differ between rows and pool"};
  const int64_t T = k.size(0);
  int64_t np, ns;
  const int32_t *pos = c.ints(a[6], &np), *slots = c.ints(a[7], &ns);
  if (np != T || ns != T) throw Bad{"positions and slot_mapping must be [T]"};
  const at::Tensor& freq = c.array(a[8]);
  if (freq.scalar_type() != at::kDouble || freq.dim() != 1)
    throw Bad{"inv_freq must be fp64 [rotary_dim / 2]"};
  const void* q = nullptr;
  void* q_out = nullptr;
  int64_t q_stride = 0, q_out_stride = 0, heads = 0;
  if (!none(a[0])) {
    const at::Tensor &qt = rows(a[0]), &ot = rows(a[3]);
    if (qt.size(0) != T || qt.size(2) != p.dim || ot.sizes() != qt.sizes() ||
        qt.scalar_type() != k.scalar_type() || ot.scalar_type() != k.scalar_type())
      throw Bad{"q and q_out must be [T, H, D] of the rows' dtype"};
    heads = qt.size(1);
    q = qt.data_ptr();
    q_out = ot.data_ptr();
    q_stride = token_stride(qt);
    q_out_stride = token_stride(ot);
  }
  const int interleaved = PyObject_IsTrue(a[9]);
  if (interleaved < 0) throw Bad{nullptr};
  const float factor = (float)number(a[10]), ks = (float)number(a[11]), vs = (float)number(a[12]);
  const float *kss = c.head_scales(a[13], p.heads), *vss = c.head_scales(a[14], p.heads);
  const int64_t k_stride = token_stride(k), v_stride = token_stride(v);
  const pa_dtype type = dtype(k);
  const int32_t H = int32(heads), rotary = int32(2 * freq.numel());
  const double* f = static_cast<const double*>(freq.data_ptr());
  Released r;
  return pa_rope_and_cache(q, q_stride, q_out, q_out_stride, k.data_ptr(), k_stride, v.data_ptr(),
                           v_stride, p.k, p.v, pos, slots, f, rotary, interleaved, factor, T, H,
                           p.heads, p.dim, p.block, p.blocks, type, p.type, ks, vs, kss, vss,
                           c.stream);
}

pa_status tree_attention(Args a) {
  const Call c(a[12]);
  const at::Tensor &q = c.array(a[0]), &out = c.array(a[3]);
  if (q.dim() != 3 || out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type())
    throw Bad{"q and out must be [T, H, D] of one dtype"};
  const Pools p(c, a[1], a[2]);
  const int64_t T = q.size(0), D = q.size(2);
  const int32_t H = int32(q.size(1));
  if (D != p.dim) throw Bad{"head size differs between q and the pool"};
  int64_t nq, nl, np;
  const int32_t *qsl = c.ints(a[4], &nq), *lens = c.ints(a[5], &nl), *pos = c.ints(a[6], &np);
  const at::Tensor &mask = c.array(a[7]), &tables = c.array(a[8]);
  const int32_t *mask_ptr = c.ints(a[7]), *table_ptr = c.ints(a[8]);
  if (mask.dim() != 2 || mask.size(0) != T || np != T)
    throw Bad{"tree_mask must be [T, mask_words] and positions [T]"};
  const int32_t S = int32(nq - 1);
  if (nl != S || tables.dim() != 2 || tables.size(0) != S)
    throw Bad{"seq_lens must be [S] and block_tables [S, max_blocks]"};
  const int32_t max_blocks = int32(tables.size(1));
  const float* sinks = c.floats(a[13], H, -1, "sinks must be a contiguous fp32 [num_heads] tensor");
  float* lse =
      c.floats(a[14], H, T, "lse must be a contiguous fp32 [num_heads, num_tokens] tensor");
  const float scale = (float)number(a[9]), ks = (float)number(a[15]), vs = (float)number(a[16]);
  const int32_t window = integer(a[10]), words = int32(mask.size(1));
  const float *kss = c.head_scales(a[17], p.heads), *vss = c.head_scales(a[18], p.heads);
  const pa_dtype type = dtype(q);
  const Workspace ws(c, a[11], [&] {
    return pa_tree_attention_workspace_size(S, T, H, p.heads, p.dim, max_blocks, p.block);
  });
  Released r;
  return pa_tree_attention(q.data_ptr(), p.k, p.v, out.data_ptr(), qsl, lens, pos, mask_ptr,
                           table_ptr, S, T, words, H, p.heads, p.dim, p.block, p.blocks, max_blocks,
                           type, p.type, scale, window, sinks, lse, ks, vs, kss, vss, ws.ptr, ws.bytes,
                           c.stream);
}

pa_status tree_commit(Args a) {
  const Call c(a[6]);
  const Pools p(c, a[0], a[1]);
  const at::Tensor &tables = c.array(a[2]), &acc = c.array(a[4]);
  int64_t nctx, nnum;
  const int32_t *table_ptr = c.ints(a[2]), *ctx = c.ints(a[3], &nctx), *accepted = c.ints(a[4]),
                *num = c.ints(a[5], &nnum);
  if (acc.dim() != 2 || tables.dim() != 2)
    throw Bad{"accepted must be [S, max_accepted], block_tables [S, max_blocks]"};
  const int64_t S = acc.size(0);
  if (nctx != S || nnum != S || tables.size(0) != S)
    throw Bad{"context_lens and num_accepted must be [S]"};
  const int32_t seqs = int32(S), most = int32(acc.size(1)), max_blocks = int32(tables.size(1));
  Released r;
  return pa_tree_commit(p.k, p.v, table_ptr, ctx, accepted, num, seqs, most, p.heads, p.dim, p.block,
                        p.blocks, max_blocks, p.type, c.stream);
}

pa_status copy_blocks(Args a) {
  const Call c(a[3]);
  const Pools p(c, a[0], a[1], true);
  const at::Tensor& pairs = c.array(a[2]);
  const int32_t* ptr = c.ints(a[2]);
  if (pairs.dim() != 2 || pairs.size(1) != 2) throw Bad{"block_pairs must be [n, 2]"};
  const int64_t n = pairs.size(0);
  Released r;
  return pa_copy_blocks(p.k, p.v, ptr, n, p.heads, p.dim, p.block, p.blocks, p.type,
                        c.stream);
}

// The arrays of the page bookkeeping: tables, lengths, one or two lists, counts, free list and its
// length, block size.
struct Books {
  int32_t *tables, *lens, *refs, *free_list, *free_count;
  const int32_t *rows, *other;
  int32_t n, num_rows, max_blocks, block;
  int64_t blocks;
  Books(const Call& c, PyObject* t, PyObject* l, PyObject* r, PyObject* o, Args rest)
      : other(nullptr) {
    const at::Tensor& tt = c.array(t);
    int64_t nl, nr, no, nb, nf, nc;
    tables = c.ints(t);
    lens = c.ints(l, &nl);
    if (tt.dim() != 2 || nl != tt.size(0))
      throw Bad{"block_tables must be [rows, max_blocks] and seq_lens [rows]"};
    rows = c.ints(r, &nr);
    no = nr;
    if (o) other = c.ints(o, &no);
    if (no != nr) throw Bad{"the lists must have one length"};
    refs = c.ints(rest[0], &nb);
    free_list = c.ints(rest[1], &nf);
    free_count = c.ints(rest[2], &nc);
    if (nf != nb || nc != 1)
      throw Bad{"ref_counts and free_list must be [num_blocks], free_count [1]"};
    block = integer(rest[3]);
    n = int32(nr);
    num_rows = int32(tt.size(0));
    max_blocks = int32(tt.size(1));
    blocks = nb;
  }
};

pa_status fork_sequences(Args a) {
  const Call c(a[9]);
  const Books b(c, a[0], a[1], a[2], a[3], a + 4);
  const at::Tensor& pairs = c.array(a[8]);
  int32_t* ptr = c.ints(a[8]);
  if (pairs.dim() != 2 || pairs.size(0) != b.n || pairs.size(1) != 2)
    throw Bad{"block_pairs must be [n, 2]"};
  Released r;
  return pa_fork_sequences(b.tables, b.lens, b.rows, b.other, b.n, b.num_rows, b.max_blocks, b.block,
                           b.refs, b.free_list, b.free_count, b.blocks, ptr, c.stream);
}
pa_status grow_sequences(Args a) {
  const Call c(a[8]);
  const Books b(c, a[0], a[1], a[2], a[3], a + 4);
  Released r;
  return pa_grow_sequences(b.tables, b.lens, b.rows, b.other, b.n, b.num_rows, b.max_blocks, b.block,
                           b.refs, b.free_list, b.free_count, b.blocks, c.stream);
}
pa_status trim_sequences(Args a) {
  const Call c(a[8]);
  const Books b(c, a[0], a[1], a[2], a[3], a + 4);
  Released r;
  return pa_trim_sequences(b.tables, b.lens, b.rows, b.other, b.n, b.num_rows, b.max_blocks, b.block,
                           b.refs, b.free_list, b.free_count, b.blocks, c.stream);
}
pa_status free_sequences(Args a) {
  const Call c(a[7]);
  const Books b(c, a[0], a[1], a[2], nullptr, a + 3);
  Released r;
  return pa_free_sequences(b.tables, b.lens, b.rows, b.n, b.num_rows, b.max_blocks, b.block, b.refs,
                           b.free_list, b.free_count, b.blocks, c.stream);
}

// pa_window_attention's arguments; with WEIGH pa_attention_key_weights', which has two more at the end.
template <bool WEIGH>
pa_status window_attention(Args a) {
  const Call c(a[12]);
  const at::Tensor &q = c.array(a[0]), &out = c.array(a[3]);
  if (q.dim() != 3 || out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type())
    throw Bad{"q and out must be [T, H, D] of one dtype"};
  const Pools p(c, a[1], a[2]);
  const int64_t T = q.size(0);
  const int32_t H = int32(q.size(1));
  if (q.size(2) != p.dim) throw Bad{"head size differs between q and the pool"};
  int64_t nq, nl, np;
  const int32_t *qsl = c.ints(a[4], &nq), *lens = c.ints(a[5], &nl), *pos = c.ints(a[6], &np);
  const at::Tensor& tables = c.array(a[7]);
  const int32_t* table_ptr = c.ints(a[7]);
  if (np != T) throw Bad{"positions must be [T]"};
  const int32_t S = int32(nq - 1);
  if (nl != S || tables.dim() != 2 || tables.size(0) != S)
    throw Bad{"seq_lens must be [S] and block_tables [S, max_blocks]"};
  const int32_t max_blocks = int32(tables.size(1));
  const float scale = (float)number(a[8]), ks = (float)number(a[15]), vs = (float)number(a[16]);
  const int32_t window = integer(a[9]), first = integer(a[10]);
  const float* sinks = c.floats(a[13], H, -1, "sinks must be a contiguous fp32 [num_heads] tensor");
  float* lse =
      c.floats(a[14], H, T, "lse must be a contiguous fp32 [num_heads, num_tokens] tensor");
  const float *kss = c.head_scales(a[17], p.heads), *vss = c.head_scales(a[18], p.heads);
  const pa_dtype type = dtype(q);
  if constexpr (WEIGH) {
    const at::Tensor& w = c.array(a[19]);
    if (w.scalar_type() != at::kFloat || w.dim() != 3 || w.size(0) != S || w.size(1) != p.heads)
      throw Bad{"key_weights must be fp32 [num_seqs, num_kv_heads, length]"};
    const int32_t observed = integer(a[20]);
    float* wp = static_cast<float*>(w.data_ptr());
    const int64_t len = w.size(2);
    const Workspace ws(c, a[11], [&] {
      return pa_attention_key_weights_workspace_size(S, T, H, p.heads, p.dim, max_blocks, p.block);
    });
    Released r;
    return pa_attention_key_weights(q.data_ptr(), p.k, p.v, out.data_ptr(), qsl, lens, pos, table_ptr,
                                    wp, len, observed, S, T, H, p.heads, p.dim, p.block, p.blocks,
                                    max_blocks, type, p.type, scale, window, first, sinks, lse, ks, vs,
                                    kss, vss, ws.ptr, ws.bytes, c.stream);
  } else {
    const Workspace ws(c, a[11], [&] {
      return pa_window_attention_workspace_size(S, T, H, p.heads, p.dim, max_blocks, p.block);
    });
    Released r;
    return pa_window_attention(q.data_ptr(), p.k, p.v, out.data_ptr(), qsl, lens, pos, table_ptr, S, T,
                               H, p.heads, p.dim, p.block, p.blocks, max_blocks, type, p.type, scale,
                               window, first, sinks, lse, ks, vs, kss, vss, ws.ptr, ws.bytes, c.stream);
  }
}

pa_status evict_keys(Args a) {
  const Call c(a[9]);
  const Pools p(c, a[0], a[1]);
  const at::Tensor& tables = c.array(a[2]);
  int64_t nl, nn;
  const int32_t *table_ptr = c.ints(a[2]), *lens = c.ints(a[3], &nl), *new_lens = c.ints(a[4], &nn);
  if (tables.dim() != 2 || nl != tables.size(0) || nn != nl)
    throw Bad{"block_tables must be [S, max_blocks], seq_lens and new_lens [S]"};
  const int32_t S = int32(nl), max_blocks = int32(tables.size(1));
  float* w = nullptr;
  int64_t len = 0;
  if (!none(a[5])) {
    const at::Tensor& t = c.array(a[5]);
    if (t.scalar_type() != at::kFloat || t.dim() != 3 || t.size(0) != S || t.size(1) != p.heads)
      throw Bad{"key_weights must be fp32 [num_seqs, num_kv_heads, length]"};
    // (an array without an element has no address, and is not "no weights": its keys are refused)
    static float empty;
    w = t.numel() ? static_cast<float*>(t.data_ptr()) : &empty;
    len = t.size(2);
  }
  const int32_t first = integer(a[6]), recent = integer(a[7]);
  const Workspace ws(c, a[8], [&] {
    return pa_evict_keys_workspace_size(S, p.heads, max_blocks, p.block);
  });
  Released r;
  return pa_evict_keys(p.k, p.v, table_ptr, lens, new_lens, w, len, first, recent, S, p.heads, p.dim,
                       p.block, p.blocks, max_blocks, p.type, ws.ptr, ws.bytes, c.stream);
}

template <pa_status (*F)(Args), int N>
PyObject* entry(PyObject*, Args args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(args));
  } catch (const Bad& e) {
    if (e.what) PyErr_SetString(PyExc_ValueError, e.what);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <pa_status (*F)(Args), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {
    method<rope_and_cache, 16>("rope_and_cache"), method<tree_attention, 19>("tree_attention"),
    method<tree_commit, 7>("tree_commit"),        method<copy_blocks, 4>("copy_blocks"),
    method<fork_sequences, 10>("fork_sequences"), method<grow_sequences, 9>("grow_sequences"),
    method<trim_sequences, 9>("trim_sequences"),  method<free_sequences, 8>("free_sequences"),
    method<window_attention<false>, 19>("window_attention"),
    method<window_attention<true>, 21>("attention_key_weights"),
    method<evict_keys, 10>("evict_keys"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods,
                       nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
