// Python side of the paged-cache calls: looks the tensors over, allocates outputs and workspaces where
// the caller left them out, and calls the C ABI (include/fa.h) with their addresses.
//
// These are the calls of a serving step, a few microseconds of GPU work each when the batch is small.
// Checked and marshalled in Python a call took the host 18 us (append, 3 of them the launch) to 28 us
// (decode: two launches, two outputs, a workspace), here 4 and 8.  The library's functions come from
// the handle of the libfa.so that the package has loaded (bind()), errors go up as the package's FaError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <dlfcn.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <type_traits>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fa.h"

namespace {

struct Library {
  decltype(&fa_append_paged) append = nullptr;
  decltype(&fa_append_paged_q4) append_q4 = nullptr;
  decltype(&fa_gather_paged_q4) gather_q4 = nullptr;
  decltype(&fa_decode_paged_q4) decode_q4 = nullptr;
  decltype(&fa_decode_paged_q4_workspace_size) decode_q4_ws = nullptr;
  decltype(&fa_fwd_paged_q4) fwd_q4 = nullptr;
  decltype(&fa_fwd_paged_q4_workspace_size) fwd_q4_ws = nullptr;
  decltype(&fa_last_error_message) message = nullptr;
};
Library lib;
PyObject* fa_error = nullptr;

// A refused call: FaError with this status, raised through the torch macros' catch.
struct Refused {
  int status;
  char text[400];
};

[[noreturn]] void refuse(const char* fmt, ...) {
  Refused r;
  r.status = FA_ERR_INVALID_ARG;
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(r.text, sizeof r.text, fmt, ap);
  va_end(ap);
  throw r;
}

void done(fa_status_t status) {
  if (status == FA_OK) return;
  Refused r;
  r.status = status;
  snprintf(r.text, sizeof r.text, "%s", lib.message());
  throw r;
}

PyObject* raise(const Refused& r) {
  PyObject* e = PyObject_CallFunction(fa_error, "is", r.status, r.text);
  if (e) {
    PyErr_SetObject(fa_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// The text of sizes, for messages.
struct Shape {
  char text[96];
  explicit Shape(c10::IntArrayRef s) {
    int n = snprintf(text, sizeof text, "[");
    // (a size has 19 digits at most: 21 characters with the comma before it, and the bracket and the 0 behind)
    const int room = static_cast<int>(sizeof text) - 23 - 5;
    for (size_t i = 0; i < s.size(); ++i) {
      if (n > room) {
        n += snprintf(text + n, sizeof text - n, ", ...");
        break;
      }
      n += snprintf(text + n, sizeof text - n, "%s%lld", i ? ", " : "", static_cast<long long>(s[i]));
    }
    snprintf(text + n, sizeof text - n, "]");
  }
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor, is %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& ranked(PyObject* o, const char* name, int dim, const char* layout) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dim) refuse("%s must be %s, is %s", name, layout, Shape(t.sizes()).text);
  return t;
}

// The tensors of a call are on one GPU; ``device`` is its index (-1 until the first).
void check(const at::Tensor& t, const char* name, c10::ScalarType type, std::initializer_list<int64_t> shape, int& device) {
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor, is on %s", name, t.device().str().c_str());
  if (device < 0) device = t.get_device();
  if (t.get_device() != device) refuse("%s must be a CUDA tensor on the cache's device %d, is on %d", name, device, static_cast<int>(t.get_device()));
  if (t.scalar_type() != type) refuse("%s must be %s, is %s", name, c10::toString(type), c10::toString(t.scalar_type()));
  const c10::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want) refuse("%s must be %s, is %s", name, Shape(want).text, Shape(t.sizes()).text);
}

template <typename P>
P* dense(const at::Tensor& t, const char* name, c10::ScalarType type, std::initializer_list<int64_t> shape, int& device) {
  check(t, name, type, shape, device);
  if (!t.is_contiguous()) refuse("%s must be dense", name);
  return static_cast<P*>(t.data_ptr());
}

// Packed tokens [total, heads, d]: each token's heads dense, tokens ``stride`` elements apart.
const fa_bf16_t* tokens(const at::Tensor& t, const char* name, std::initializer_list<int64_t> shape, int& device, long long* stride) {
  check(t, name, at::kBFloat16, shape, device);
  if (t.numel() && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2)))) refuse("%s must be dense in its last two dimensions", name);
  *stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);   // (a single token's is any number)
  return static_cast<const fa_bf16_t*>(t.data_ptr());
}

struct Cache4 {
  int device = -1;
  int64_t blocks, heads, block_size, d;
  fa_e2m1x2_t *k, *v;
  fa_e4m3_t *ks, *vs;
  Cache4(PyObject* k_codes, PyObject* k_scales, PyObject* v_codes, PyObject* v_scales) {
    const at::Tensor& c = ranked(k_codes, "k_codes", 4, "[num_blocks, H_kv, block_size, d/2]");
    blocks = c.size(0);
    heads = c.size(1);
    block_size = c.size(2);
    d = 2 * c.size(3);
    const at::Tensor& s = tensor(k_scales, "k_scales");
    const c10::ScalarType type = s.scalar_type() == at::kByte ? at::kByte : at::kFloat8_e4m3fn;
    k = dense<fa_e2m1x2_t>(c, "k_codes", at::kByte, {blocks, heads, block_size, d / 2}, device);
    v = dense<fa_e2m1x2_t>(tensor(v_codes, "v_codes"), "v_codes", at::kByte, {blocks, heads, block_size, d / 2}, device);
    ks = dense<fa_e4m3_t>(s, "k_scales", type, {blocks, heads, block_size, d / 16}, device);
    vs = dense<fa_e4m3_t>(tensor(v_scales, "v_scales"), "v_scales", type, {blocks, heads, block_size, d / 16}, device);
  }
};

// Sizes go to the C ABI as ints.
int narrow(int64_t n, const char* name) {
  if (n < INT32_MIN || n > INT32_MAX) refuse("%s = %lld is too large", name, static_cast<long long>(n));
  return static_cast<int>(n);
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s must be an integer, is %s", name, Py_TYPE(o)->tp_name);
  }
  return v;
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s must be a number, is %s", name, Py_TYPE(o)->tp_name);
  }
  return static_cast<float>(v);
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {                                                  // (several elements, say)
    PyErr_Clear();
    refuse("%s must be true or false, is %s", name, Py_TYPE(o)->tp_name);
  }
  return v == 1;
}

// Where a call runs: on ``device``, and on its current stream (None) or on a stream that is given by its
// handle or as an object that has one.  What the call allocates then belongs to that stream, as under
// torch.cuda.stream(): a workspace freed on return is not handed to work of another stream beside it.
struct Where {
  c10::cuda::CUDAGuard guard;
  c10::cuda::OptionalCUDAStreamGuard other;
  void* stream;
  Where(PyObject* o, int device) : guard(static_cast<c10::DeviceIndex>(device)) {
    if (!given(o)) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
      return;
    }
    if (PyLong_Check(o)) {
      stream = PyLong_AsVoidPtr(o);
    } else {
      PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
      const bool has = h && PyLong_Check(h);
      stream = has ? PyLong_AsVoidPtr(h) : nullptr;
      Py_XDECREF(h);
      if (!has) {
        PyErr_Clear();
        refuse("stream must be a stream, its handle or None, is %s", Py_TYPE(o)->tp_name);
      }
    }
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse("a stream's handle must be an address");
    }
    // (cudaStreamLegacy is torch's default stream, whose handle is 0; of other odd handles there are none)
    cudaStream_t handle = static_cast<cudaStream_t>(stream);
    if (handle == cudaStreamLegacy) handle = nullptr;
    other.reset_stream(c10::cuda::getStreamFromExternal(handle, static_cast<c10::DeviceIndex>(device)));
  }
};

// (not through the dispatcher: 1.7 us a tensor)
at::Tensor make(c10::IntArrayRef shape, c10::ScalarType type, int device) {
  return at::Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device)), std::nullopt));
}

// The caller's workspace, or ``need`` bytes for the call where it has none of that size (``own``: allowed to).
struct Workspace {
  c10::DataPtr held;
  void* ptr = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, size_t need, int device, bool own) {
    if (given(o)) {
      const at::Tensor& t = tensor(o, "workspace");
      if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous()) refuse("the workspace must be dense and on the cache's device");
      ptr = t.data_ptr();
      bytes = t.nbytes();
    }
    if (own && need > 16 && bytes < need) {
      held = c10::cuda::CUDACachingAllocator::get()->allocate(need);
      ptr = held.get();
      bytes = need;
    }
  }
};

#define FA_BEGIN HANDLE_TH_ERRORS try {
#define FA_END                  \
  }                             \
  catch (const Refused& r) {    \
    return raise(r);            \
  }                             \
  END_HANDLE_TH_ERRORS

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("%lld arguments instead of %lld", static_cast<long long>(n), static_cast<long long>(want));
}

// (q, k, v, q_out, k_cache, k_scales, v_cache, v_scales, cos, sin, cu_seqlens, seqlens_k, block_table,
//  descale_k, descale_v, interleaved, stream): k_scales None for the bf16 cache; q_out None with q: made.
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FA_BEGIN
  count(n, 17);
  const bool q4 = given(a[5]);
  int device = -1;
  int64_t blocks, heads, block_size, d;
  void *kc, *vc;
  fa_e4m3_t *ks = nullptr, *vs = nullptr;
  if (q4) {
    const Cache4 c(a[4], a[5], a[6], a[7]);
    device = c.device; blocks = c.blocks; heads = c.heads; block_size = c.block_size; d = c.d;
    kc = c.k; vc = c.v; ks = c.ks; vs = c.vs;
  } else {
    const at::Tensor& c = ranked(a[4], "k_cache", 4, "[num_blocks, block_size, H_kv, d]");
    blocks = c.size(0); block_size = c.size(1); heads = c.size(2); d = c.size(3);
    kc = dense<void>(c, "k_cache", at::kBFloat16, {blocks, block_size, heads, d}, device);
    vc = dense<void>(tensor(a[6], "v_cache"), "v_cache", at::kBFloat16, {blocks, block_size, heads, d}, device);
  }
  const at::Tensor& k = ranked(a[1], "k", 3, "[total, H_kv, d]");
  const at::Tensor& table = ranked(a[12], "block_table", 2, "[n_seqs, max_blocks]");
  const int64_t total = k.size(0), seqs = table.size(0);
  long long sq = 0, sk, sv;
  const fa_bf16_t* pk = tokens(k, "k", {total, heads, d}, device, &sk);
  const fa_bf16_t* pv = tokens(tensor(a[2], "v"), "v", {total, heads, d}, device, &sv);
  const Where on(a[16], device);
  const fa_bf16_t* pq = nullptr;
  fa_bf16_t* po = nullptr;
  int64_t H = 0;
  at::Tensor q_out;
  if (given(a[0])) {
    const at::Tensor& q = ranked(a[0], "q", 3, "[total, H, d]");
    H = q.size(1);
    pq = tokens(q, "q", {total, H, d}, device, &sq);
    q_out = given(a[3]) ? tensor(a[3], "q_out") : make({total, H, d}, at::kBFloat16, device);
    po = dense<fa_bf16_t>(q_out, "q_out", at::kBFloat16, {total, H, d}, device);
  } else if (given(a[3])) {
    refuse("q and q_out go together");
  }
  if (given(a[8]) != given(a[9])) refuse("cos and sin go together");
  const float *cos = nullptr, *sin = nullptr;
  int64_t half = 0, positions = 0;
  if (given(a[8])) {
    const at::Tensor& c = ranked(a[8], "cos", 2, "[n_positions, rotary_dim/2]");
    positions = c.size(0);
    half = c.size(1);
    cos = dense<float>(c, "cos", at::kFloat, {positions, half}, device);
    sin = dense<float>(tensor(a[9], "sin"), "sin", at::kFloat, {positions, half}, device);
  }
  const int* cu = dense<int>(tensor(a[10], "cu_seqlens"), "cu_seqlens", at::kInt, {seqs + 1}, device);
  const int* lens = dense<int>(tensor(a[11], "seqlens_k"), "seqlens_k", at::kInt, {seqs}, device);
  const int* tab = dense<int>(table, "block_table", at::kInt, {seqs, table.size(1)}, device);
  const int ints[] = {narrow(seqs, "n_seqs"), narrow(H, "H"), narrow(heads, "H_kv"), narrow(total, "total"), narrow(table.size(1), "max_blocks"),
                      narrow(block_size, "block_size"), narrow(blocks, "num_blocks"), narrow(d, "d"), narrow(2 * half, "rotary_dim"),
                      truth(a[15], "interleaved") ? 1 : 0, narrow(positions, "n_positions")};
  if (q4)
    done(lib.append_q4(pq, pk, pv, po, static_cast<fa_e2m1x2_t*>(kc), ks, static_cast<fa_e2m1x2_t*>(vc), vs, cos, sin, cu, lens, tab, ints[0],
                       ints[1], ints[2], ints[3], sq, sk, sv, ints[4], ints[5], ints[6], ints[7], ints[8], ints[9], ints[10],
                       number(a[13], "descale_k"), number(a[14], "descale_v"), on.stream));
  else
    done(lib.append(pq, pk, pv, po, static_cast<fa_bf16_t*>(kc), static_cast<fa_bf16_t*>(vc), cos, sin, cu, lens, tab, ints[0], ints[1], ints[2],
                    ints[3], sq, sk, sv, ints[4], ints[5], ints[6], ints[7], ints[8], ints[9], ints[10], on.stream));
  if (!q_out.defined()) Py_RETURN_NONE;
  if (given(a[3])) {
    Py_INCREF(a[3]);
    return a[3];
  }
  return THPVariable_Wrap(q_out);
  FA_END
}

PyObject* two(const at::Tensor& x, PyObject* had_x, const at::Tensor& y, PyObject* had_y) {
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  for (int i = 0; i < 2; ++i) {
    PyObject* had = i ? had_y : had_x;
    PyObject* o = had;
    if (given(had)) Py_INCREF(had);
    else o = THPVariable_Wrap(i ? y : x);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// (k_codes, k_scales, v_codes, v_scales, k, v, total, cu_seqlens, seqlens_k, block_table, descale_k,
//  descale_v, stream): k and v None: made, of ``total`` rows.
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FA_BEGIN
  count(n, 13);
  Cache4 c(a[0], a[1], a[2], a[3]);
  const at::Tensor& table = ranked(a[9], "block_table", 2, "[n_seqs, max_blocks]");
  const int64_t seqs = table.size(0);
  const int64_t total = given(a[4]) ? ranked(a[4], "k", 3, "[total, H_kv, d]").size(0) : integer(a[6], "total");
  if (total < 0) refuse("total must be >= 0 (got %lld)", static_cast<long long>(total));
  const Where on(a[12], c.device);
  const at::Tensor k = given(a[4]) ? tensor(a[4], "k") : make({total, c.heads, c.d}, at::kBFloat16, c.device);
  const at::Tensor v = given(a[5]) ? tensor(a[5], "v") : make({total, c.heads, c.d}, at::kBFloat16, c.device);
  fa_bf16_t* pk = dense<fa_bf16_t>(k, "k", at::kBFloat16, {total, c.heads, c.d}, c.device);
  fa_bf16_t* pv = dense<fa_bf16_t>(v, "v", at::kBFloat16, {total, c.heads, c.d}, c.device);
  const int* cu = dense<int>(tensor(a[7], "cu_seqlens"), "cu_seqlens", at::kInt, {seqs + 1}, c.device);
  const int* lens = dense<int>(tensor(a[8], "seqlens_k"), "seqlens_k", at::kInt, {seqs}, c.device);
  const int* tab = dense<int>(table, "block_table", at::kInt, {seqs, table.size(1)}, c.device);
  done(lib.gather_q4(c.k, c.ks, c.v, c.vs, pk, pv, cu, lens, tab, narrow(seqs, "n_seqs"), narrow(c.heads, "H_kv"), narrow(total, "total"),
                     narrow(table.size(1), "max_blocks"), narrow(c.block_size, "block_size"), narrow(c.blocks, "num_blocks"), narrow(c.d, "d"),
                     number(a[10], "descale_k"), number(a[11], "descale_v"), on.stream));
  return two(k, a[4], v, a[5]);
  FA_END
}

// (q, k_codes, k_scales, v_codes, v_scales, o, lse, block_table, seqlens_k, max_seqlen_k, scale, descale_k,
//  descale_v, n_splits, ws, stream, own): ``own``: outputs and workspace that are None are made, and a
// scale of None is 1 / sqrt(d).
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FA_BEGIN
  count(n, 17);
  const bool own = truth(a[16], "own");
  Cache4 c(a[1], a[2], a[3], a[4]);
  const at::Tensor& q = ranked(a[0], "q", 4, "[B, H, 1, d]");
  const at::Tensor& table = ranked(a[7], "block_table", 2, "[B, max_blocks]");
  const int64_t B = q.size(0), H = q.size(1);
  if (c.d != q.size(3)) refuse("k_codes must be [num_blocks, H_kv, block_size, %lld/2]", static_cast<long long>(q.size(3)));
  const fa_bf16_t* pq = dense<fa_bf16_t>(q, "q", at::kBFloat16, {B, H, 1, c.d}, c.device);
  const int* tab = dense<int>(table, "block_table", at::kInt, {B, table.size(1)}, c.device);
  const int* lens = dense<int>(tensor(a[8], "seqlens_k"), "seqlens_k", at::kInt, {B}, c.device);
  const int max_k = narrow(integer(a[9], "max_seqlen_k"), "max_seqlen_k"), splits = narrow(integer(a[13], "n_splits"), "n_splits");
  const int b = narrow(B, "B"), h = narrow(H, "H"), hkv = narrow(c.heads, "H_kv"), d = narrow(c.d, "d");
  const float scale = given(a[10]) ? number(a[10], "scale") : 1.f / std::sqrt(static_cast<float>(d));
  const Where on(a[15], c.device);
  const at::Tensor o = own && !given(a[5]) ? make({B, H, 1, c.d}, at::kBFloat16, c.device) : tensor(a[5], "o");
  const at::Tensor lse = own && !given(a[6]) ? make({B, H, 1}, at::kFloat, c.device) : tensor(a[6], "lse");
  fa_bf16_t* po = dense<fa_bf16_t>(o, "o", at::kBFloat16, {B, H, 1, c.d}, c.device);
  float* pl = dense<float>(lse, "lse", at::kFloat, {B, H, 1}, c.device);
  const Workspace ws(a[14], own ? lib.decode_q4_ws(b, h, hkv, max_k, d, splits) : 0, c.device, own);
  done(lib.decode_q4(pq, c.k, c.ks, c.v, c.vs, po, pl, tab, lens, b, h, hkv, narrow(table.size(1), "max_blocks"), narrow(c.block_size, "block_size"),
                     narrow(c.blocks, "num_blocks"), max_k, d, scale, number(a[11], "descale_k"), number(a[12], "descale_v"), splits,
                     ws.ptr, ws.bytes, on.stream));
  return two(o, a[5], lse, a[6]);
  FA_END
}

// (q, k_codes, k_scales, v_codes, v_scales, o, lse, cu_seqlens_q, seqlens_k, block_table, max_seqlen_q,
//  max_seqlen_k, scale, descale_k, descale_v, causal, n_splits, ws, stream, own): as decode().
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  FA_BEGIN
  count(n, 20);
  const bool own = truth(a[19], "own");
  Cache4 c(a[1], a[2], a[3], a[4]);
  const at::Tensor& q = ranked(a[0], "q", 3, "[total_q, H, d]");
  const at::Tensor& table = ranked(a[9], "block_table", 2, "[n_seqs, max_blocks]");
  const int64_t total = q.size(0), H = q.size(1), seqs = table.size(0);
  if (c.d != q.size(2)) refuse("k_codes must be [num_blocks, H_kv, block_size, %lld/2]", static_cast<long long>(q.size(2)));
  const fa_bf16_t* pq = dense<fa_bf16_t>(q, "q", at::kBFloat16, {total, H, c.d}, c.device);
  const int* cu = dense<int>(tensor(a[7], "cu_seqlens_q"), "cu_seqlens_q", at::kInt, {seqs + 1}, c.device);
  const int* lens = dense<int>(tensor(a[8], "seqlens_k"), "seqlens_k", at::kInt, {seqs}, c.device);
  const int* tab = dense<int>(table, "block_table", at::kInt, {seqs, table.size(1)}, c.device);
  const int max_q = narrow(integer(a[10], "max_seqlen_q"), "max_seqlen_q"), max_k = narrow(integer(a[11], "max_seqlen_k"), "max_seqlen_k");
  const int splits = narrow(integer(a[16], "n_splits"), "n_splits");
  const int s = narrow(seqs, "n_seqs"), t = narrow(total, "total_q"), h = narrow(H, "H"), hkv = narrow(c.heads, "H_kv"), d = narrow(c.d, "d");
  const float scale = given(a[12]) ? number(a[12], "scale") : 1.f / std::sqrt(static_cast<float>(d));
  const Where on(a[18], c.device);
  const at::Tensor o = own && !given(a[5]) ? make({total, H, c.d}, at::kBFloat16, c.device) : tensor(a[5], "o");
  const at::Tensor lse = own && !given(a[6]) ? make({H, total}, at::kFloat, c.device) : tensor(a[6], "lse");
  fa_bf16_t* po = dense<fa_bf16_t>(o, "o", at::kBFloat16, {total, H, c.d}, c.device);
  float* pl = dense<float>(lse, "lse", at::kFloat, {H, total}, c.device);
  const Workspace ws(a[17], own ? lib.fwd_q4_ws(s, h, hkv, t, max_q, max_k, d, splits) : 0, c.device, own);
  done(lib.fwd_q4(pq, c.k, c.ks, c.v, c.vs, po, pl, cu, lens, tab, s, h, hkv, t, max_q, narrow(table.size(1), "max_blocks"),
                  narrow(c.block_size, "block_size"), narrow(c.blocks, "num_blocks"), max_k, d, scale, number(a[13], "descale_k"),
                  number(a[14], "descale_v"), truth(a[15], "causal") ? 1 : 0, splits, ws.ptr, ws.bytes,
                  on.stream));
  return two(o, a[5], lse, a[6]);
  FA_END
}

// (FaError, handle of libfa.so)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) return PyErr_Format(PyExc_TypeError, "bind(FaError, handle)");
  void* h = PyLong_AsVoidPtr(a[1]);
  if (!h && PyErr_Occurred()) return nullptr;
  bool ok = true;
  auto find = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(h, name));
    ok = ok && f;
  };
  find(lib.append, "fa_append_paged");
  find(lib.append_q4, "fa_append_paged_q4");
  find(lib.gather_q4, "fa_gather_paged_q4");
  find(lib.decode_q4, "fa_decode_paged_q4");
  find(lib.decode_q4_ws, "fa_decode_paged_q4_workspace_size");
  find(lib.fwd_q4, "fa_fwd_paged_q4");
  find(lib.fwd_q4_ws, "fa_fwd_paged_q4_workspace_size");
  find(lib.message, "fa_last_error_message");
  if (!ok) return PyErr_Format(PyExc_RuntimeError, "libfa.so lacks a paged-cache function");
  Py_INCREF(a[0]);
  Py_XSETREF(fa_error, a[0]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}

PyMethodDef methods[] = {{"bind", fast<bind>(), METH_FASTCALL, nullptr},     {"append", fast<append>(), METH_FASTCALL, nullptr},
                         {"gather", fast<gather>(), METH_FASTCALL, nullptr}, {"decode", fast<decode>(), METH_FASTCALL, nullptr},
                         {"forward", fast<forward>(), METH_FASTCALL, nullptr}, {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
