// Native half of the Python binding for the operators around the product: it
// checks torch tensors, allocates outputs and workspaces and calls the C ABI.
// (In Python the same took 10 to 25 us a call, longer than most calls run.)
//
// Every function takes positional arguments and returns its tensors, or the
// status of the C call as an integer where that is not QMM_OK.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/cuda/CUDAEvent.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/qmm.h"

namespace {

// A Python exception of the given type, as a C++ one.
struct Refused {
  PyObject* type;
  const char* message;
};
[[noreturn]] void value_error(const char* m) { throw Refused{PyExc_ValueError, m}; }
[[noreturn]] void type_error(const char* m) { throw Refused{PyExc_TypeError, m}; }

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) type_error("a tensor is needed");
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, nullptr};
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, nullptr};
  return v;
}
int narrow(int64_t v) {
  if (v < 0 || v > 0x7fffffff) value_error("a size is out of range");
  return static_cast<int>(v);
}
bool is(const at::Tensor& t, at::ScalarType dtype, at::IntArrayRef shape) {
  return t.scalar_type() == dtype && t.sizes() == shape && t.is_contiguous();
}
const void* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

// The device and stream of a call.  One rule for a call on another stream than the
// current one: it waits for what the current one has been given so far (the inputs
// may still be computed there, and the allocator may hand out memory that it still
// works on), and every tensor of the call is recorded on the other stream, so that
// its memory is not handed out again before the call is done.
class Call {
 public:
  Call(const at::Tensor& first, PyObject* stream)
      : device_(first.device()), current_(current_stream(device_)), run_(current_) {
    if (stream != Py_None) {
      const cudaStream_t s = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
      if (PyErr_Occurred()) throw Refused{nullptr, nullptr};
      if (s != current_.stream()) {
        run_ = c10::cuda::getStreamFromExternal(s, device_.index());
        other_ = true;
        at::cuda::CUDAEvent e;
        e.record(current_);
        e.block(run_);
      }
    }
    here(&first);
  }
  void here(const at::Tensor* t) const {
    if (t == nullptr) return;
    if (t->device() != device_) value_error("all tensors must be on one CUDA device");
    if (other_) c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(), run_);
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) const {
    const at::Tensor t = at::detail::empty_cuda(shape, dtype, device_, std::nullopt);
    here(&t);
    return t;
  }
  void* stream() const { return run_.stream(); }

 private:
  static c10::cuda::CUDAStream current_stream(c10::Device device) {
    if (!device.is_cuda()) value_error("the tensors must be CUDA tensors");
    if (c10::cuda::current_device() != device.index()) value_error("the current CUDA device must be the tensors' device");
    return c10::cuda::getCurrentCUDAStream(device.index());
  }
  c10::Device device_;
  c10::cuda::CUDAStream current_, run_;
  bool other_ = false;
};

PyObject* one(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* two(const at::Tensor& a, const at::Tensor& b) {
  PyObject* r = PyTuple_New(2);
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b));
  return r;
}
PyObject* status(qmm_status rc) { return PyLong_FromLong(rc); }

// (x, format, bits, group, values, codes, scales, stream) -> (codes, scales)
PyObject* quantize_mx(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const int format = narrow(integer(a[1]));
  const int64_t bits = integer(a[2]), g = integer(a[3]);
  const at::Tensor* const values = maybe(a[4]);
  if (x.dim() != 2 || (x.scalar_type() != at::kFloat && x.scalar_type() != at::kBFloat16))
    type_error("x must be a bfloat16 or float32 matrix");
  const int64_t R = x.size(0), K = x.size(1), ld = R > 1 ? x.stride(0) : K;
  if (K % 32 != 0) value_error("K must be a multiple of 32");
  if ((K > 1 && x.stride(1) != 1) || ld < K) value_error("the elements of a row of x must be contiguous, and its rows apart");
  if (values != nullptr && !is(*values, at::kBFloat16, x.sizes()))
    value_error("values must be a contiguous bfloat16 tensor of x's shape");
  Call call(x, a[7]);
  call.here(values);
  const int64_t words[2] = {R, K * bits / 32}, groups[2] = {R, K / g};
  at::Tensor codes, scales;
  if (a[5] == Py_None) {
    codes = call.empty(words, at::kInt);
    scales = call.empty(groups, at::kByte);
  } else {
    codes = tensor(a[5]);
    scales = tensor(a[6]);
    call.here(&codes);
    call.here(&scales);
    if (!is(codes, at::kInt, words) || !is(scales, at::kByte, groups))
      value_error("out must be contiguous (int32 [R, K*bits/32], uint8 [R, K/g])");
  }
  const qmm_status rc =
      qmm_quantize_mx(x.data_ptr(), x.scalar_type() == at::kFloat ? QMM_OUT_F32 : QMM_OUT_BF16, R, K, ld, format,
                      static_cast<uint32_t*>(codes.data_ptr()), static_cast<uint8_t*>(scales.data_ptr()),
                      const_cast<void*>(ptr(values)), call.stream());
  return rc == QMM_OK ? two(codes, scales) : status(rc);
}

// (xq, x_scales, wq, w_scales, format, group, out, fp32, stream) -> out
PyObject* matmul_mx(PyObject* const* a) {
  const at::Tensor &xq = tensor(a[0]), &xs = tensor(a[1]), &wq = tensor(a[2]), &ws = tensor(a[3]);
  const int64_t g = integer(a[5]);
  const at::Tensor* const given = maybe(a[6]);
  const at::ScalarType dtype = PyObject_IsTrue(a[7]) ? at::kFloat : at::kBFloat16;
  if (xq.dim() != 2 || wq.dim() != 2) value_error("codes must be matrices");
  const int64_t M = xq.size(0), words = xq.size(1), N = wq.size(0), K = words * 8;
  if (!is(xq, at::kInt, {M, words}) || !is(wq, at::kInt, {N, words}))
    value_error("xq and wq must be contiguous int32 [M, K/8] and [N, K/8]");
  if (!is(xs, at::kByte, {M, K / g}) || !is(ws, at::kByte, {N, K / g}))
    value_error("x_scales and w_scales must be contiguous uint8 [M, K/g] and [N, K/g]");
  Call call(xq, a[8]);
  call.here(&xs);
  call.here(&wq);
  call.here(&ws);
  call.here(given);
  if (given != nullptr && !is(*given, dtype, {M, N})) value_error("out must be a contiguous [M, N] tensor of out_dtype");
  const at::Tensor out = given != nullptr ? *given : call.empty({M, N}, dtype);
  const qmm_status rc = qmm_matmul_mx(static_cast<const uint32_t*>(xq.data_ptr()), static_cast<const uint8_t*>(xs.data_ptr()),
                                      static_cast<const uint32_t*>(wq.data_ptr()), static_cast<const uint8_t*>(ws.data_ptr()),
                                      narrow(M), narrow(N), narrow(K), narrow(integer(a[4])), out.data_ptr(),
                                      dtype == at::kFloat ? QMM_OUT_F32 : QMM_OUT_BF16, call.stream());
  return rc == QMM_OK ? one(out) : status(rc);
}

// A cache from (k_cache, v_cache, block_table, lengths, q_lens, k_scale, v_scale) for B sequences.
qmm_paged_cache paged_cache(const Call& call, PyObject* const* a, int64_t B, const at::Tensor** q_lens) {
  const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]), &table = tensor(a[2]), &lengths = tensor(a[3]);
  *q_lens = maybe(a[4]);
  call.here(&k);
  call.here(&v);
  call.here(&table);
  call.here(&lengths);
  call.here(*q_lens);
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
    value_error("k_cache and v_cache must be [pages, page_size, heads, D] of one shape and dtype");
  const bool bf16 = k.scalar_type() == at::kBFloat16;
  if (!bf16 && k.scalar_type() != at::kFloat8_e4m3fn) type_error("the cache must be bfloat16 or float8_e4m3fn");
  if (k.stride(3) != 1 || v.stride(3) != 1) value_error("the D elements of a head must be contiguous");
  if (table.dim() != 2 || table.size(0) != B || table.scalar_type() != at::kInt || (table.size(1) > 1 && table.stride(1) != 1))
    value_error("block_table must be int32 [B, max_pages] with contiguous rows");
  if (!is(lengths, at::kInt, {B})) value_error("lengths must be contiguous int32 [B]");
  if (*q_lens != nullptr && !is(**q_lens, at::kInt, {B})) value_error("q_lens must be contiguous int32 [B]");
  qmm_paged_cache c = {};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.k_page = k.stride(0), c.k_token = k.stride(1), c.k_head = k.stride(2);
  c.v_page = v.stride(0), c.v_token = v.stride(1), c.v_head = v.stride(2);
  c.block_table = static_cast<const int32_t*>(table.data_ptr());
  c.lengths = static_cast<const int32_t*>(lengths.data_ptr());
  c.table_stride = B > 1 ? table.stride(0) : table.size(1);
  c.num_pages = k.size(0);
  c.max_pages = narrow(table.size(1));
  c.page_size = narrow(k.size(1));
  c.heads = narrow(k.size(2));
  c.head_dim = narrow(k.size(3));
  c.dtype = bf16 ? QMM_KV_BF16 : QMM_KV_E4M3;
  c.k_scale = static_cast<float>(real(a[5]));
  c.v_scale = static_cast<float>(real(a[6]));
  return c;
}

// Distance of the [B, M] rows of t [B, M, heads, D]: one for all; a row's elements are contiguous.
int64_t row_distance(const at::Tensor& t) {
  if (t.scalar_type() != at::kBFloat16) type_error("queries and new keys and values must be bfloat16");
  const int64_t B = t.size(0), M = t.size(1), heads = t.size(2), D = t.size(3);
  const int64_t ld = M > 1 ? t.stride(1) : B > 1 ? t.stride(0) : heads * D;
  if ((D > 1 && t.stride(3) != 1) || (heads > 1 && t.stride(2) != D) || (B > 1 && M > 1 && t.stride(0) != M * ld))
    value_error("the heads of a row must be contiguous and its rows evenly apart");
  return ld;
}

// (k_new, v_new, k_cache, v_cache, block_table, lengths, q_lens, k_scale, v_scale, stream) -> None
PyObject* kv_append(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]);
  if (k.dim() != 4 || k.sizes() != v.sizes()) value_error("k_new and v_new must be [B, M, heads, D] of one shape");
  Call call(k, a[9]);
  call.here(&v);
  const at::Tensor* q_lens;
  const qmm_paged_cache c = paged_cache(call, a + 2, k.size(0), &q_lens);
  if (k.size(2) != c.heads || k.size(3) != c.head_dim) value_error("k_new and the cache must have the same heads and D");
  const qmm_status rc = qmm_kv_append(&c, k.data_ptr(), row_distance(k), v.data_ptr(), row_distance(v), narrow(k.size(0)),
                                      narrow(k.size(1)), static_cast<const int32_t*>(ptr(q_lens)), call.stream());
  if (rc != QMM_OK) return status(rc);
  Py_RETURN_NONE;
}

// (q, k_cache, v_cache, block_table, lengths, q_lens, k_scale, v_scale, scale, window, sinks, out, return_lse,
//  workspace, stream) -> out or (out, lse)
PyObject* paged_attention(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0]);
  if (q.dim() != 4) value_error("q must be [B, M, q_heads, D]");
  const int64_t B = q.size(0), M = q.size(1), Hq = q.size(2), D = q.size(3);
  Call call(q, a[14]);
  const at::Tensor* q_lens;
  const qmm_paged_cache c = paged_cache(call, a + 1, B, &q_lens);
  if (D != c.head_dim) value_error("q and the cache must have the same D");
  const int64_t ld = row_distance(q);
  const at::Tensor *const given = maybe(a[11]), *const space = maybe(a[13]);
  call.here(given);
  call.here(space);
  if (given != nullptr && !is(*given, at::kBFloat16, q.sizes())) value_error("out must be a contiguous bfloat16 tensor of q's shape");
  if (space != nullptr && (space->scalar_type() != at::kByte || !space->is_contiguous()))
    value_error("workspace must be a contiguous uint8 tensor");
  const at::Tensor out = given != nullptr ? *given : call.empty(q.sizes(), at::kBFloat16);
  at::Tensor lse;
  const bool with_lse = PyObject_IsTrue(a[12]);
  if (with_lse) lse = call.empty({B, M, Hq}, at::kFloat);
  const int b = narrow(B), m = narrow(M), hq = narrow(Hq);
  const at::Tensor ws = space != nullptr
                            ? *space
                            : call.empty({static_cast<int64_t>(qmm_paged_attention_workspace(b, m, hq, c.heads, c.head_dim))}, at::kByte);
  const float scale = a[8] == Py_None ? 1.f / std::sqrt(static_cast<float>(D)) : static_cast<float>(real(a[8]));
  const int64_t window = integer(a[9]), sinks = integer(a[10]);
  const auto clip = [](int64_t v) { return static_cast<int>(v > 0x7fffffff ? 0x7fffffff : v < -1 ? -1 : v); };
  const qmm_status rc = qmm_paged_attention(&c, q.data_ptr(), ld, b, m, hq, static_cast<const int32_t*>(ptr(q_lens)), scale,
                                            clip(window), clip(sinks), out.data_ptr(),
                                            with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, ws.data_ptr(), ws.numel(),
                                            call.stream());
  if (rc != QMM_OK) return status(rc);
  return with_lse ? two(out, lse) : one(out);
}

// (logits, draft_tokens, draft_probs, uniform, noise, temperature, draft_lens, stream) -> (tokens, accepted)
PyObject* verify_draft(PyObject* const* a) {
  const at::Tensor& logits = tensor(a[0]);
  if (logits.dim() != 3 || logits.size(1) < 1 || logits.size(2) < 1) value_error("logits must be [B, k+1, V]");
  const bool f32 = logits.scalar_type() == at::kFloat;
  if (!f32 && logits.scalar_type() != at::kBFloat16) type_error("logits must be bfloat16 or float32");
  const int64_t B = logits.size(0), rows = logits.size(1), V = logits.size(2), k = rows - 1;
  if (V > 1 && logits.stride(2) != 1) value_error("the elements of a row of logits must be contiguous");
  const at::Tensor &draft = tensor(a[1]), &uniform = tensor(a[3]), &noise = tensor(a[4]), &temperature = tensor(a[5]);
  const at::Tensor *const probs = maybe(a[2]), *const lens = maybe(a[6]);
  if (!is(draft, at::kInt, {B, k}) || !is(uniform, at::kFloat, {B, k}))
    value_error("draft_tokens and uniform must be contiguous int32 and float32 [B, k]");
  if (!is(noise, at::kFloat, {B, V}) || !is(temperature, at::kFloat, {B}))
    value_error("noise and temperature must be contiguous float32 [B, V] and [B]");
  if (probs != nullptr && !is(*probs, at::kFloat, {B, k, V})) value_error("draft_probs must be contiguous float32 [B, k, V]");
  if (lens != nullptr && !is(*lens, at::kInt, {B})) value_error("draft_lens must be contiguous int32 [B]");
  Call call(logits, a[7]);
  for (const at::Tensor* t : {&draft, &uniform, &noise, &temperature, probs, lens}) call.here(t);
  const at::Tensor tokens = call.empty({B, rows}, at::kInt), accepted = call.empty({B}, at::kInt);
  const qmm_status rc = qmm_verify_draft(
      logits.data_ptr(), f32 ? QMM_OUT_F32 : QMM_OUT_BF16, B > 1 ? logits.stride(0) : rows * V, rows > 1 ? logits.stride(1) : V,
      static_cast<const int32_t*>(draft.data_ptr()), static_cast<const float*>(ptr(probs)),
      static_cast<const float*>(uniform.data_ptr()), static_cast<const float*>(noise.data_ptr()),
      static_cast<const float*>(temperature.data_ptr()), static_cast<const int32_t*>(ptr(lens)), narrow(B), narrow(k), narrow(V),
      static_cast<int32_t*>(tokens.data_ptr()), static_cast<int32_t*>(accepted.data_ptr()), call.stream());
  return rc == QMM_OK ? two(tokens, accepted) : status(rc);
}

// Argument count and exceptions of a function above.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed", N);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    if (r.type != nullptr) PyErr_SetString(r.type, r.message);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(quantize_mx, 8),       ENTRY(matmul_mx, 9),    ENTRY(kv_append, 10),
                         ENTRY(paged_attention, 15),  ENTRY(verify_draft, 8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmm_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_torch() { return PyModule_Create(&module); }
