// marshal.cpp -- argument marshalling of the serving-step calls for Python.
//
// A step calls several small operators whose kernels run for a few
// microseconds each, so reading a dozen tensors through Python attributes
// (some 20 us a call on the GPU hosts' cores) would cost more than the work.
// This module takes the torch tensors themselves: it checks devices, types,
// shapes and strides, and passes addresses, sizes and the stream to the C ABI
// of libpa.so.  It computes nothing.
//
// Every function returns the call's pa_status_t; a check that fails raises
// the package's PaError (PA_ERR_INVALID_ARG with the reason).  C++ exceptions
// do not leave it.
#include <Python.h>

#include <exception>
#include <initializer_list>
#include <string>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pa.h"

namespace {

PyObject* g_error = nullptr;  // the package's PaError

struct Refused : std::exception {
  std::string why;
  int status;
  explicit Refused(std::string w, int s = PA_ERR_INVALID_ARG) : why(std::move(w)), status(s) {}
  const char* what() const noexcept override { return why.c_str(); }
};

void require(bool ok, const char* why) {
  if (!ok) throw Refused(why);
}

// The arguments of one call, taken in order.
struct Args {
  PyObject* const* at;
  Py_ssize_t n, i = 0;
  PyObject* next() {
    if (i >= n) throw Refused("too few arguments");
    return at[i++];
  }
  const at::Tensor& tensor(const char* name) {
    const at::Tensor* t = maybe(name);
    if (!t) throw Refused(std::string(name) + " must be a tensor");
    return *t;
  }
  const at::Tensor* maybe(const char* name) {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
  }
  int32_t i32(const char* name) {
    const long long v = PyLong_AsLongLong(next());
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused(std::string(name) + " must be an integer");
    }
    if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " is out of range");
    return static_cast<int32_t>(v);
  }
  float f32(const char* name) {
    const double v = PyFloat_AsDouble(next());
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused(std::string(name) + " must be a number");
    }
    return static_cast<float>(v);
  }
  bool flag() {
    const int v = PyObject_IsTrue(next());
    if (v < 0) {
      PyErr_Clear();
      throw Refused("a flag must be true or false");
    }
    return v == 1;
  }
  // a stream handle, or None for the current stream of the tensors' device
  cudaStream_t stream(const at::Tensor& first) {
    require(first.is_cuda() && first.device().index() == c10::cuda::current_device(),
            "the tensors must be on the current CUDA device");
    PyObject* o = next();
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(first.device().index()).stream();
    void* s = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused("stream must be a CUDA stream");
    }
    return static_cast<cudaStream_t>(s);
  }
};

template <typename P = void>
P* addr(const at::Tensor* t) {
  return t ? static_cast<P*>(t->data_ptr()) : nullptr;
}
template <typename P = void>
P* addr(const at::Tensor& t) {
  return static_cast<P*>(t.data_ptr());
}

pa_dtype_t dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return PA_F32;
    case at::kBFloat16: return PA_BF16;
    case at::kHalf: return PA_F16;
    default: throw Refused("dtype must be float32, bfloat16 or float16", PA_ERR_UNSUPPORTED);
  }
}

struct Named {
  const char* name;
  const at::Tensor* t;
};

// Every tensor given is on `first`'s device and contiguous.
void same_device(const at::Tensor& first, std::initializer_list<Named> ts) {
  for (const Named& x : ts) {
    if (!x.t) continue;
    if (x.t->device() != first.device())
      throw Refused(std::string(x.name) + " must be on the device of the other tensors");
    if (!x.t->is_contiguous()) throw Refused(std::string(x.name) + " must be contiguous");
  }
}

void are_int32(std::initializer_list<Named> ts) {
  for (const Named& x : ts)
    if (x.t && x.t->scalar_type() != at::kInt)
      throw Refused(std::string(x.name) + " must be int32");
}

int32_t dim32(int64_t v) {
  if (v > INT32_MAX) throw Refused("a tensor's extent passes 32 bits", PA_ERR_UNSUPPORTED);
  return static_cast<int32_t>(v);
}

bool is(const at::Tensor& t, std::initializer_list<int64_t> shape) {
  return t.sizes() == c10::IntArrayRef(shape.begin(), shape.size());
}

struct Cache {
  int32_t blocks, heads, block_size, dim;
};

// Shapes of a pair of caches in the standard or the split-x layout.
Cache caches(const at::Tensor& k, const at::Tensor& v, bool split_x) {
  Cache c;
  if (split_x) {
    require(k.dim() == 5, "split-x k_cache must be 5-D");
    require(k.size(4) * k.element_size() == 16, "split-x key groups are 16 bytes");
    c = {dim32(k.size(0)), dim32(k.size(1)), dim32(k.size(3)), dim32(k.size(2) * k.size(4))};
    require(is(v, {c.blocks, c.heads, c.dim, c.block_size}), "v_cache must match k_cache");
  } else {
    require(k.dim() == 4, "k_cache must be 4-D");
    c = {dim32(k.size(0)), dim32(k.size(1)), dim32(k.size(2)), dim32(k.size(3))};
    require(v.sizes() == k.sizes(), "v_cache must match k_cache");
  }
  require(v.scalar_type() == k.scalar_type(), "the caches must share one dtype");
  return c;
}

void status_word(const at::Tensor* status) {
  if (status)
    require(status->scalar_type() == at::kInt && status->numel() >= 1, "status must be int32");
}

// ---- the calls ----------------------------------------------------------------

int plan_step(Args& in) {
  const at::Tensor& ctx = in.tensor("ctx_lens");
  const at::Tensor& fresh = in.tensor("new_lens");
  const at::Tensor& free = in.tensor("free_blocks");
  const at::Tensor& count = in.tensor("free_count");
  const at::Tensor& tables = in.tensor("block_tables");
  const at::Tensor& start = in.tensor("query_start");
  const at::Tensor& lens = in.tensor("seq_lens");
  const at::Tensor& pos = in.tensor("positions");
  const at::Tensor& slots = in.tensor("slots");
  const at::Tensor& left = in.tensor("free_left");
  pa_plan_params_t p{};
  p.block_size = in.i32("block_size");
  p.num_blocks = in.i32("num_blocks");
  const at::Tensor* base = in.maybe("base_len");
  const at::Tensor* status = in.maybe("status");
  cudaStream_t stream = in.stream(ctx);
  same_device(ctx, {{"ctx_lens", &ctx}, {"new_lens", &fresh}, {"free_blocks", &free},
                    {"free_count", &count}, {"block_tables", &tables}, {"query_start", &start},
                    {"seq_lens", &lens}, {"positions", &pos}, {"slots", &slots},
                    {"free_left", &left}, {"base_len", base}, {"status", status}});
  are_int32({{"ctx_lens", &ctx}, {"new_lens", &fresh}, {"free_blocks", &free},
             {"free_count", &count}, {"block_tables", &tables}, {"query_start", &start},
             {"seq_lens", &lens}, {"positions", &pos}, {"free_left", &left}, {"base_len", base}});
  status_word(status);
  require(slots.scalar_type() == at::kLong, "slots must be int64");
  require(ctx.dim() == 1, "ctx_lens must be [B]");
  const int64_t B = ctx.size(0);
  require(is(fresh, {B}) && is(lens, {B}) && is(start, {B + 1}),
          "lengths must be [B] and query_start [B + 1]");
  require(tables.dim() == 2 && tables.size(0) == B, "block_tables must be [B, ..]");
  require(free.dim() == 1 && count.numel() == 1 && left.numel() == 1,
          "free_blocks must be 1-D, free_count and free_left one element");
  require(!base || base->numel() == 1, "base_len must be one element");
  require(slots.dim() == 1 && pos.sizes() == slots.sizes(), "positions and slots must be [T]");
  p.num_seqs = dim32(B);
  p.max_blocks_per_seq = dim32(tables.size(1));
  p.max_tokens = dim32(slots.size(0));
  p.max_free = dim32(free.size(0));
  return pa_plan_step(&p, addr<int32_t>(ctx), addr<int32_t>(fresh), addr<int32_t>(free),
                      addr<int32_t>(count), addr<int32_t>(base), addr<int32_t>(tables),
                      addr<int32_t>(start), addr<int32_t>(lens), addr<int32_t>(pos),
                      addr<int64_t>(slots), addr<int32_t>(left), addr<int32_t>(status), stream);
}

int qk_norm_rope(Args& in) {
  const at::Tensor& q = in.tensor("q");
  const at::Tensor& k = in.tensor("k");
  const at::Tensor& v = in.tensor("v");
  const at::Tensor* pos = in.maybe("positions");
  const at::Tensor& slots = in.tensor("slots");
  const at::Tensor* cos_sin = in.maybe("cos_sin");
  const at::Tensor& q_out = in.tensor("q_out");
  const at::Tensor* k_cache = in.maybe("k_cache");
  const at::Tensor* v_cache = in.maybe("v_cache");
  const at::Tensor* qw = in.maybe("q_weight");
  const at::Tensor* kw = in.maybe("k_weight");
  pa_rope_params_t p{};
  p.eps = in.f32("eps");
  p.weight_offset = in.f32("weight_offset");
  const bool interleaved = in.flag();
  p.block_size = in.i32("block_size");
  p.num_blocks = in.i32("num_blocks");
  const at::Tensor* k_out = in.maybe("k_out");
  const at::Tensor* v_out = in.maybe("v_out");
  const bool split_x = in.flag();
  const at::Tensor* status = in.maybe("status");
  cudaStream_t stream = in.stream(q);
  require(q.dim() == 3 && k.dim() == 3, "q must be [T, Hq, D] and k, v [T, Hkv, D]");
  const int64_t T = q.size(0), hq = q.size(1), d = q.size(2), hkv = k.size(1);
  for (const at::Tensor* t : {&k, &v}) {
    require(t->device() == q.device(), "q, k and v must be on one device");
    require(is(*t, {T, hkv, d}), "q must be [T, Hq, D] and k, v [T, Hkv, D]");
  }
  for (const at::Tensor* t : {&q, &k, &v})
    require((t->stride(2) == 1 || d == 1) && (t->stride(1) == d || t->size(1) == 1),
            "heads must be contiguous within a row");
  same_device(q, {{"positions", pos}, {"slots", &slots}, {"cos_sin", cos_sin}, {"q_out", &q_out},
                  {"k_cache", k_cache}, {"v_cache", v_cache}, {"q_weight", qw}, {"k_weight", kw},
                  {"k_out", k_out}, {"v_out", v_out}, {"status", status}});
  status_word(status);
  const at::ScalarType dt = q.scalar_type();
  for (const at::Tensor* t : {&k, &v, &q_out, k_cache, v_cache, qw, kw, k_out, v_out})
    require(!t || t->scalar_type() == dt,
            "q, k, v, weights, caches and outputs must share one dtype");
  require(q_out.sizes() == q.sizes(), "q_out must be [T, Hq, D]");
  require(slots.scalar_type() == at::kLong && is(slots, {T}), "slots must be int64 [T]");
  require(!pos || (pos->scalar_type() == at::kInt && is(*pos, {T})), "positions must be int32 [T]");
  require(!qw == !kw, "give both weights or neither");
  for (const at::Tensor* t : {qw, kw}) require(!t || is(*t, {d}), "weights must be [D]");
  for (const at::Tensor* t : {k_out, v_out})
    require(!t || t->sizes() == k.sizes(), "k_out and v_out must be [T, Hkv, D]");
  if (cos_sin) {
    require(cos_sin->scalar_type() == at::kFloat && cos_sin->dim() == 2 && pos,
            "cos_sin must be float32 [max_position, rotary_dim], with positions");
    p.max_position = dim32(cos_sin->size(0));
    p.rotary_dim = dim32(cos_sin->size(1));
  }
  require(!k_cache == !v_cache, "give both caches or neither");
  if (k_cache) {
    const Cache c = caches(*k_cache, *v_cache, split_x);
    require(c.heads == hkv && c.dim == d, "the caches' heads and head_dim must be k's");
    p.block_size = c.block_size;
    p.num_blocks = c.blocks;
  } else {  // not used without caches
    if (p.block_size == 0) p.block_size = 1;
    if (p.num_blocks == 0) p.num_blocks = 1;
  }
  p.num_tokens = dim32(T);
  p.num_heads = dim32(hq);
  p.num_kv_heads = dim32(hkv);
  p.head_dim = dim32(d);
  p.q_stride = q.stride(0);
  p.k_stride = k.stride(0);
  p.v_stride = v.stride(0);
  p.dtype = dtype_code(q);
  p.flags = (interleaved ? PA_ROPE_INTERLEAVED : 0) | (split_x ? PA_FLAG_SPLIT_X : 0);
  return pa_qk_norm_rope(&p, addr(q), addr(k), addr(v), addr(qw), addr(kw), addr<float>(cos_sin),
                         addr<int32_t>(pos), addr<int64_t>(slots), addr(q_out), addr(k_out),
                         addr(v_out), addr(k_cache), addr(v_cache), addr<int32_t>(status), stream);
}

// q, k_cache, v_cache, block_tables, seq_lens, out, workspace of a decode step,
// checked, and its parameters.
struct Step {
  const at::Tensor *q, *kc, *vc, *bt, *sl, *out, *ws;
  pa_params_t p;
};

void read_step(Args& in, Step& s) {
  s.q = &in.tensor("q");
  s.kc = &in.tensor("k_cache");
  s.vc = &in.tensor("v_cache");
  s.bt = &in.tensor("block_tables");
  s.sl = &in.tensor("seq_lens");
  s.out = &in.tensor("out");
  s.ws = &in.tensor("workspace");
  s.p = pa_params_t{};
  s.p.max_seq_len = in.i32("max_seq_len");
  s.p.scale = in.f32("scale");
  s.p.partition_size = in.i32("partition_size");
  s.p.flags = in.i32("flags");
  same_device(*s.q, {{"q", s.q}, {"k_cache", s.kc}, {"v_cache", s.vc}, {"block_tables", s.bt},
                     {"seq_lens", s.sl}, {"out", s.out}, {"workspace", s.ws}});
  are_int32({{"block_tables", s.bt}, {"seq_lens", s.sl}});
  const Cache c = caches(*s.kc, *s.vc, (s.p.flags & PA_FLAG_SPLIT_X) != 0);
  require(s.q->dim() == 3 && s.q->size(2) == c.dim, "q must be [B, Hq, D] with k_cache's head_dim");
  require(s.q->scalar_type() == s.kc->scalar_type(), "q and the caches must share one dtype");
  require(s.out->sizes() == s.q->sizes(), "out must have q's shape");
  const int64_t B = s.q->size(0);
  require(s.bt->dim() == 2 && s.bt->size(0) == B && is(*s.sl, {B}),
          "block_tables must be [B, ..] and seq_lens [B]");
  s.p.num_seqs = dim32(B);
  s.p.num_heads = dim32(s.q->size(1));
  s.p.num_kv_heads = c.heads;
  s.p.head_dim = c.dim;
  s.p.block_size = c.block_size;
  s.p.num_blocks = c.blocks;
  s.p.max_blocks_per_seq = dim32(s.bt->size(1));
  s.p.kv_dtype = dtype_code(*s.kc);
  s.p.out_dtype = dtype_code(*s.out);
}

int decode_window(Args& in) {
  Step s;
  read_step(in, s);
  pa_window_t w{in.i32("window"), in.i32("num_sinks")};
  cudaStream_t stream = in.stream(*s.q);
  return pa_decode_window(&s.p, &w, addr(*s.q), addr(*s.kc), addr(*s.vc), addr<int32_t>(*s.bt),
                          addr<int32_t>(*s.sl), addr(*s.ws), s.ws->nbytes(), addr(*s.out), stream);
}

int decode_prefix(Args& in) {
  Step s;
  read_step(in, s);
  const at::Tensor& blocks = in.tensor("prefix_blocks");
  const at::Tensor& len = in.tensor("prefix_len");
  pa_prefix_t x{in.i32("max_prefix_len"), 0};
  cudaStream_t stream = in.stream(*s.q);
  same_device(*s.q, {{"prefix_blocks", &blocks}, {"prefix_len", &len}});
  are_int32({{"prefix_blocks", &blocks}, {"prefix_len", &len}});
  require(blocks.dim() == 1 && len.numel() == 1,
          "prefix_blocks must be 1-D and prefix_len one element");
  x.max_prefix_blocks = dim32(blocks.size(0));
  return pa_decode_prefix(&s.p, &x, addr(*s.q), addr(*s.kc), addr(*s.vc), addr<int32_t>(blocks),
                          addr<int32_t>(len), addr<int32_t>(*s.bt), addr<int32_t>(*s.sl),
                          addr(*s.ws), s.ws->nbytes(), addr(*s.out), stream);
}

int prefill_window(Args& in) {
  const at::Tensor& q = in.tensor("q");
  const at::Tensor& k = in.tensor("k");
  const at::Tensor& v = in.tensor("v");
  const at::Tensor& kc = in.tensor("k_cache");
  const at::Tensor& vc = in.tensor("v_cache");
  const at::Tensor& bt = in.tensor("block_tables");
  const at::Tensor& qs = in.tensor("query_start");
  const at::Tensor& cl = in.tensor("ctx_lens");
  const at::Tensor& out = in.tensor("out");
  pa_prefill_params_t p{};
  p.max_query_len = in.i32("max_query_len");
  p.max_ctx_len = in.i32("max_ctx_len");
  p.scale = in.f32("scale");
  p.flags = in.i32("flags");
  pa_window_t w{in.i32("window"), in.i32("num_sinks")};
  cudaStream_t stream = in.stream(q);
  same_device(q, {{"q", &q}, {"k", &k}, {"v", &v}, {"k_cache", &kc}, {"v_cache", &vc},
                  {"block_tables", &bt}, {"query_start", &qs}, {"ctx_lens", &cl}, {"out", &out}});
  are_int32({{"block_tables", &bt}, {"query_start", &qs}, {"ctx_lens", &cl}});
  const Cache c = caches(kc, vc, (p.flags & PA_FLAG_SPLIT_X) != 0);
  require(q.dim() == 3 && bt.dim() == 2, "q must be [T, Hq, D] and block_tables [B, ..]");
  const int64_t T = q.size(0), B = bt.size(0);
  require(q.size(2) == c.dim && is(k, {T, c.heads, c.dim}) && is(v, {T, c.heads, c.dim}) &&
              out.sizes() == q.sizes(),
          "prefill tensor shapes disagree");
  for (const at::Tensor* t : {&k, &v, &kc})
    require(t->scalar_type() == q.scalar_type(), "q, k, v and the caches must share one dtype");
  require(is(qs, {B + 1}) && is(cl, {B}), "query_start must be [B + 1] and ctx_lens [B]");
  p.num_seqs = dim32(B);
  p.num_heads = dim32(q.size(1));
  p.num_kv_heads = c.heads;
  p.head_dim = c.dim;
  p.block_size = c.block_size;
  p.num_blocks = c.blocks;
  p.max_blocks_per_seq = dim32(bt.size(1));
  p.total_tokens = dim32(T);
  p.kv_dtype = dtype_code(kc);
  p.out_dtype = dtype_code(out);
  return pa_prefill_window(&p, &w, addr(q), addr(k), addr(v), addr(kc), addr(vc),
                           addr<int32_t>(bt), addr<int32_t>(qs), addr<int32_t>(cl), addr(out),
                           stream);
}

// ---- the module -----------------------------------------------------------------

PyObject* refuse(int status, const char* why) {
  if (!g_error) {
    PyErr_SetString(PyExc_RuntimeError, why);
    return nullptr;
  }
  PyObject* e = PyObject_CallFunction(g_error, "is", status, why);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

template <int (*F)(Args&)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    Args in{args, n};
    return PyLong_FromLong(F(in));
  } catch (const Refused& r) {
    return refuse(r.status, r.what());
  } catch (const std::exception& e) {
    return refuse(PA_ERR_INVALID_ARG, e.what());
  }
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <int (*F)(Args&)>
constexpr PyCFunction fn() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F>));
}

PyMethodDef methods[] = {
    {"plan_step", fn<plan_step>(), METH_FASTCALL, nullptr},
    {"qk_norm_rope", fn<qk_norm_rope>(), METH_FASTCALL, nullptr},
    {"decode_window", fn<decode_window>(), METH_FASTCALL, nullptr},
    {"decode_prefix", fn<decode_prefix>(), METH_FASTCALL, nullptr},
    {"prefill_window", fn<prefill_window>(), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, "The exception class that refusals raise."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal",
                      "Marshalling of the serving-step calls of libpa.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// What this file was compiled against: the torch and Python whose layout of
// tensors it reads, and the compiler.
#ifndef PA_MARSHAL_STAMP
#error "PA_MARSHAL_STAMP: the build's description of torch, Python and compiler"
#endif

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", PA_MARSHAL_STAMP) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
