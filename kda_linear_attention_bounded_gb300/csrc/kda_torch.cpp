// Argument checks and marshalling of the calls beside the KDA layers, for torch tensors: what a call costs on the host
// is a few C++ accessors a tensor instead of as many Python attributes (a decode call 12 us before, see the Python
// wrappers for the interface).  The C entry points' addresses are handed over once (bind), so that the library is the one
// the package has loaded.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <exception>
#include <string>
#include <vector>

#include "kda.h"

namespace {

decltype(&kda_gdn_chunk_prefill) g_prefill = nullptr;
decltype(&kda_gdn_recurrent_verify) g_verify = nullptr;
decltype(&kda_gdn_decode) g_decode = nullptr;
decltype(&kda_paged_attention) g_paged = nullptr;
decltype(&kda_step_tables) g_tables = nullptr;
decltype(&kda_rotary_to_pages) g_rotary = nullptr;
decltype(&kda_fork_requests) g_fork = nullptr;
decltype(&kda_release_requests) g_release = nullptr;
decltype(&kda_compact_pages) g_compact = nullptr;
decltype(&kda_copy_pages) g_copy = nullptr;
decltype(&kda_shared_prefix_attention) g_prefix = nullptr;

constexpr int64_t kD = 128;

struct Refused {};   // a Python error is set

[[noreturn]] void refuse(const std::string &what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused{};
}
std::string n(int64_t x) { return std::to_string(x); }

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a tensor", name);
    throw Refused{};
  }
  const at::Tensor &t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided) refuse(std::string(name) + ": expected a strided tensor");
  return t;
}
int cuda_device(const at::Tensor &t, const char *name) {
  if (!t.is_cuda()) refuse(std::string(name) + ": expected a CUDA tensor");
  return t.get_device();
}
bool on(const at::Tensor &t, int dev) { return t.is_cuda() && t.get_device() == dev; }

int64_t integer(PyObject *o, const char *name) {
  PyObject *i = PyNumber_Index(o);   // (whole numbers alone: not 2.9, not "16")
  if (!i) {
    PyErr_Format(PyExc_TypeError, "%s: expected a whole number", name);
    throw Refused{};
  }
  const int64_t x = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (x == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + ": out of range");
  }
  return x;
}
int int32(PyObject *o, const char *name) {
  const int64_t x = integer(o, name);
  if (x < INT_MIN || x > INT_MAX) refuse(std::string(name) + ": out of range");
  return static_cast<int>(x);
}
int int32(int64_t x, const char *name) {
  if (x < INT_MIN || x > INT_MAX) refuse(std::string(name) + ": out of range");
  return static_cast<int>(x);
}
float scale_of(PyObject *o) {
  if (o == Py_None) return 0.08838834764831845f;   // 128^-1/2
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused{};
  return static_cast<float>(x);
}

// A contiguous tensor of this type, device and shape.
void *exact(PyObject *o, const char *name, at::ScalarType type, int dev, at::IntArrayRef shape) {
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != type || !on(t, dev) || t.sizes() != shape || !t.is_contiguous()) {
    std::string want, got;
    for (int64_t s : shape) want += (want.empty() ? "" : ", ") + n(s);
    for (int64_t s : t.sizes()) got += (got.empty() ? "" : ", ") + n(s);
    refuse(std::string(name) + ": expected a contiguous " + c10::toString(type) + " tensor [" + want + "] on cuda:" + n(dev) +
           ", got " + c10::toString(t.scalar_type()) + " [" + got + "] on " + t.device().str());
  }
  return t.data_ptr();
}
struct Rows {
  uint16_t *at;
  int64_t stride;
};
// bf16 [tokens, H, 128] with contiguous heads, and its token stride
Rows rows3(PyObject *o, const char *name, int dev, int64_t tokens, int64_t H) {
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16 || !on(t, dev) || t.dim() != 3 || t.size(0) != tokens || t.size(1) != H ||
      t.size(2) != kD || t.stride(2) != 1 || (H > 1 && t.stride(1) != kD))
    refuse(std::string(name) + ": expected a bf16 tensor [" + n(tokens) + ", " + n(H) + ", 128] on cuda:" + n(dev) +
           " with contiguous heads");
  return {static_cast<uint16_t *>(t.data_ptr()), tokens > 1 ? t.stride(0) : H * kD};
}
// bf16 [tokens, H], heads contiguous
Rows rows2(PyObject *o, const char *name, int dev, int64_t tokens, int64_t H) {
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16 || !on(t, dev) || t.dim() != 2 || t.size(0) != tokens || t.size(1) != H ||
      (H > 1 && t.stride(1) != 1))
    refuse(std::string(name) + ": expected a bf16 tensor [" + n(tokens) + ", " + n(H) + "] on cuda:" + n(dev) + ", heads contiguous");
  return {static_cast<uint16_t *>(t.data_ptr()), tokens > 1 ? t.stride(0) : H};
}
struct Workspace {
  void *at;
  size_t bytes;
};
Workspace workspace_of(PyObject *o, int dev) {
  const at::Tensor &t = tensor(o, "workspace");
  if (t.scalar_type() != at::kByte || !on(t, dev) || !t.is_contiguous())
    refuse("workspace: expected a contiguous uint8 tensor on cuda:" + n(dev));
  return {t.data_ptr(), static_cast<size_t>(t.numel())};
}
struct Pool {
  float *at;
  int slots;
};
Pool pool_of(PyObject *o, int dev, int64_t Hv) {
  const at::Tensor &t = tensor(o, "state_pool");
  if (t.scalar_type() != at::kFloat || !on(t, dev) || t.dim() != 4 || t.size(1) != Hv || t.size(2) != kD || t.size(3) != kD ||
      !t.is_contiguous())
    refuse("state_pool: expected a contiguous fp32 tensor [slots, " + n(Hv) + ", 128, 128] on cuda:" + n(dev));
  return {static_cast<float *>(t.data_ptr()), int32(t.size(0), "state_pool")};
}
// The given raw stream (an integer), or the device's current one (None)
void *stream_of(PyObject *o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused{};
  return p;
}

struct GdnTokens {
  int dev;
  int64_t tokens;
  int Hk, Hv;
  Rows q, k, v, a, beta;
  const float *A_log, *dt_bias;
  float scale;
};
// arguments 0 .. 6: q, k, v, a, beta_logits, A_log, dt_bias; and the scale
GdnTokens gdn_tokens(PyObject *const *x, PyObject *scale) {
  GdnTokens g;
  const at::Tensor &q = tensor(x[0], "q");
  g.dev = cuda_device(q, "q");
  const at::Tensor &v = tensor(x[2], "v");
  if (q.dim() != 3 || v.dim() != 3) refuse("q, k, v: expected bf16 tensors [tokens, heads, 128]");
  g.tokens = q.size(0);
  g.Hk = int32(q.size(1), "q");
  g.Hv = int32(v.size(1), "v");
  if (g.Hk < 1 || g.Hv < 1 || g.Hv % g.Hk)
    refuse("v: " + n(g.Hv) + " value heads are not a multiple of q's and k's " + n(g.Hk));
  g.q = rows3(x[0], "q", g.dev, g.tokens, g.Hk);
  g.k = rows3(x[1], "k", g.dev, g.tokens, g.Hk);
  if (g.k.stride != g.q.stride) refuse("q and k must share one token stride");
  g.v = rows3(x[2], "v", g.dev, g.tokens, g.Hv);
  g.a = rows2(x[3], "a", g.dev, g.tokens, g.Hv);
  g.beta = rows2(x[4], "beta_logits", g.dev, g.tokens, g.Hv);
  g.A_log = static_cast<const float *>(exact(x[5], "A_log", at::kFloat, g.dev, {g.Hv}));
  g.dt_bias = static_cast<const float *>(exact(x[6], "dt_bias", at::kFloat, g.dev, {g.Hv}));
  g.scale = scale_of(scale);
  return g;
}
int64_t count_of(PyObject *o, const char *name) { return tensor(o, name).numel(); }

template <typename F>
PyObject *guarded(Py_ssize_t have, Py_ssize_t want, F body) {
  try {
    if (have != want) {
      PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
      return nullptr;
    }
    if (!g_prefix) {
      PyErr_SetString(PyExc_RuntimeError, "the library has not been bound");
      return nullptr;
    }
    return PyLong_FromLong(body());
  } catch (const Refused &) {
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
// The C call, with the device current and without the interpreter's lock (a full launch queue blocks).
template <typename F>
int call(int dev, F body) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = body();
  Py_END_ALLOW_THREADS
  return rc;
}

// q, k, v, a, beta_logits, A_log, dt_bias, scale, cu_seqlens, cu_seqlens_host, state_pool, slot_ids, flags, out,
// final_state, workspace, stream
PyObject *gdn_chunk_prefill(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 17, [&] {
    const GdnTokens g = gdn_tokens(x, x[7]);
    const at::Tensor &host = tensor(x[9], "cu_seqlens_host");
    if (host.is_cuda() || host.scalar_type() != at::kInt || host.dim() != 1 || host.numel() < 1 || !host.is_contiguous())
      refuse("cu_seqlens_host: expected host memory of [sequences + 1] entries");
    const int32_t *cu_host = static_cast<const int32_t *>(host.data_ptr());
    const int64_t N = host.numel() - 1;
    if (cu_host[N] > g.tokens)
      refuse("cu_seqlens_host: its last entry " + n(cu_host[N]) + " lies behind the " + n(g.tokens) + " tokens");
    const auto *cu = static_cast<const int32_t *>(exact(x[8], "cu_seqlens", at::kInt, g.dev, {N + 1}));
    const int flags = int32(x[12], "flags");
    Pool pool = {nullptr, 0};
    const int32_t *slots = nullptr;
    if (flags & (KDA_LOAD_INITIAL | KDA_FINAL_TO_POOL)) {
      if (x[10] == Py_None || x[11] == Py_None) refuse("load_initial and final_to_pool need state_pool and slot_ids");
      pool = pool_of(x[10], g.dev, g.Hv);
      slots = static_cast<const int32_t *>(exact(x[11], "slot_ids", at::kInt, g.dev, {N}));
    }
    const Rows out = rows3(x[13], "out", g.dev, g.tokens, g.Hv);
    float *final = flags & KDA_FINAL_TO_POOL
                       ? nullptr
                       : static_cast<float *>(exact(x[14], "final_state", at::kFloat, g.dev, {N, g.Hv, kD, kD}));
    const Workspace ws = workspace_of(x[15], g.dev);
    void *stream = stream_of(x[16], g.dev);
    const int num_seqs = int32(N, "cu_seqlens_host");
    return call(g.dev, [&] {
      return g_prefill(g.q.at, g.k.at, g.q.stride, g.v.at, g.v.stride, g.a.at, g.a.stride, g.beta.at, g.beta.stride, g.A_log,
                       g.dt_bias, g.scale, cu, cu_host, num_seqs, g.Hk, g.Hv, pool.at, pool.slots, slots, flags, out.at,
                       out.stride, final, ws.at, ws.bytes, stream);
    });
  });
}

// q, k, v, a, beta_logits, A_log, dt_bias, scale, state_pool, slot_ids, T, out, intermediate_states, workspace, stream
PyObject *gdn_recurrent_verify(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 15, [&] {
    const int T = int32(x[10], "T");
    const GdnTokens g = gdn_tokens(x, x[7]);
    const int64_t B = count_of(x[9], "slot_ids");
    if (g.tokens != B * T) refuse("q: " + n(g.tokens) + " tokens for " + n(B) + " requests x " + n(T));
    const Pool pool = pool_of(x[8], g.dev, g.Hv);
    const auto *slots = static_cast<const int32_t *>(exact(x[9], "slot_ids", at::kInt, g.dev, {B}));
    const Rows out = rows3(x[11], "out", g.dev, g.tokens, g.Hv);
    auto *inter = static_cast<float *>(exact(x[12], "intermediate_states", at::kFloat, g.dev, {B, T, g.Hv, kD, kD}));
    const Workspace ws = workspace_of(x[13], g.dev);
    void *stream = stream_of(x[14], g.dev);
    const int requests = int32(B, "slot_ids");
    return call(g.dev, [&] {
      return g_verify(g.q.at, g.k.at, g.q.stride, g.v.at, g.v.stride, g.a.at, g.a.stride, g.beta.at, g.beta.stride, g.A_log,
                      g.dt_bias, g.scale, requests, T, g.Hk, g.Hv, pool.at, pool.slots, slots, out.at, out.stride, inter, ws.at,
                      ws.bytes, stream);
    });
  });
}

// q, k, v, a, beta_logits, A_log, dt_bias, scale, state_pool, slot_ids, out, workspace, stream
PyObject *gdn_decode(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 13, [&] {
    const GdnTokens g = gdn_tokens(x, x[7]);
    const Pool pool = pool_of(x[8], g.dev, g.Hv);
    const auto *slots = static_cast<const int32_t *>(exact(x[9], "slot_ids", at::kInt, g.dev, {g.tokens}));
    const Rows out = rows3(x[10], "out", g.dev, g.tokens, g.Hv);
    const Workspace ws = workspace_of(x[11], g.dev);
    void *stream = stream_of(x[12], g.dev);
    const int requests = int32(g.tokens, "q");
    return call(g.dev, [&] {
      return g_decode(g.q.at, g.k.at, g.q.stride, g.v.at, g.v.stride, g.a.at, g.a.stride, g.beta.at, g.beta.stride, g.A_log,
                      g.dt_bias, g.scale, requests, g.Hk, g.Hv, pool.at, pool.slots, slots, out.at, out.stride, ws.at, ws.bytes,
                      stream);
    });
  });
}

struct Pages {
  const uint16_t *at;
  int64_t stride[3];
};
Pages pages_of(const at::Tensor &t, const char *name, int dev) {
  if (t.scalar_type() != at::kBFloat16 || !on(t, dev) || t.dim() != 4 || t.size(3) != kD || t.stride(3) != 1)
    refuse(std::string(name) + ": expected a bf16 tensor [pages, page_size, Hk, 128] on cuda:" + n(dev) + ", channels contiguous");
  Pages p;
  p.at = static_cast<const uint16_t *>(t.data_ptr());
  for (int i = 0; i < 3; ++i) p.stride[i] = t.size(i) == 1 ? 0 : t.stride(i);
  return p;
}
struct Table {
  int32_t *at;
  int64_t stride;
  int requests, width;
};
Table table_of(const at::Tensor &t, int dev) {
  if (t.scalar_type() != at::kInt || !on(t, dev) || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    refuse("block_table: expected an int32 tensor [requests, width] on cuda:" + n(dev) + " with contiguous rows");
  const Table b = {static_cast<int32_t *>(t.data_ptr()), t.size(0) > 1 ? t.stride(0) : t.size(1), int32(t.size(0), "block_table"),
                   int32(t.size(1), "block_table")};
  if (b.stride < b.width) refuse("block_table: its rows overlap");
  return b;
}

// The tensors of an attention over pages: q, k_pages, v_pages, block_table, seq_lens, then T, scale, out, lse
struct PagedCall {
  int dev, T, num_pages, page, Hq, Hk, requests;
  float scale;
  Rows q, out;
  Pages k, v;
  Table table;
  const int32_t *lens;
  float *lse;
};
PagedCall paged_call(PyObject *const *x, PyObject *T, PyObject *scale, PyObject *out, PyObject *lse) {
  PagedCall c;
  c.T = int32(T, "T");
  c.scale = scale_of(scale);
  const at::Tensor &q = tensor(x[0], "q");
  c.dev = cuda_device(q, "q");
  const int64_t B = count_of(x[4], "seq_lens");
  if (q.dim() != 3) refuse("q: expected a bf16 tensor [B*T, Hq, 128]");
  const int64_t Hq = q.size(1);
  c.q = rows3(x[0], "q", c.dev, B * c.T, Hq);
  const at::Tensor &kt = tensor(x[1], "k_pages"), &vt = tensor(x[2], "v_pages");
  c.k = pages_of(kt, "k_pages", c.dev);
  c.v = pages_of(vt, "v_pages", c.dev);
  if (kt.sizes() != vt.sizes()) refuse("k_pages and v_pages must have one shape");
  c.table = table_of(tensor(x[3], "block_table"), c.dev);
  if (c.table.requests != B) refuse("block_table: " + n(c.table.requests) + " rows for " + n(B) + " requests");
  c.lens = static_cast<const int32_t *>(exact(x[4], "seq_lens", at::kInt, c.dev, {B}));
  c.out = rows3(out, "out", c.dev, B * c.T, Hq);
  c.lse = lse == Py_None ? nullptr : static_cast<float *>(exact(lse, "lse", at::kFloat, c.dev, {B * c.T, Hq}));
  c.num_pages = int32(kt.size(0), "k_pages");
  c.page = int32(kt.size(1), "k_pages");
  c.Hk = int32(kt.size(2), "k_pages");
  c.Hq = int32(Hq, "q");
  c.requests = int32(B, "seq_lens");
  return c;
}

// q, k_pages, v_pages, block_table, seq_lens, T, scale, out, lse, workspace, stream
PyObject *paged_attention(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 11, [&] {
    const PagedCall c = paged_call(x, x[5], x[6], x[7], x[8]);
    const Workspace ws = workspace_of(x[9], c.dev);
    void *stream = stream_of(x[10], c.dev);
    return call(c.dev, [&] {
      return g_paged(c.q.at, c.q.stride, c.k.at, c.k.stride[0], c.k.stride[1], c.k.stride[2], c.v.at, c.v.stride[0],
                     c.v.stride[1], c.v.stride[2], c.num_pages, c.page, c.table.at, c.table.stride, c.table.width, c.lens,
                     c.requests, c.T, c.Hq, c.Hk, c.scale, c.out.at, c.out.stride, c.lse, ws.at, ws.bytes, stream);
    });
  });
}

// q, k_pages, v_pages, block_table, seq_lens, prefix_lens, group_starts, T, scale, out, lse, workspace, stream
PyObject *shared_prefix_attention(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 13, [&] {
    const PagedCall c = paged_call(x, x[7], x[8], x[9], x[10]);
    const int64_t G = count_of(x[5], "prefix_lens");
    const auto *prefix = static_cast<const int32_t *>(exact(x[5], "prefix_lens", at::kInt, c.dev, {G}));
    const auto *starts = static_cast<const int32_t *>(exact(x[6], "group_starts", at::kInt, c.dev, {G + 1}));
    const Workspace ws = workspace_of(x[11], c.dev);
    void *stream = stream_of(x[12], c.dev);
    const int groups = int32(G, "prefix_lens");
    return call(c.dev, [&] {
      return g_prefix(c.q.at, c.q.stride, c.k.at, c.k.stride[0], c.k.stride[1], c.k.stride[2], c.v.at, c.v.stride[0],
                      c.v.stride[1], c.v.stride[2], c.num_pages, c.page, c.table.at, c.table.stride, c.table.width, c.lens,
                      c.requests, c.T, prefix, starts, groups, c.Hq, c.Hk, c.scale, c.out.at, c.out.stride, c.lse, ws.at,
                      ws.bytes, stream);
    });
  });
}

// q, k, v, positions, slot_map, inv_freq, k_pages, v_pages, axes, interleaved, mscale, out, workspace, stream
PyObject *rotary_to_pages(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 14, [&] {
    const int interleaved = int32(x[9], "interleaved");
    const double mscale = PyFloat_AsDouble(x[10]);
    if (mscale == -1.0 && PyErr_Occurred()) throw Refused{};
    const at::Tensor &q = tensor(x[0], "q"), &kt = tensor(x[6], "k_pages"), &vt = tensor(x[7], "v_pages"),
                     &pos = tensor(x[3], "positions");
    const int dev = cuda_device(q, "q");
    if (q.dim() != 3) refuse("q: expected a bf16 tensor [tokens, Hq, 128]");
    const int64_t tokens = q.size(0), Hq = q.size(1), half = count_of(x[5], "inv_freq");
    const Pages kp = pages_of(kt, "k_pages", dev), vp = pages_of(vt, "v_pages", dev);
    if (kt.sizes() != vt.sizes()) refuse("k_pages and v_pages must have one shape");
    const int64_t Hk = kt.size(2);
    const Rows qr = rows3(x[0], "q", dev, tokens, Hq), kr = rows3(x[1], "k", dev, tokens, Hk), vr = rows3(x[2], "v", dev, tokens, Hk);
    if (pos.scalar_type() != at::kInt || !on(pos, dev) || pos.dim() < 1 || pos.dim() > 2 || pos.size(-1) != tokens ||
        (tokens > 1 && pos.stride(-1) != 1))
      refuse("positions: expected an int32 tensor [" + n(tokens) + "] or [axes, " + n(tokens) + "] on cuda:" + n(dev) +
             " with contiguous rows");
    const int64_t rows = pos.dim() == 2 ? pos.size(0) : 1, row_stride = rows > 1 ? pos.stride(0) : tokens;
    const auto *slots = static_cast<const int64_t *>(exact(x[4], "slot_map", at::kLong, dev, {tokens}));
    const auto *freq = static_cast<const float *>(exact(x[5], "inv_freq", at::kFloat, dev, {half}));
    const uint8_t *axes = nullptr;
    if (x[8] != Py_None) {
      if (!PyBytes_Check(x[8])) {
        PyErr_SetString(PyExc_TypeError, "axes: expected bytes");
        throw Refused{};
      }
      if (PyBytes_GET_SIZE(x[8]) != half)
        refuse("axes: expected one for each of the " + n(half) + " frequencies, got " + n(PyBytes_GET_SIZE(x[8])));
      axes = reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(x[8]));
    }
    const Rows out = rows3(x[11], "out", dev, tokens, Hq);
    const Workspace ws = workspace_of(x[12], dev);
    void *stream = stream_of(x[13], dev);
    const int count = int32(tokens, "q"), hq = int32(Hq, "q"), hk = int32(Hk, "k_pages"), num_axes = int32(rows, "positions"),
              R = int32(2 * half, "inv_freq"), num_pages = int32(kt.size(0), "k_pages"), page = int32(kt.size(1), "k_pages");
    return call(dev, [&] {
      return g_rotary(qr.at, qr.stride, kr.at, kr.stride, vr.at, vr.stride, count, hq, hk, static_cast<const int32_t *>(pos.data_ptr()),
                      row_stride, num_axes, slots, freq, R, axes, interleaved, static_cast<float>(mscale),
                      const_cast<uint16_t *>(kp.at), kp.stride[0], kp.stride[1], kp.stride[2], const_cast<uint16_t *>(vp.at),
                      vp.stride[0], vp.stride[1], vp.stride[2], num_pages, page, out.at, out.stride, ws.at, ws.bytes, stream);
    });
  });
}

// block_table, seq_lens, parents, children, free_pages, page_size, copy_src, copy_dst, pages_used, workspace, stream
PyObject *fork_requests(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 11, [&] {
    const int page = int32(x[5], "page_size");
    const at::Tensor &t = tensor(x[0], "block_table");
    const int dev = cuda_device(t, "block_table");
    const Table table = table_of(t, dev);
    auto ints = [&](int i, const char *name, int64_t count) {
      return static_cast<int32_t *>(exact(x[i], name, at::kInt, dev, {count}));
    };
    const int64_t forks = count_of(x[2], "parents"), free = count_of(x[4], "free_pages");
    int32_t *lens = ints(1, "seq_lens", table.requests), *parents = ints(2, "parents", forks), *children = ints(3, "children", forks),
            *pages = ints(4, "free_pages", free), *src = ints(6, "copy_src", forks), *dst = ints(7, "copy_dst", forks),
            *used = ints(8, "pages_used", 1);
    const Workspace ws = workspace_of(x[9], dev);
    void *stream = stream_of(x[10], dev);
    const int count = int32(forks, "parents"), num_free = int32(free, "free_pages");
    return call(dev, [&] {
      return g_fork(table.at, table.stride, table.width, lens, table.requests, parents, children, count, pages, num_free, page,
                    src, dst, used, ws.at, ws.bytes, stream);
    });
  });
}

// block_table, seq_lens, rows, page_size, free_pages, num_free, workspace, stream
PyObject *release_requests(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 8, [&] {
    const int page = int32(x[3], "page_size");
    const at::Tensor &t = tensor(x[0], "block_table");
    const int dev = cuda_device(t, "block_table");
    const Table table = table_of(t, dev);
    const int64_t rows = count_of(x[2], "rows"), pages = count_of(x[4], "free_pages");
    auto ints = [&](int i, const char *name, int64_t count) {
      return static_cast<int32_t *>(exact(x[i], name, at::kInt, dev, {count}));
    };
    int32_t *lens = ints(1, "seq_lens", table.requests), *ended = ints(2, "rows", rows), *list = ints(4, "free_pages", pages),
            *num = ints(5, "num_free", 1);
    const Workspace ws = workspace_of(x[6], dev);
    void *stream = stream_of(x[7], dev);
    const int num_rows = int32(rows, "rows"), num_pages = int32(pages, "free_pages");
    return call(dev, [&] {
      return g_release(table.at, table.stride, table.width, lens, table.requests, ended, num_rows, page, list, num_pages, num,
                       ws.at, ws.bytes, stream);
    });
  });
}

// block_table, seq_lens, page_size, new_table, copy_src, copy_dst, free_pages, num_free, workspace, stream
PyObject *compact_pages(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 10, [&] {
    const int page = int32(x[2], "page_size");
    const at::Tensor &t = tensor(x[0], "block_table"), &nt = tensor(x[3], "new_table");
    const int dev = cuda_device(t, "block_table");
    const Table table = table_of(t, dev);
    if (nt.sizes() != t.sizes()) refuse("block_table and new_table must have one shape");
    if (nt.scalar_type() != at::kInt || !on(nt, dev) || (nt.size(1) > 1 && nt.stride(1) != 1))
      refuse("new_table: expected an int32 tensor [requests, width] on cuda:" + n(dev) + " with contiguous rows");
    const int64_t new_stride = nt.size(0) > 1 ? nt.stride(0) : nt.size(1);
    if (new_stride < table.width) refuse("new_table: its rows overlap");
    const int64_t pages = count_of(x[6], "free_pages"), room = count_of(x[4], "copy_src");
    auto ints = [&](int i, const char *name, int64_t count) {
      return static_cast<int32_t *>(exact(x[i], name, at::kInt, dev, {count}));
    };
    if (room < pages / 2) refuse("copy_src: " + n(room) + " places for up to " + n(pages / 2) + " copies");
    int32_t *lens = ints(1, "seq_lens", table.requests), *src = ints(4, "copy_src", room), *dst = ints(5, "copy_dst", room),
            *list = ints(6, "free_pages", pages), *num = ints(7, "num_free", 1);
    const Workspace ws = workspace_of(x[8], dev);
    void *stream = stream_of(x[9], dev);
    const int num_pages = int32(pages, "free_pages"), places = int32(room, "copy_src");
    return call(dev, [&] {
      return g_compact(table.at, table.stride, table.width, lens, table.requests, page, num_pages,
                       static_cast<int32_t *>(nt.data_ptr()), new_stride, src, dst, places, list, num, ws.at, ws.bytes, stream);
    });
  });
}

// buffers (list or tuple), copy_src, copy_dst, workspace, stream
PyObject *copy_pages(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 5, [&] {
    if (!PyList_Check(x[0]) && !PyTuple_Check(x[0])) {
      PyErr_SetString(PyExc_TypeError, "buffers: expected a list or a tuple of tensors");
      throw Refused{};
    }
    const Py_ssize_t many = PySequence_Fast_GET_SIZE(x[0]);
    if (many < 1) refuse("buffers: expected at least one tensor");
    std::vector<kda_page_buffer> buffers(static_cast<size_t>(many));
    int dev = 0;
    int64_t pages = 0;
    for (Py_ssize_t i = 0; i < many; ++i) {
      const at::Tensor &t = tensor(PySequence_Fast_GET_ITEM(x[0], i), "buffers");
      if (i == 0) dev = cuda_device(t, "buffers");
      if (!on(t, dev) || t.dim() < 1) refuse("buffers: expected tensors [pages, ...] on cuda:" + n(dev));
      if (i == 0) pages = t.size(0);
      if (t.size(0) != pages) refuse("buffers: " + n(t.size(0)) + " pages beside " + n(pages));
      int64_t inner = 1;
      for (int64_t d = t.dim() - 1; d >= 1; --d) {
        if (t.size(d) > 1 && t.stride(d) != inner) refuse("buffers: a page has to be contiguous");
        inner *= t.size(d);
      }
      const int64_t bytes = inner * t.element_size();
      buffers[static_cast<size_t>(i)] = {t.data_ptr(), pages > 1 ? t.stride(0) * static_cast<int64_t>(t.element_size()) : bytes, bytes};
    }
    const int64_t count = count_of(x[1], "copy_src");
    const auto *src = static_cast<const int32_t *>(exact(x[1], "copy_src", at::kInt, dev, {count}));
    const auto *dst = static_cast<const int32_t *>(exact(x[2], "copy_dst", at::kInt, dev, {count}));
    const Workspace ws = workspace_of(x[3], dev);
    void *stream = stream_of(x[4], dev);
    const int num_pages = int32(pages, "buffers"), copies = int32(count, "copy_src"), num = int32(many, "buffers");
    return call(dev, [&] { return g_copy(buffers.data(), num, num_pages, src, dst, copies, ws.at, ws.bytes, stream); });
  });
}

// block_table, seq_lens, new_lens, free_pages, page_size, cu_seqlens, kv_lens, positions, slot_map, pages_used,
// workspace, stream
PyObject *step_tables(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  return guarded(argc, 12, [&] {
    const int page = int32(x[4], "page_size");
    const at::Tensor &t = tensor(x[0], "block_table");
    const int dev = cuda_device(t, "block_table");
    const Table table = table_of(t, dev);
    const int64_t B = table.requests, rows = count_of(x[8], "slot_map"), free = count_of(x[3], "free_pages");
    auto ints = [&](int i, const char *name, int64_t count) {
      return static_cast<int32_t *>(exact(x[i], name, at::kInt, dev, {count}));
    };
    int32_t *cu = ints(5, "cu_seqlens", B + 1), *kv = ints(6, "kv_lens", B), *pos = ints(7, "positions", rows);
    auto *map = static_cast<int64_t *>(exact(x[8], "slot_map", at::kLong, dev, {rows}));
    int32_t *used = ints(9, "pages_used", 1), *old = ints(1, "seq_lens", B), *fresh = ints(2, "new_lens", B),
            *pages = ints(3, "free_pages", free);
    const int num_free = int32(free, "free_pages");
    const Workspace ws = workspace_of(x[10], dev);
    void *stream = stream_of(x[11], dev);
    return call(dev, [&] {
      return g_tables(table.at, table.stride, table.width, old, fresh, table.requests, pages, num_free, page, rows, cu, kv, pos,
                      map, used, ws.at, ws.bytes, stream);
    });
  });
}

// bind(addresses of the C entry points, in the order below)
PyObject *bind(PyObject *, PyObject *const *x, Py_ssize_t argc) {
  constexpr int kCalls = 11;
  if (argc != kCalls) {
    PyErr_SetString(PyExc_TypeError, "bind: eleven addresses");
    return nullptr;
  }
  void *at[kCalls];
  for (int i = 0; i < kCalls; ++i) {
    at[i] = PyLong_AsVoidPtr(x[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
      return nullptr;
    }
  }
  g_prefill = reinterpret_cast<decltype(g_prefill)>(at[0]);
  g_verify = reinterpret_cast<decltype(g_verify)>(at[1]);
  g_decode = reinterpret_cast<decltype(g_decode)>(at[2]);
  g_paged = reinterpret_cast<decltype(g_paged)>(at[3]);
  g_tables = reinterpret_cast<decltype(g_tables)>(at[4]);
  g_rotary = reinterpret_cast<decltype(g_rotary)>(at[5]);
  g_fork = reinterpret_cast<decltype(g_fork)>(at[6]);
  g_release = reinterpret_cast<decltype(g_release)>(at[7]);
  g_compact = reinterpret_cast<decltype(g_compact)>(at[8]);
  g_copy = reinterpret_cast<decltype(g_copy)>(at[9]);
  g_prefix = reinterpret_cast<decltype(g_prefix)>(at[10]);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}
PyMethodDef methods[] = {{"bind", fast<bind>(), METH_FASTCALL, nullptr},
                         {"gdn_chunk_prefill", fast<gdn_chunk_prefill>(), METH_FASTCALL, nullptr},
                         {"gdn_recurrent_verify", fast<gdn_recurrent_verify>(), METH_FASTCALL, nullptr},
                         {"gdn_decode", fast<gdn_decode>(), METH_FASTCALL, nullptr},
                         {"paged_attention", fast<paged_attention>(), METH_FASTCALL, nullptr},
                         {"step_tables", fast<step_tables>(), METH_FASTCALL, nullptr},
                         {"rotary_to_pages", fast<rotary_to_pages>(), METH_FASTCALL, nullptr},
                         {"fork_requests", fast<fork_requests>(), METH_FASTCALL, nullptr},
                         {"release_requests", fast<release_requests>(), METH_FASTCALL, nullptr},
                         {"compact_pages", fast<compact_pages>(), METH_FASTCALL, nullptr},
                         {"copy_pages", fast<copy_pages>(), METH_FASTCALL, nullptr},
                         {"shared_prefix_attention", fast<shared_prefix_attention>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_torch() { return PyModule_Create(&module); }
