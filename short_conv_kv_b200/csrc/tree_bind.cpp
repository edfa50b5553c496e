// Argument marshalling of the drafted-tree and eviction calls: tensors in, one C
// ABI call out.  Decode steps make these calls once a layer, and the same checks in
// Python took 20 us a call, more than most of the kernels (here: 4 us).
//
// bind() takes the addresses of the C entry points, so that the module works
// with whichever library the Python side has loaded.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <optional>
#include <string>

#include "sconv_kv.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

[[noreturn]] void bad_type(const std::string& what) { throw py::type_error(what); }
[[noreturn]] void bad_value(const std::string& what) { throw py::value_error(what); }

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    case at::kFloat: return "float32";
    case at::kByte: return "uint8";
    default: return "bfloat16";
  }
}

int device_of(const Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

void on_device(const Tensor& t, const char* name, int dev) {
  if (device_of(t) != dev)
    bad_value(std::string(name) + " must be on " +
              (dev < 0 ? std::string("a CUDA device") : "device " + std::to_string(dev)));
}

void has_type(const Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type) bad_type(std::string(name) + " must be " + type_name(type));
}

// Pointer of a contiguous tensor.
template <typename T>
T* dense(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  has_type(t, name, type);
  if (t.sizes() != shape || !t.is_contiguous()) {
    std::string s = std::string(name) + " must be contiguous [";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    bad_value(s + "]");
  }
  on_device(t, name, dev);
  return static_cast<T*>(t.data_ptr());
}
template <typename T>
T* dense(const Maybe& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return t ? dense<T>(*t, name, type, shape, dev) : nullptr;
}

struct Seqs : sconv_kv_paged_t {};

Seqs paged(const Tensor& lens, const Tensor& table, int dev, const Tensor* cu = nullptr,
           const Tensor* parents = nullptr, int64_t tokens = 0, int max_draft = 0) {
  Seqs s = {};
  if (table.scalar_type() != at::kInt || table.dim() != 2 ||
      (table.size(1) > 1 && table.stride(1) != 1))
    bad_type("block_table must be int32 [num_seqs, pages] with unit page stride");
  on_device(table, "block_table", dev);
  const int64_t S = table.size(0), width = table.size(1);
  if (S > 1 && table.stride(0) < width) bad_value("block_table's rows must not overlap");
  if (S > INT32_MAX) bad_value("too many sequences");
  if (cu) {
    s.cu_draft = dense<int32_t>(*cu, "cu_draft", at::kInt, {S + 1}, dev);
    s.parents = dense<int32_t>(*parents, "parents", at::kInt, {tokens}, dev);
  }
  s.num_tokens = tokens;
  s.num_seqs = static_cast<int32_t>(S);
  s.max_draft = max_draft;
  s.context_lens = dense<int32_t>(lens, "context_lens", at::kInt, {S}, dev);
  s.block_table = static_cast<const int32_t*>(table.data_ptr());
  s.table_width = width;
  s.table_stride = S > 1 ? table.stride(0) : width;
  return s;
}

// The caches of a call: bf16 K and V, or MXFP8 codes with their scales; V may be absent.
struct Cache {
  sconv_kv_cache_layout_t lay = {};
  void *k = nullptr, *v = nullptr;
  uint8_t *ks = nullptr, *vs = nullptr;
};

Cache caches(const Tensor& k, const Maybe& ks, const Maybe& v, const Maybe& vs, int dev) {
  Cache c;
  const bool mx = ks.has_value();
  const at::ScalarType type = mx ? at::kByte : at::kBFloat16;
  if (k.scalar_type() != type || (v && v->scalar_type() != type))
    bad_type(mx ? "MXFP8 code caches must be uint8" : "caches must be bfloat16");
  if (k.dim() != 4 || k.stride(3) != 1)
    bad_value("cache must be [num_pages, page_size, Hkv, D] with dim stride 1");
  if (v && (v->sizes() != k.sizes() || v->strides() != k.strides()))
    bad_value("K and V caches must have the same type, shape and strides");
  on_device(k, "the K cache", dev);
  if (v) on_device(*v, "the V cache", dev);
  for (const Maybe* s : {&ks, &vs}) {
    if (!*s) continue;
    const Tensor& t = **s;
    if (t.scalar_type() != at::kByte || t.dim() != 4 || t.size(0) != k.size(0) ||
        t.size(1) != k.size(1) || t.size(2) != k.size(2) || t.size(3) != k.size(3) / 32 ||
        t.stride(3) != 1 || t.stride(0) * 32 != k.stride(0) || t.stride(1) * 32 != k.stride(1) ||
        t.stride(2) * 32 != k.stride(2))
      bad_value("scale caches must be uint8 [num_pages, page_size, Hkv, D/32] with strides equal "
                "to the data strides / 32");
    on_device(t, "a scale cache", dev);
  }
  if (k.size(2) > INT32_MAX || k.size(3) > INT32_MAX) bad_value("cache too large");
  c.lay.num_pages = k.size(0);
  c.lay.page_size = k.size(1);
  c.lay.num_kv_heads = k.size(2);
  c.lay.head_dim = k.size(3);
  c.lay.stride_page = k.stride(0);
  c.lay.stride_slot = k.stride(1);
  c.lay.stride_head = k.stride(2);
  c.k = k.data_ptr();
  if (v) c.v = v->data_ptr();
  if (ks) c.ks = static_cast<uint8_t*>(ks->data_ptr());
  if (vs) c.vs = static_cast<uint8_t*>(vs->data_ptr());
  return c;
}

// Whether two of the n1 x n2 rows of `len` elements at i * s1 + j * s2 share an element.
bool rows_overlap(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t len) {
  if (n1 <= 0 || n2 <= 0 || len <= 0) return false;
  if (n2 == 1 || (n1 > 1 && s1 < s2)) {
    std::swap(n1, n2);
    std::swap(s1, s2);
  }
  // n2 = 1: a single row; else s2 is the smaller stride of those in use
  if (n2 > 1 && s2 < len) return true;
  for (int64_t i = 1; i < n1 && i * s1 < (n2 - 1) * s2 + len; ++i) {
    // from the last of the n2 rows that begins at or before this one, and to the next of them
    const int64_t off = i * s1 % s2;
    if (off < len || (off > s2 - len && i * s1 / s2 + 1 < n2)) return true;
  }
  return false;
}

// bf16 [T, Hq, D] with unit dim stride.
struct Heads {
  void* p;
  int64_t tok, head;
};
Heads heads(const Tensor& x, const char* name, int dev) {
  has_type(x, name, at::kBFloat16);
  if (x.dim() != 3 || x.stride(2) != 1)
    bad_value(std::string(name) + " must be [T, Hq, D] with unit dim stride");
  on_device(x, name, dev);
  const int64_t T = x.size(0), H = x.size(1), D = x.size(2);
  // a dimension of size 1 has a stride of its own making
  return {x.data_ptr(), T > 1 ? x.stride(0) : H * D, H > 1 ? x.stride(1) : D};
}

// Raw rows k and v: [T, Hkv, D] or [T, Hkv*D], channels contiguous.
int64_t raw_rows(const Tensor& k, const Tensor& v, int dev) {
  int64_t stride[2];
  int n = 0;
  for (const Tensor* t : {&k, &v}) {
    const char* name = n ? "v" : "k";
    has_type(*t, name, at::kBFloat16);
    int64_t C;
    if (t->dim() == 3) {
      if (t->stride(2) != 1 || (t->size(1) > 1 && t->stride(1) != t->size(2)))
        bad_value(std::string(name) + ": heads and head_dim must be contiguous");
      C = t->size(1) * t->size(2);
    } else {
      if (t->dim() != 2 || t->stride(1) != 1)
        bad_value(std::string(name) + " must be [T, Hkv, D] or [T, Hkv*D]");
      C = t->size(1);
    }
    on_device(*t, name, dev);
    if (t->size(0) > 1 && t->stride(0) < C) bad_value(std::string(name) + "'s rows must not overlap");
    stride[n++] = t->size(0) > 1 ? t->stride(0) : std::max(t->stride(0), C);
  }
  if (k.sizes() != v.sizes() || stride[0] != stride[1])
    bad_value("k and v must share shape and row stride");
  return stride[0];
}

// fp32 [S, Hkv, positions].
struct Weights {
  float* p = nullptr;
  int64_t positions = 0, seq = 0, head = 0;
};
Weights weight_rows(const Maybe& t, const char* name, int64_t S, int64_t H, int dev) {
  Weights w;
  if (!t) return w;
  has_type(*t, name, at::kFloat);
  if (t->dim() != 3 || t->size(0) != S || t->size(1) != H || (t->size(2) > 1 && t->stride(2) != 1))
    bad_value(std::string(name) + " must be [" + std::to_string(S) + ", " + std::to_string(H) +
              ", positions] with unit position stride");
  w.positions = t->size(2);
  if (rows_overlap(S, t->stride(0), H, t->stride(1), w.positions))
    bad_value(std::string(name) + "'s rows must not overlap");
  on_device(*t, name, dev);
  w.p = static_cast<float*>(t->data_ptr());
  w.seq = t->stride(0);
  w.head = t->stride(1);
  return w;
}

int* flag(const Maybe& err, int dev) { return dense<int>(err, "err_flag", at::kInt, {1}, dev); }

// The call itself, with the tensors' device current, on `stream` or the
// device's current one (-1).
template <typename F>
int call(int dev, int64_t stream, F fn) {
  if (dev < 0) bad_value("the tensors must be on a CUDA device");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  void* s = stream >= 0 ? reinterpret_cast<void*>(stream)
                        : static_cast<void*>(c10::cuda::getCurrentCUDAStream(dev).stream());
  const py::gil_scoped_release release;
  return fn(s);
}

// ------------------------------------------------------------ the entry points

#define SCONV_ENTRIES(X)                                                                       \
  X(sconv_kv_tree_step) X(sconv_kv_tree_step_mxfp8) X(sconv_kv_tree_attention)                 \
  X(sconv_kv_tree_attention_mxfp8) X(sconv_kv_attention_weights)                               \
  X(sconv_kv_attention_weights_mxfp8) X(sconv_kv_tree_accept) X(sconv_kv_tree_accept_mxfp8)    \
  X(sconv_kv_evict) X(sconv_kv_evict_mxfp8)

struct {
#define SCONV_FIELD(n) decltype(&::n) n;
  SCONV_ENTRIES(SCONV_FIELD)
#undef SCONV_FIELD
} lib;

void bind(const py::dict& at) {
#define SCONV_BIND(n) lib.n = reinterpret_cast<decltype(&::n)>(at[#n].cast<uintptr_t>());
  SCONV_ENTRIES(SCONV_BIND)
#undef SCONV_BIND
}

int tree_step(const Tensor& k, const Tensor& v, const Tensor& cu, const Tensor& parents,
              const Tensor& wk, const Tensor& wv, const Tensor& gk, const Tensor& gv, double eps,
              const Maybe& state, const Tensor& slots, const Tensor& kc, const Maybe& ks,
              const Tensor& vc, const Maybe& vs, const Maybe& state_indices, const Maybe& err,
              int64_t stream, const Maybe& state_positions) {
  const int dev = device_of(k);
  const int64_t rs = raw_rows(k, v, dev), T = k.size(0);
  const Cache c = caches(kc, ks, vc, vs, dev);
  if (cu.dim() != 1 || cu.size(0) < 1) bad_value("cu_draft must be [num_seqs + 1]");
  const int64_t S = cu.size(0) - 1, H = c.lay.num_kv_heads, D = c.lay.head_dim, C = H * D;
  if (k.numel() != T * C) bad_value("k's rows must have the cache's heads");
  if (wk.dim() != 2) bad_value("conv_w_k must be [W, Hkv*D]");
  const int64_t W = wk.size(0);
  const bool per_head = gk.dim() == 2;
  const int64_t g1[1] = {D}, g2[2] = {H, D};
  const at::IntArrayRef gs = per_head ? at::IntArrayRef(g2, 2) : at::IntArrayRef(g1, 1);
  const auto* cup = dense<int32_t>(cu, "cu_draft", at::kInt, {S + 1}, dev);
  const auto* par = dense<int32_t>(parents, "parents", at::kInt, {T}, dev);
  const void* wkp = dense<void>(wk, "conv_w_k", at::kBFloat16, {W, C}, dev);
  const void* wvp = dense<void>(wv, "conv_w_v", at::kBFloat16, {W, C}, dev);
  const auto* gkp = dense<float>(gk, "gamma_k", at::kFloat, gs, dev);
  const auto* gvp = dense<float>(gv, "gamma_v", at::kFloat, gs, dev);
  const auto* sl = dense<int64_t>(slots, "slot_mapping", at::kLong, {T}, dev);
  const void* st = nullptr;
  int64_t pool = 0;
  if (W > 1) {
    if (!state || state->dim() != 3) bad_value("conv_state must be [pool, W-1, 2*Hkv*D]");
    pool = state->size(0);
    st = dense<void>(*state, "conv_state", at::kBFloat16, {pool, W - 1, 2 * C}, dev);
  }
  const auto* si = dense<int32_t>(state_indices, "state_indices", at::kInt, {S}, dev);
  sconv_kv_options_t o = {};
  o.gamma_head_stride = per_head ? D : 0;
  o.state_positions = dense<int64_t>(state_positions, "state_positions", at::kLong, {S}, dev);
  const sconv_kv_options_t* opt = per_head || state_positions ? &o : nullptr;
  int* e = flag(err, dev);
  const int iS = static_cast<int>(S), iW = static_cast<int>(std::min<int64_t>(W, INT32_MAX));
  const int iH = static_cast<int>(H), iD = static_cast<int>(D);
  const void *kp = k.data_ptr(), *vp = v.data_ptr();
  return call(dev, stream, [&](void* s) {
    const float f = static_cast<float>(eps);
    return ks ? lib.sconv_kv_tree_step_mxfp8(kp, vp, rs, T, cup, par, iS, wkp, wvp, gkp, gvp, f, iW,
                                             iH, iD, st, si, pool, sl, c.k, c.ks, c.v, c.vs, &c.lay,
                                             opt, e, s)
              : lib.sconv_kv_tree_step(kp, vp, rs, T, cup, par, iS, wkp, wvp, gkp, gvp, f, iW, iH,
                                       iD, st, si, pool, sl, c.k, c.v, &c.lay, opt, e, s);
  });
}

// 1: all is well, but there is no workspace.
int tree_attention(const Tensor& q, const Tensor& cu, const Tensor& parents, const Tensor& lens,
                   const Tensor& table, const Tensor& kc, const Maybe& ks, const Tensor& vc,
                   const Maybe& vs, double scale, int max_draft, const Tensor& out,
                   const Maybe& lse, const Maybe& workspace, const Maybe& err, int64_t stream) {
  const int dev = device_of(q);
  const Cache c = caches(kc, ks, vc, vs, dev);
  const Heads hq = heads(q, "q", dev);
  const int64_t T = q.size(0), HQ = q.size(1), D = q.size(2);
  if (D != c.lay.head_dim) bad_value("q and the cache differ in head_dim");
  if (out.sizes() != q.sizes()) bad_value("out must have q's shape");
  const Heads ho = heads(out, "out", dev);
  if (rows_overlap(T, ho.tok, HQ, ho.head, D)) bad_value("out's rows must not overlap");
  auto* l = dense<float>(lse, "lse", at::kFloat, {T, HQ}, dev);
  const Seqs seqs = paged(lens, table, dev, &cu, &parents, T, max_draft);
  int* e = flag(err, dev);
  if (!workspace) {
    if (dev < 0) bad_value("the tensors must be on a CUDA device");
    return 1;
  }
  void* ws = dense<void>(*workspace, "workspace", at::kByte, {workspace->numel()}, dev);
  const int64_t bytes = workspace->numel();
  const int iq = static_cast<int>(HQ), ih = static_cast<int>(c.lay.num_kv_heads);
  const int id = static_cast<int>(D);
  return call(dev, stream, [&](void* s) {
    const float f = static_cast<float>(scale);
    return ks ? lib.sconv_kv_tree_attention_mxfp8(hq.p, hq.tok, hq.head, iq, ih, id, f, &seqs, c.k,
                                                  c.ks, c.v, c.vs, &c.lay, ho.p, ho.tok, ho.head, l,
                                                  ws, bytes, e, s)
              : lib.sconv_kv_tree_attention(hq.p, hq.tok, hq.head, iq, ih, id, f, &seqs, c.k, c.v,
                                            &c.lay, ho.p, ho.tok, ho.head, l, ws, bytes, e, s);
  });
}

int attention_weights(const Tensor& q, const Tensor& lse, const Tensor& cu, const Tensor& parents,
                      const Tensor& lens, const Tensor& table, const Tensor& kc, const Maybe& ks,
                      double scale, int max_draft, const Tensor& weights, const Maybe& err,
                      int64_t stream) {
  const int dev = device_of(q);
  const Cache c = caches(kc, ks, std::nullopt, std::nullopt, dev);
  const Heads hq = heads(q, "q", dev);
  const int64_t T = q.size(0), HQ = q.size(1), D = q.size(2);
  if (D != c.lay.head_dim) bad_value("q and the cache differ in head_dim");
  const auto* l = dense<float>(lse, "lse", at::kFloat, {T, HQ}, dev);
  const Seqs seqs = paged(lens, table, dev, &cu, &parents, T, max_draft);
  const Weights w = weight_rows(weights, "weights", seqs.num_seqs, c.lay.num_kv_heads, dev);
  int* e = flag(err, dev);
  const int iq = static_cast<int>(HQ), ih = static_cast<int>(c.lay.num_kv_heads);
  const int id = static_cast<int>(D);
  return call(dev, stream, [&](void* s) {
    const float f = static_cast<float>(scale);
    return ks ? lib.sconv_kv_attention_weights_mxfp8(hq.p, hq.tok, hq.head, iq, ih, id, f, l, &seqs,
                                                     c.k, c.ks, &c.lay, w.p, w.positions, w.seq,
                                                     w.head, e, s)
              : lib.sconv_kv_attention_weights(hq.p, hq.tok, hq.head, iq, ih, id, f, l, &seqs, c.k,
                                               &c.lay, w.p, w.positions, w.seq, w.head, e, s);
  });
}

int tree_accept(const Tensor& k, const Tensor& v, const Tensor& cu, const Tensor& parents,
                const Tensor& leaves, const Tensor& lens, const Tensor& table, int W,
                const Maybe& state, const Tensor& kc, const Maybe& ks, const Tensor& vc,
                const Maybe& vs, const Tensor& new_lens, const Maybe& weights,
                const Maybe& state_indices, const Maybe& state_positions, const Maybe& err,
                int64_t stream) {
  const int dev = device_of(k);
  const int64_t rs = raw_rows(k, v, dev);
  const Cache c = caches(kc, ks, vc, vs, dev);
  const int64_t H = c.lay.num_kv_heads, D = c.lay.head_dim;
  if (k.numel() != k.size(0) * H * D) bad_value("k's rows must have the cache's heads");
  const Seqs seqs = paged(lens, table, dev, &cu, &parents, k.size(0), SCONV_KV_MAX_DRAFT);
  const int64_t S = seqs.num_seqs;
  const auto* lv = dense<int32_t>(leaves, "leaves", at::kInt, {S}, dev);
  auto* nl = dense<int32_t>(new_lens, "new_lens", at::kInt, {S}, dev);
  const auto* si = dense<int32_t>(state_indices, "state_indices", at::kInt, {S}, dev);
  const auto* sp = dense<int64_t>(state_positions, "state_positions", at::kLong, {S}, dev);
  void* st = nullptr;
  int64_t pool = 0;
  if (W != 1) {
    if (!state || state->dim() != 3) bad_value("conv_state must be [pool, W-1, 2*Hkv*D]");
    pool = state->size(0);
    st = dense<void>(*state, "conv_state", at::kBFloat16, {pool, W - 1, 2 * H * D}, dev);
  }
  const Weights w = weight_rows(weights, "weights", S, H, dev);
  int* e = flag(err, dev);
  const int ih = static_cast<int>(H), id = static_cast<int>(D);
  const void *kp = k.data_ptr(), *vp = v.data_ptr();
  return call(dev, stream, [&](void* s) {
    return ks ? lib.sconv_kv_tree_accept_mxfp8(kp, vp, rs, &seqs, lv, W, ih, id, st, si, pool, sp,
                                               c.k, c.ks, c.v, c.vs, &c.lay, w.p, w.positions,
                                               w.seq, w.head, nl, e, s)
              : lib.sconv_kv_tree_accept(kp, vp, rs, &seqs, lv, W, ih, id, st, si, pool, sp, c.k,
                                         c.v, &c.lay, w.p, w.positions, w.seq, w.head, nl, e, s);
  });
}

int evict(const Tensor& weights, const Tensor& lens, const Tensor& table, const Tensor& kc,
          const Maybe& ks, const Tensor& vc, const Maybe& vs, int sinks, int recent,
          const Tensor& kept, const Tensor& new_lens, const Maybe& weights_out, const Maybe& err,
          int64_t stream) {
  const int dev = device_of(weights);
  const Cache c = caches(kc, ks, vc, vs, dev);
  const Seqs seqs = paged(lens, table, dev);
  const int64_t S = seqs.num_seqs, H = c.lay.num_kv_heads;
  if (kept.dim() != 3) bad_value("kept must be [num_seqs, Hkv, keep]");
  const int64_t keep = kept.size(2);
  auto* kp = dense<int32_t>(kept, "kept", at::kInt, {S, H, keep}, dev);
  auto* nl = dense<int32_t>(new_lens, "new_lens", at::kInt, {S}, dev);
  const Weights w = weight_rows(weights, "weights", S, H, dev);
  const Weights wo = weight_rows(weights_out, "weights_out", S, H, dev);
  int* e = flag(err, dev);
  const int ik = static_cast<int>(std::min<int64_t>(keep, INT32_MAX));
  const int ih = static_cast<int>(H), id = static_cast<int>(c.lay.head_dim);
  return call(dev, stream, [&](void* s) {
    return ks ? lib.sconv_kv_evict_mxfp8(w.p, w.positions, w.seq, w.head, &seqs, ik, sinks, recent,
                                         ih, id, c.k, c.ks, c.v, c.vs, &c.lay, kp, nl, wo.p,
                                         wo.positions, wo.seq, wo.head, e, s)
              : lib.sconv_kv_evict(w.p, w.positions, w.seq, w.head, &seqs, ik, sinks, recent, ih,
                                   id, c.k, c.v, &c.lay, kp, nl, wo.p, wo.positions, wo.seq,
                                   wo.head, e, s);
  });
}

}  // namespace

PYBIND11_MODULE(_tree, m) {
  m.doc() = "Argument marshalling of the drafted-tree and eviction calls (see binding.py).";
  m.def("bind", &bind);
  m.def("tree_step", &tree_step);
  m.def("tree_attention", &tree_attention);
  m.def("attention_weights", &attention_weights);
  m.def("tree_accept", &tree_accept);
  m.def("evict", &evict);
}
