// C ABI of the drafted-tree operators and the eviction: argument checks, launch
// geometry and dispatch.  See include/sconv_kv.h for the contract.
//
// sconv_kv.cu, the entry points of the step itself, is part of this
// translation unit: both share its helpers (launch, argument checks, the caches
// of device properties and the text of the last CUDA error).
#include "sconv_kv.cu"

#include <math.h>

#include <algorithm>

#include "tree_instances.h"

namespace {

using sconv::AcceptParams;
using sconv::AttendParams;
using sconv::CacheParts;
using sconv::EvictParams;
using sconv::PagedSeqs;
using sconv::TreeStepParams;
using sconv::WeighParams;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

// launch() with the grid's x dimension in clusters of c CTAs.
int launch_clusters(const void* fn, dim3 grid, int c, int threads, size_t smem, void** args,
                    void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    snprintf(g_cuda_error, sizeof g_cuda_error, "%s: %s", cudaGetErrorName(e),
             cudaGetErrorString(e));
    return SCONV_KV_ERR_CUDA;
  }
  g_cuda_error[0] = '\0';
  return SCONV_KV_OK;
}

// Cache layout and paged sequences; the kernels keep a row's offset in 32
// bits, in units of 8 elements.
int check_paged(const sconv_kv_paged_t* seqs, const sconv_kv_cache_layout_t* layout, int H, int D,
                bool drafted, bool mx, int* err, PagedSeqs* Q) {
  if (H < 1 || H > (1 << 15) || !head_dim_ok(D)) return SCONV_KV_ERR_SHAPE;
  if (layout->num_kv_heads != H || layout->head_dim != D) return SCONV_KV_ERR_SHAPE;
  if (layout->num_pages < 1 || layout->num_pages > INT32_MAX || layout->page_size < 1 ||
      layout->page_size > INT32_MAX || layout->stride_head < D || layout->stride_slot < 1 ||
      layout->stride_page < 1)
    return SCONV_KV_ERR_SHAPE;
  const int unit = mx ? 32 : 8;
  if (layout->stride_head % unit || layout->stride_slot % unit || layout->stride_page % unit)
    return SCONV_KV_ERR_ALIGN;
  const __int128 last =
      static_cast<__int128>(layout->num_pages - 1) * layout->stride_page +
      static_cast<__int128>(layout->page_size - 1) * layout->stride_slot;
  if (last / 8 >= static_cast<__int128>(0xffffffffu)) return SCONV_KV_ERR_SHAPE;
  if (seqs->table_width < 1 || seqs->table_stride < seqs->table_width ||
      seqs->table_width > INT32_MAX || seqs->table_width * layout->page_size > INT32_MAX)
    return SCONV_KV_ERR_SHAPE;
  if (drafted && (seqs->max_draft < 1 || seqs->max_draft > SCONV_KV_MAX_DRAFT))
    return SCONV_KV_ERR_SHAPE;
  if (!seqs->context_lens || !seqs->block_table) return SCONV_KV_ERR_NULL;
  // (an empty tensor may have a NULL pointer)
  if (drafted && (!seqs->cu_draft || (!seqs->parents && seqs->num_tokens > 0)))
    return SCONV_KV_ERR_NULL;
  memset(Q, 0, sizeof *Q);
  if (drafted) {
    Q->cu = seqs->cu_draft;
    Q->parents = seqs->parents;
    Q->num_tokens = seqs->num_tokens;
    Q->max_draft = seqs->max_draft;
  }
  Q->lens = seqs->context_lens;
  Q->table = seqs->block_table;
  Q->table_stride = seqs->table_stride;
  // (kernels step up to 2^16 positions past the end)
  Q->capacity = std::min<int64_t>(seqs->table_width * layout->page_size, INT32_MAX - 65536);
  Q->num_seqs = seqs->num_seqs;
  Q->num_pages = static_cast<int>(layout->num_pages);
  Q->page_size = static_cast<int>(layout->page_size);
  // division by page_size (positions are below 2^31)
  const uint32_t d = static_cast<uint32_t>(layout->page_size);
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  Q->page_shift = l;
  Q->page_mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - d)) / d + 1);
  Q->stride_page = layout->stride_page;
  Q->stride_slot = layout->stride_slot;
  Q->stride_head = layout->stride_head;
  Q->page8 = static_cast<uint32_t>(layout->stride_page / 8);
  Q->slot8 = static_cast<uint32_t>(layout->stride_slot / 8);
  Q->err = err;
  return SCONV_KV_OK;
}

// An empty call (no sequence, or no drafted token) enqueues nothing.
int check_counts(const sconv_kv_paged_t* seqs, bool drafted, bool* empty) {
  if (!seqs) return SCONV_KV_ERR_NULL;
  if (seqs->num_seqs < 0 || (drafted && (seqs->num_tokens < 0 || seqs->num_tokens > INT32_MAX)))
    return SCONV_KV_ERR_SHAPE;
  *empty = seqs->num_seqs == 0 || (drafted && seqs->num_tokens == 0);
  return SCONV_KV_OK;
}

int check_cache(const void* k, const void* v, const void* ks, const void* vs, bool need_v,
                bool mx) {
  if (!k || (need_v && !v) || (mx && (!ks || (need_v && !vs)))) return SCONV_KV_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16)) return SCONV_KV_ERR_ALIGN;
  return SCONV_KV_OK;
}

CacheParts parts_of(const void* k, const void* v, const void* ks, const void* vs,
                    const sconv_kv_cache_layout_t* layout) {
  const int64_t row = layout->head_dim / 32;
  const bool packed = ks && aligned(ks, static_cast<size_t>(row)) &&
                      layout->stride_head / 32 % row == 0 && layout->stride_slot / 32 % row == 0 &&
                      layout->stride_page / 32 % row == 0;
  const bool words = layout->stride_slot / 32 % 4 == 0 && layout->stride_page / 32 % 4 == 0;
  auto raw = [](const void* p) { return const_cast<uint8_t*>(static_cast<const uint8_t*>(p)); };
  return {raw(k), raw(v), raw(ks), raw(vs), packed ? 1 : 0,
          packed && aligned(vs, static_cast<size_t>(row)) ? 1 : 0, words ? 1 : 0};
}

int check_heads(int HQ, int H, int64_t tok, int64_t head, int D) {
  if (H < 1 || HQ < H || HQ % H || HQ > sconv::kMaxQueryHeads) return SCONV_KV_ERR_SHAPE;
  if (head < D || tok < 1) return SCONV_KV_ERR_SHAPE;
  if (tok % 8 || head % 8) return SCONV_KV_ERR_ALIGN;
  return SCONV_KV_OK;
}

// How a call's attention is laid out: rows an M-tile, keys a tile, and the
// CTAs that share the tiles.  Up to 16 rows a K/V head (8 with D = 256, whose
// accumulators would not fit) go to attend_rows_kernel, more to
// attend_tc_kernel.
struct AttendPlan {
  const void* fn;
  int units;  // of attend_tc_kernel's ring; 0: attend_rows_kernel
  int rows;
  int tile;
  int threads;
  size_t smem;
  int mtiles;  // of a (sequence, K/V head)
  int parts;
};

int plan_attend(int num_seqs, int max_draft, int HQ, int H, int D, bool mx, AttendPlan* A) {
  const int rows = max_draft * (HQ / H);
  if (rows <= (D == 256 ? 8 : 16)) {
    const int nt = rows <= 8 ? 1 : 2;
    A->units = 0;
    A->rows = 8 * nt;
    A->tile = sconv::kRowsTile;
    A->threads = 32 * sconv::kRowsWarps;
    A->smem = sconv::attend_rows_smem(D, nt);
    A->fn = reinterpret_cast<const void*>(sconv::pick_attend_rows(D, nt, mx));
    if (!A->fn) return SCONV_KV_ERR_UNSUPPORTED;
  } else {
    const sconv::AttendTc t = sconv::pick_attend_tc(D, mx, rows);
    A->units = t.units;
    A->rows = t.rows;
    A->tile = t.tile;
    A->threads = t.threads;
    A->smem = t.smem;
    A->fn = reinterpret_cast<const void*>(t.fn);
  }
  A->mtiles = (rows + A->rows - 1) / A->rows;
  if (static_cast<int64_t>(num_seqs) * A->mtiles > INT32_MAX) return SCONV_KV_ERR_SHAPE;  // the join's grid
  if (!smem_attr_set(A->fn, A->smem)) return SCONV_KV_ERR_CUDA;
  A->parts = sm_count() * (A->units ? 1 : resident_per_sm(A->fn, A->threads, A->smem, 2));
  return SCONV_KV_OK;
}

// Workspace: prefix, then partial (m, l), then partial o.
int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }
int64_t workspace_need(int num_seqs, int D, int parts, int rows) {
  return round256(8 * (static_cast<int64_t>(num_seqs) + 2)) +
         round256(2ll * parts * rows * 8) + round256(2ll * parts * rows * D * 4);
}

int attention_impl(const void* q, int64_t q_tok, int64_t q_head, int HQ, int H, int D, float scale,
                   const sconv_kv_paged_t* seqs, const void* k, const uint8_t* ks, const void* v,
                   const uint8_t* vs, const sconv_kv_cache_layout_t* layout, void* out,
                   int64_t o_tok, int64_t o_head, float* lse, void* workspace,
                   int64_t workspace_bytes, int* err, void* stream, bool mx) {
  bool empty = false;
  int rc = check_counts(seqs, true, &empty);
  if (rc != SCONV_KV_OK || empty) return rc;
  if (!q || !out || !workspace || !layout) return SCONV_KV_ERR_NULL;
  rc = check_cache(k, v, ks, vs, true, mx);
  if (rc != SCONV_KV_OK) return rc;
  AttendParams P;
  memset(&P, 0, sizeof P);
  rc = check_paged(seqs, layout, H, D, true, mx, err, &P.s);
  if (rc == SCONV_KV_OK) rc = check_heads(HQ, H, q_tok, q_head, D);
  if (rc == SCONV_KV_OK) rc = check_heads(HQ, H, o_tok, o_head, D);
  if (rc != SCONV_KV_OK) return rc;
  if (!isfinite(scale)) return SCONV_KV_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4))
    return SCONV_KV_ERR_ALIGN;
  AttendPlan A;
  rc = plan_attend(seqs->num_seqs, seqs->max_draft, HQ, H, D, mx, &A);
  if (rc != SCONV_KV_OK) return rc;
  if (workspace_bytes < workspace_need(seqs->num_seqs, D, A.parts, A.rows))
    return SCONV_KV_ERR_SCRATCH;
  P.c = parts_of(k, v, ks, vs, layout);
  P.q = static_cast<const uint16_t*>(q);
  P.q_tok = q_tok;
  P.q_head = q_head;
  P.out = static_cast<uint16_t*>(out);
  P.o_tok = o_tok;
  P.o_head = o_head;
  P.lse = lse;
  P.HQ = HQ;
  P.H = H;
  P.g = HQ / H;
  P.scale_log2 = scale * sconv::kLog2e;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  P.prefix = reinterpret_cast<int64_t*>(w);
  w += round256(8 * (static_cast<int64_t>(seqs->num_seqs) + 2));
  P.part_ml = reinterpret_cast<float2*>(w);
  w += round256(2ll * A.parts * A.rows * 8);
  P.part_o = reinterpret_cast<float*>(w);
  P.parts = A.parts;
  {
    void* args[] = {&P, &A.rows, &A.units};  // attend_rows_kernel takes the first
    rc = launch(A.fn, dim3(A.parts), dim3(A.threads), args, A.smem, stream);
    if (rc != SCONV_KV_OK) return rc;
  }
  const int rows = std::min(A.rows, seqs->max_draft * P.g);
  int split = rows <= 16;
  void* args[] = {&P, &A.rows, &A.tile, &A.mtiles, &split};
  return launch(reinterpret_cast<const void*>(sconv::pick_attend_join(D)),
                dim3(static_cast<unsigned>(seqs->num_seqs) * A.mtiles, H, split ? rows : (rows + 3) / 4),
                dim3(128), args, 0, stream);
}

int weights_impl(const void* q, int64_t q_tok, int64_t q_head, int HQ, int H, int D, float scale,
                 const float* lse, const sconv_kv_paged_t* seqs, const void* k, const uint8_t* ks,
                 const sconv_kv_cache_layout_t* layout, float* weights, int64_t positions, int64_t w_seq,
                 int64_t w_head, int* err, void* stream, bool mx) {
  bool empty = false;
  int rc = check_counts(seqs, true, &empty);
  if (rc != SCONV_KV_OK || empty) return rc;
  if (!q || !lse || !weights || !layout) return SCONV_KV_ERR_NULL;
  rc = check_cache(k, nullptr, ks, nullptr, false, mx);
  if (rc != SCONV_KV_OK) return rc;
  WeighParams W;
  memset(&W, 0, sizeof W);
  AttendParams& P = W.a;
  rc = check_paged(seqs, layout, H, D, true, mx, err, &P.s);
  if (rc == SCONV_KV_OK) rc = check_heads(HQ, H, q_tok, q_head, D);
  if (rc != SCONV_KV_OK) return rc;
  if (!isfinite(scale) || positions < 0 || w_seq < 0 || w_head < 0) return SCONV_KV_ERR_SHAPE;
  P.s.capacity = std::min(P.s.capacity, positions);
  if (!aligned(q, 16) || !aligned(weights, 4) || !aligned(lse, 4)) return SCONV_KV_ERR_ALIGN;
  P.c = parts_of(k, nullptr, ks, nullptr, layout);
  P.q = static_cast<const uint16_t*>(q);
  P.q_tok = q_tok;
  P.q_head = q_head;
  P.lse = const_cast<float*>(lse);
  P.HQ = HQ;
  P.H = H;
  P.g = HQ / H;
  P.scale_log2 = scale * sconv::kLog2e;
  W.weights = weights;
  W.w_seq = w_seq;
  W.w_head = w_head;
  if (D == 256 || seqs->max_draft * P.g <= 16) {  // both sides: weigh.cuh
    const void* f = reinterpret_cast<const void*>(sconv::pick_weigh(D, mx));
    const size_t smem = sconv::weigh_smem(D);
    const int threads = 32 * sconv::kWeighWarps;
    if (!smem_attr_set(f, smem)) return SCONV_KV_ERR_CUDA;
    void* args[] = {&W};
    return launch(f, dim3(sm_count() * resident_per_sm(f, threads, smem, 2)), dim3(threads), args,
                  smem, stream);
  }
  sconv::WeighTc T = sconv::pick_weigh_tc(D, mx, seqs->max_draft * P.g);
  const void* f = reinterpret_cast<const void*>(T.fn);
  if (!smem_attr_set(f, T.smem)) return SCONV_KV_ERR_CUDA;
  void* args[] = {&W, &T.rows, &T.units};
  return launch(f, dim3(sm_count()), dim3(T.threads), args, T.smem, stream);
}

int step_impl(const void* k, const void* v, int64_t row_stride, int64_t num_tokens,
              const int32_t* cu, const int32_t* parents, int num_seqs, const void* wk,
              const void* wv, const float* gk, const float* gv, float eps, int W, int H, int D,
              const void* state, const int32_t* state_indices, int64_t pool,
              const int64_t* slots, void* kc, uint8_t* ks, void* vc, uint8_t* vs,
              const sconv_kv_cache_layout_t* layout, const sconv_kv_options_t* options, int* err,
              void* stream, bool mx) {
  if (num_seqs < 0 || num_tokens < 0 || num_tokens > INT32_MAX) return SCONV_KV_ERR_SHAPE;
  if (num_seqs == 0 || num_tokens == 0) return SCONV_KV_OK;
  TreeStepParams A;
  memset(&A, 0, sizeof A);
  int rc = validate_common(k, v, row_stride, wk, wv, gk, gv, W, H, D, const_cast<void*>(state),
                           pool, slots, kc, vc, layout, &A.s, ks, vs, mx);
  if (rc == SCONV_KV_OK) rc = apply_options(options, D, &A.s);
  if (rc != SCONV_KV_OK) return rc;
  if (!cu || !parents) return SCONV_KV_ERR_NULL;
  A.s.num_tokens = num_tokens;
  A.s.cu_seqlens = cu;
  A.s.num_seqs = num_seqs;
  A.s.eps = eps;
  A.s.state_indices = state_indices;
  A.s.err = err;
  A.parents = parents;
  const bool lv = uses_layout_variants(options);
  const sconv::TreeStepFn fn = sconv::pick_tree_step(W, D, mx, lv);
  if (!fn) return SCONV_KV_ERR_UNSUPPORTED;
  // tokens a block: one while the blocks do not fill the GPU, up to eight
  int tokens = static_cast<int>(std::clamp<int64_t>(num_tokens / (4 * sm_count()), 1, 8));
  const unsigned grid = static_cast<unsigned>((num_tokens + tokens - 1) / tokens);
  void* args[] = {&A, &tokens};
  return launch(reinterpret_cast<const void*>(fn), dim3(grid), dim3(256), args, 0, stream);
}

int accept_impl(const void* k, const void* v, int64_t row_stride, const sconv_kv_paged_t* seqs,
                const int32_t* leaves, int W, int H, int D, void* state,
                const int32_t* state_indices, int64_t pool, const int64_t* state_positions,
                void* kc, uint8_t* ks, void* vc, uint8_t* vs,
                const sconv_kv_cache_layout_t* layout, float* weights, int64_t positions, int64_t w_seq,
                int64_t w_head, int32_t* new_lens, int* err, void* stream, bool mx) {
  if (!seqs) return SCONV_KV_ERR_NULL;
  if (seqs->num_seqs < 0 || seqs->num_tokens < 0 || seqs->num_tokens > INT32_MAX)
    return SCONV_KV_ERR_SHAPE;
  if (seqs->num_seqs == 0) return SCONV_KV_OK;
  if (!layout || !leaves || !new_lens || !seqs->context_lens) return SCONV_KV_ERR_NULL;
  // with no drafted token at all the lengths are still to be written; no
  // token tensor is read then
  if (seqs->num_tokens > 0 && (!k || !v)) return SCONV_KV_ERR_NULL;
  int rc = check_cache(kc, vc, ks, vs, true, mx);
  if (rc != SCONV_KV_OK) return rc;
  AcceptParams A;
  memset(&A, 0, sizeof A);
  rc = check_paged(seqs, layout, H, D, true, mx, err, &A.q);
  if (rc != SCONV_KV_OK) return rc;
  if (W < 1 || W > SCONV_KV_MAX_W || pool < 0 || row_stride < static_cast<int64_t>(H) * D ||
      (weights && (positions < 0 || w_seq < 0 || w_head < 0)))
    return SCONV_KV_ERR_SHAPE;
  if (weights) A.q.capacity = std::min(A.q.capacity, positions);
  if (W > 1 && !state) return SCONV_KV_ERR_NULL;
  // (the blocks of a sequence read both while the first of them writes)
  if (new_lens == seqs->context_lens || new_lens == leaves) return SCONV_KV_ERR_SHAPE;
  if (row_stride % 8 || !aligned(k, 16) || !aligned(v, 16) || !aligned(state, 16) ||
      !aligned(weights, 4))
    return SCONV_KV_ERR_ALIGN;
  A.c = parts_of(kc, vc, ks, vs, layout);
  A.mx = mx;
  A.H = H;
  A.D = D;
  A.leaves = leaves;
  A.new_lens = new_lens;
  A.weights = weights;
  A.w_seq = w_seq;
  A.w_head = w_head;
  A.k = static_cast<const uint16_t*>(k);
  A.v = static_cast<const uint16_t*>(v);
  A.row_stride = row_stride;
  A.W = W;
  A.state = static_cast<uint16_t*>(state);
  A.state_indices = state_indices;
  A.pool = pool;
  A.state_pos = state_positions;
  // enough slices for one vector a thread, fewer when the sequences fill the GPU
  const int64_t vecs = static_cast<int64_t>(H) * D / 8;
  const int64_t fill = (8ll * sm_count() + seqs->num_seqs - 1) / seqs->num_seqs;
  const unsigned slices = static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>({(vecs + 255) / 256, fill, 64})));
  void* args[] = {&A};
  return launch(reinterpret_cast<const void*>(sconv::accept_fn()),
                            dim3(static_cast<unsigned>(seqs->num_seqs), slices), dim3(256), args, 0,
                            stream);
}

int evict_impl(const float* weights, int64_t positions, int64_t w_seq, int64_t w_head, const sconv_kv_paged_t* seqs,
               int keep, int sinks, int recent, int H, int D, void* kc, uint8_t* ks, void* vc,
               uint8_t* vs, const sconv_kv_cache_layout_t* layout, int32_t* kept,
               int32_t* new_lens, float* weights_out, int64_t o_positions, int64_t o_seq, int64_t o_head, int* err,
               void* stream, bool mx) {
  bool empty = false;
  int rc = check_counts(seqs, false, &empty);
  if (rc != SCONV_KV_OK || empty) return rc;
  if (!weights || !layout || !kept || !new_lens) return SCONV_KV_ERR_NULL;
  rc = check_cache(kc, vc, ks, vs, true, mx);
  if (rc != SCONV_KV_OK) return rc;
  EvictParams A;
  memset(&A, 0, sizeof A);
  rc = check_paged(seqs, layout, H, D, false, mx, err, &A.q);
  if (rc != SCONV_KV_OK) return rc;
  if (keep < 1 || keep > INT32_MAX - 65536 || sinks < 0 || recent < 0 || static_cast<int64_t>(sinks) + recent > keep ||
      positions < 0 || w_seq < 0 || w_head < 0 || seqs->num_seqs > 65535)
    return SCONV_KV_ERR_SHAPE;
  if (weights_out && (o_positions < std::min<int64_t>(keep, positions) || o_seq < 0 || o_head < 0))
    return SCONV_KV_ERR_SHAPE;
  A.q.capacity = std::min(A.q.capacity, positions);
  if (new_lens == seqs->context_lens || weights_out == weights) return SCONV_KV_ERR_SHAPE;
  if (!aligned(weights, 4) || !aligned(weights_out, 4)) return SCONV_KV_ERR_ALIGN;
  A.c = parts_of(kc, vc, ks, vs, layout);
  A.mx = mx;
  A.H = H;
  A.D = D;
  A.weights = weights;
  A.w_seq = w_seq;
  A.w_head = w_head;
  A.weights_out = weights_out;
  A.o_seq = o_seq;
  A.o_head = o_head;
  A.keep = keep;
  A.sinks = sinks;
  A.recent = recent;
  A.kept = kept;
  A.new_lens = new_lens;
  // Clusters: as many CTAs a (sequence, head) as fill the GPU, while each has 2048 of the positions that a
  // sequence can have.  The lengths are on the device, so that is what the block table or the
  // weights' rows hold, whichever is less, for contexts of any length.  (16 sequences of 8 heads: 2 a
  // selection, 1 a movement, 8 of either for a single sequence.)
  const int64_t units = static_cast<int64_t>(H) * seqs->num_seqs;
  auto spread = [&](int64_t n, int64_t per) {
    int c = 1;
    while (c < sconv::kMaxCluster && n * c < per * sm_count() && c * 2048ll < A.q.capacity) c *= 2;
    return c;
  };
  {
    const int c = spread(units, 1);
    // a slice's keys, of such a sequence, if they fit
    const int64_t slice = (A.q.capacity / c + 1025) / 1024 * 1024 + 1024;
    int room = static_cast<int>(std::min<int64_t>(slice, 48 * 1024));
    const void* fn = sconv::evict_select_fn();
    const size_t smem = 4 * (static_cast<size_t>(room) + 128);  // read four keys at a time
    if (!smem_attr_set(fn, smem)) return SCONV_KV_ERR_CUDA;
    void* args[] = {&A, &room};
    rc = launch_clusters(fn, dim3(H * c, seqs->num_seqs), c, sconv::kSelectThreads, smem, args, stream);
    if (rc != SCONV_KV_OK) return rc;
  }
  const int c = spread(2 * units, 1);
  void* args[] = {&A};
  return launch_clusters(reinterpret_cast<const void*>(sconv::pick_evict_move(D, mx)),
                         dim3(2 * H * c, seqs->num_seqs), c, sconv::kMoveThreads, 0, args, stream);
}

}  // namespace

extern "C" {

int sconv_kv_tree_step(const void* k, const void* v, int64_t row_stride, int64_t num_tokens,
                       const int32_t* cu_draft, const int32_t* parents, int num_seqs,
                       const void* conv_w_k, const void* conv_w_v, const float* gamma_k,
                       const float* gamma_v, float eps, int W, int num_kv_heads, int head_dim,
                       const void* conv_state, const int32_t* state_indices,
                       int64_t state_pool_size, const int64_t* slot_mapping, void* k_cache,
                       void* v_cache, const sconv_kv_cache_layout_t* layout,
                       const sconv_kv_options_t* options, int* err_flag, void* stream) {
  return step_impl(k, v, row_stride, num_tokens, cu_draft, parents, num_seqs, conv_w_k, conv_w_v,
                   gamma_k, gamma_v, eps, W, num_kv_heads, head_dim, conv_state, state_indices,
                   state_pool_size, slot_mapping, k_cache, nullptr, v_cache, nullptr, layout,
                   options, err_flag, stream, false);
}

int sconv_kv_tree_step_mxfp8(const void* k, const void* v, int64_t row_stride, int64_t num_tokens,
                             const int32_t* cu_draft, const int32_t* parents, int num_seqs,
                             const void* conv_w_k, const void* conv_w_v, const float* gamma_k,
                             const float* gamma_v, float eps, int W, int num_kv_heads,
                             int head_dim, const void* conv_state, const int32_t* state_indices,
                             int64_t state_pool_size, const int64_t* slot_mapping, void* k_data,
                             uint8_t* k_scale, void* v_data, uint8_t* v_scale,
                             const sconv_kv_cache_layout_t* layout,
                             const sconv_kv_options_t* options, int* err_flag, void* stream) {
  return step_impl(k, v, row_stride, num_tokens, cu_draft, parents, num_seqs, conv_w_k, conv_w_v,
                   gamma_k, gamma_v, eps, W, num_kv_heads, head_dim, conv_state, state_indices,
                   state_pool_size, slot_mapping, k_data, k_scale, v_data, v_scale, layout,
                   options, err_flag, stream, true);
}

int sconv_kv_tree_attention_workspace(int num_seqs, int max_draft, int num_q_heads,
                                      int num_kv_heads, int head_dim, int64_t* bytes) {
  if (!bytes) return SCONV_KV_ERR_NULL;
  if (num_seqs < 0 || max_draft < 1 || max_draft > SCONV_KV_MAX_DRAFT || num_kv_heads < 1 ||
      num_q_heads < num_kv_heads || num_q_heads % num_kv_heads ||
      num_q_heads > sconv::kMaxQueryHeads ||
      !head_dim_ok(head_dim))
    return SCONV_KV_ERR_SHAPE;
  // enough for either store, and for calls with fewer drafted tokens, whose
  // kernel and split may be others
  int64_t need = 0;
  for (int mx = 0; mx < 2; ++mx)
    for (int n = 1; n <= max_draft; ++n) {
      AttendPlan A;
      const int rc = plan_attend(num_seqs, n, num_q_heads, num_kv_heads, head_dim, mx != 0, &A);
      if (rc != SCONV_KV_OK) return rc;
      need = std::max(need, workspace_need(num_seqs, head_dim, A.parts, A.rows));
    }
  *bytes = need;
  return SCONV_KV_OK;
}

int sconv_kv_tree_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                            int num_q_heads, int num_kv_heads, int head_dim, float scale,
                            const sconv_kv_paged_t* seqs, const void* k_cache,
                            const void* v_cache, const sconv_kv_cache_layout_t* layout, void* out,
                            int64_t out_token_stride, int64_t out_head_stride, float* lse,
                            void* workspace, int64_t workspace_bytes, int* err_flag,
                            void* stream) {
  return attention_impl(q, q_token_stride, q_head_stride, num_q_heads, num_kv_heads, head_dim,
                        scale, seqs, k_cache, nullptr, v_cache, nullptr, layout, out,
                        out_token_stride, out_head_stride, lse, workspace, workspace_bytes,
                        err_flag, stream, false);
}

int sconv_kv_tree_attention_mxfp8(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                  int num_q_heads, int num_kv_heads, int head_dim, float scale,
                                  const sconv_kv_paged_t* seqs, const void* k_data,
                                  const uint8_t* k_scale, const void* v_data,
                                  const uint8_t* v_scale, const sconv_kv_cache_layout_t* layout,
                                  void* out, int64_t out_token_stride, int64_t out_head_stride,
                                  float* lse, void* workspace, int64_t workspace_bytes,
                                  int* err_flag, void* stream) {
  return attention_impl(q, q_token_stride, q_head_stride, num_q_heads, num_kv_heads, head_dim,
                        scale, seqs, k_data, k_scale, v_data, v_scale, layout, out,
                        out_token_stride, out_head_stride, lse, workspace, workspace_bytes,
                        err_flag, stream, true);
}

int sconv_kv_attention_weights(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                               int num_q_heads, int num_kv_heads, int head_dim, float scale,
                               const float* lse, const sconv_kv_paged_t* seqs,
                               const void* k_cache, const sconv_kv_cache_layout_t* layout,
                               float* weights, int64_t positions, int64_t seq_stride,
                               int64_t head_stride,
                               int* err_flag, void* stream) {
  return weights_impl(q, q_token_stride, q_head_stride, num_q_heads, num_kv_heads, head_dim, scale,
                      lse, seqs, k_cache, nullptr, layout, weights, positions, seq_stride, head_stride,
                      err_flag, stream, false);
}

int sconv_kv_attention_weights_mxfp8(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                     int num_q_heads, int num_kv_heads, int head_dim, float scale,
                                     const float* lse, const sconv_kv_paged_t* seqs,
                                     const void* k_data, const uint8_t* k_scale,
                                     const sconv_kv_cache_layout_t* layout, float* weights, int64_t positions, int64_t seq_stride, int64_t head_stride, int* err_flag,
                                     void* stream) {
  return weights_impl(q, q_token_stride, q_head_stride, num_q_heads, num_kv_heads, head_dim, scale,
                      lse, seqs, k_data, k_scale, layout, weights, positions, seq_stride, head_stride,
                      err_flag, stream, true);
}

int sconv_kv_tree_accept(const void* k, const void* v, int64_t row_stride,
                         const sconv_kv_paged_t* seqs, const int32_t* leaves, int W,
                         int num_kv_heads, int head_dim, void* conv_state,
                         const int32_t* state_indices, int64_t state_pool_size,
                         const int64_t* state_positions, void* k_cache, void* v_cache,
                         const sconv_kv_cache_layout_t* layout, float* weights, int64_t positions, int64_t seq_stride, int64_t head_stride, int32_t* new_lens,
                         int* err_flag, void* stream) {
  return accept_impl(k, v, row_stride, seqs, leaves, W, num_kv_heads, head_dim, conv_state,
                     state_indices, state_pool_size, state_positions, k_cache, nullptr, v_cache,
                     nullptr, layout, weights, positions, seq_stride, head_stride, new_lens, err_flag, stream,
                     false);
}

int sconv_kv_tree_accept_mxfp8(const void* k, const void* v, int64_t row_stride,
                               const sconv_kv_paged_t* seqs, const int32_t* leaves, int W,
                               int num_kv_heads, int head_dim, void* conv_state,
                               const int32_t* state_indices, int64_t state_pool_size,
                               const int64_t* state_positions, void* k_data, uint8_t* k_scale,
                               void* v_data, uint8_t* v_scale,
                               const sconv_kv_cache_layout_t* layout, float* weights, int64_t positions, int64_t seq_stride, int64_t head_stride, int32_t* new_lens,
                               int* err_flag, void* stream) {
  return accept_impl(k, v, row_stride, seqs, leaves, W, num_kv_heads, head_dim, conv_state,
                     state_indices, state_pool_size, state_positions, k_data, k_scale, v_data,
                     v_scale, layout, weights, positions, seq_stride, head_stride, new_lens, err_flag, stream,
                     true);
}

int sconv_kv_evict(const float* weights, int64_t positions, int64_t seq_stride, int64_t head_stride,
                   const sconv_kv_paged_t* seqs, int keep, int sinks, int recent,
                   int num_kv_heads, int head_dim, void* k_cache, void* v_cache,
                   const sconv_kv_cache_layout_t* layout, int32_t* kept, int32_t* new_lens,
                   float* weights_out, int64_t out_positions, int64_t out_seq_stride, int64_t out_head_stride,
                   int* err_flag, void* stream) {
  return evict_impl(weights, positions, seq_stride, head_stride, seqs, keep, sinks, recent, num_kv_heads,
                    head_dim, k_cache, nullptr, v_cache, nullptr, layout, kept, new_lens,
                    weights_out, out_positions, out_seq_stride, out_head_stride, err_flag, stream, false);
}

int sconv_kv_evict_mxfp8(const float* weights, int64_t positions, int64_t seq_stride, int64_t head_stride,
                         const sconv_kv_paged_t* seqs, int keep, int sinks, int recent,
                         int num_kv_heads, int head_dim, void* k_data, uint8_t* k_scale,
                         void* v_data, uint8_t* v_scale, const sconv_kv_cache_layout_t* layout,
                         int32_t* kept, int32_t* new_lens, float* weights_out, int64_t out_positions, int64_t out_seq_stride, int64_t out_head_stride, int* err_flag,
                         void* stream) {
  return evict_impl(weights, positions, seq_stride, head_stride, seqs, keep, sinks, recent, num_kv_heads,
                    head_dim, k_data, k_scale, v_data, v_scale, layout, kept, new_lens,
                    weights_out, out_positions, out_seq_stride, out_head_stride, err_flag, stream, true);
}

}  // extern "C"
