// Paged sequences with a tree of drafted tokens: the arguments, lookups and
// checks that the drafted-tree kernels share (tree_step.cuh, attend.cuh,
// attend_tc.cuh, evict.cuh).
//
// Sequence i holds lens[i] cached tokens at positions 0 .. lens[i]-1 and its
// drafted tokens cu[i] .. cu[i+1]-1 behind them, draft j at position
// lens[i] + j.  Position p is slot p % page_size of page
// table[i, p / page_size].  parents[t] is the local index of t's parent
// (below its own), -1 for a child of the context, <= -2 for an unused token
// (padding).  A token is used if its chain of parents ends at -1.
#pragma once
#include "tma.cuh"
#include "tree_params.h"

namespace sconv {

struct SeqView {
  int64_t a;  // first packed token
  int n;      // drafted tokens
  int ctx;    // cached tokens
  bool ok;
};

__device__ __forceinline__ int page_index(const PagedSeqs& Q, int p) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(p), Q.page_mul) +
                           static_cast<uint32_t>(p)) >> Q.page_shift);
}

// Checked view of sequence i.  Whoever passes `report` raises the flags.
__device__ __forceinline__ SeqView seq_view(const PagedSeqs& Q, int i, bool report) {
  SeqView s;
  int64_t e = 0;
  s.a = 0;
  s.ok = true;
  if (Q.cu) {
    s.a = __ldg(Q.cu + i);
    e = __ldg(Q.cu + i + 1);
  }
  const int64_t n = e - s.a;
  if (s.a < 0 || n < 0 || e > Q.num_tokens) {
    if (report) raise_flag(Q.err, kFlagCuSeqlens);
    s.ok = false;
  } else if (n > Q.max_draft) {
    if (report) raise_flag(Q.err, kFlagTree);
    s.ok = false;
  }
  s.n = s.ok ? static_cast<int>(n) : 0;
  s.ctx = __ldg(Q.lens + i);
  if (s.ctx < 0 || s.ctx + static_cast<int64_t>(s.n) > Q.capacity) {
    if (report) raise_flag(Q.err, kFlagContext);
    s.ok = false;
    s.n = 0;
    s.ctx = 0;
  }
  return s;
}

// Page of position p of sequence i; a page outside the cache is flagged and
// read as page 0 (in bounds; the sequence's result is then unspecified).
// -1 with `skip_bad`.
__device__ __forceinline__ int page_of(const PagedSeqs& Q, int i, int p, bool skip_bad = false) {
  const int page = __ldg(Q.table + i * Q.table_stride + page_index(Q, p));
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(Q.num_pages)) {
    raise_flag(Q.err, kFlagSlotRange);
    return skip_bad ? -1 : 0;
  }
  return page;
}

// Element offset of position p's row (head 0) given its page.
__device__ __forceinline__ int64_t row_offset(const PagedSeqs& Q, int page, int p) {
  const int off = p - page_index(Q, p) * Q.page_size;
  return page * Q.stride_page + off * Q.stride_slot;
}

// The same in units of 8 elements (below 2^32: the host checks the cache).
__device__ __forceinline__ uint32_t row_off8(const PagedSeqs& Q, int page, int p) {
  return static_cast<uint32_t>(page) * Q.page8 +
         static_cast<uint32_t>(p - page_index(Q, p) * Q.page_size) * Q.slot8;
}
// That of a position read through `page`; ~0u at or
// behind `total`.  A page outside the cache is flagged and read as page 0.
__device__ __forceinline__ uint32_t paged_off8(const PagedSeqs& Q, int page, int p, int total) {
  if (p >= total) return ~0u;
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(Q.num_pages)) {
    raise_flag(Q.err, kFlagSlotRange);
    page = 0;
  }
  return row_off8(Q, page, p);
}

// Sequence of packed token t: the largest i in [0, S-1] with cu[i] <= t.
// One 32-way probe a round for the whole warp (all lanes, uniform t).
__device__ __forceinline__ int warp_seq_of(const int32_t* cu, int S, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = S;  // the answer lies in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const int at = lo + lane * step;
    const bool le = lane * step < len && __ldg(cu + at) <= t;
    const unsigned hit = __ballot_sync(kFullMask, le) | 1u;
    const int last = 31 - __clz(hit);
    lo += last * step;
    len = min(step, len - last * step);
  }
  return lo;
}

// Ancestor masks of a sequence's drafted tokens in shared memory, by pointer
// doubling: anc[j] = bits of j and its ancestors, 0 for an unused token.
// Threads 0 .. n-1 (n >= kMaxDraft) of the block take part; `meet` is a barrier
// among them.  A parent at or behind its own token, or an unused
// one, makes the token unused and raises the tree flag.
template <class Meet>
__device__ __forceinline__ void ancestor_masks(const PagedSeqs& Q, const SeqView& s,
                                               uint32_t (*anc)[kMaskWords], int* ptr, bool report,
                                               Meet meet) {
  const int j = threadIdx.x;
  const bool mine = j < s.n;
  uint32_t m[kMaskWords];
  int p = -2;
  bool bad = false;
  if (j < kMaxDraft) {
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) m[w] = 0;
    if (mine) {
      p = __ldg(Q.parents + s.a + j);
      bad = p >= j;
      if (bad || p < -2) p = -2;
#pragma unroll
      for (int w = 0; w < kMaskWords; ++w) m[w] = (j >> 5) == w ? 1u << (j & 31) : 0u;
    }
    ptr[j] = p;
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) anc[j][w] = m[w];
  }
  const bool unused = p == -2;
  meet();
  for (int reach = 1; reach < s.n; reach <<= 1) {
    int np = p;
    if (mine && p >= 0) {
      np = ptr[p];
#pragma unroll
      for (int w = 0; w < kMaskWords; ++w) m[w] |= anc[p][w];
    }
    meet();
    if (mine && p >= 0) {
      p = np;
      ptr[j] = p;
#pragma unroll
      for (int w = 0; w < kMaskWords; ++w) anc[j][w] = m[w];
    }
    meet();
  }
  if (mine && p == -2) {
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) anc[j][w] = 0;
    if (report && (bad || !unused)) raise_flag(Q.err, kFlagTree);
  }
  meet();
}
__device__ __forceinline__ void ancestor_masks(const PagedSeqs& Q, const SeqView& s,
                                               uint32_t (*anc)[kMaskWords], int* ptr,
                                               bool report) {  // the whole block
  ancestor_masks(Q, s, anc, ptr, report, [] { __syncthreads(); });
}

}  // namespace sconv
