// Eviction from the paged cache by accumulated attention weight (sm_100a).
//
// Per sequence and K/V head: keep the first `sinks` and the last `recent`
// positions and the (keep - sinks - recent) others of the largest weight,
// ties to the lowest position; the kept rows move to positions 0 .. keep-1 in
// their order.
//
// Selection (evict_select_kernel): the weight as an order-preserving 32-bit
// key, the k-th largest key found 8 bits at a time from histograms in shared
// memory, then one pass in position order that writes the kept positions and
// their weights.  Movement (evict_move_kernel): see there.
#pragma once
#include "paged.cuh"

namespace sconv {

// Key whose unsigned order is the weight's: -0 equals +0, NaN above +inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}


// One block a (sequence, head).
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams A) {
  grid_dependency_wait();
  allow_dependent_launch();
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int s_warp[2][kSelectThreads / 32];
  const int h = blockIdx.x, i = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lead = h == 0 && tid == 0;
  const SeqView s = seq_view(A.q, i, lead);
  if (!s.ok) return;
  const int len = s.ctx;
  if (lead) A.new_lens[i] = min(len, A.keep);
  const float* w = A.weights + i * A.w_seq + h * A.w_head;
  float* wo = A.weights_out ? A.weights_out + i * A.o_seq + h * A.o_head : nullptr;
  int32_t* kept = A.kept + (static_cast<int64_t>(i) * A.H + h) * A.keep;
  if (len <= A.keep) {
    for (int p = tid; p < A.keep; p += kSelectThreads) {
      kept[p] = p < len ? p : -1;
      if (wo && p < len) wo[p] = w[p];
    }
    return;
  }
  const int lo = A.sinks, hi = len - A.recent;  // candidates
  int need = A.keep - A.sinks - A.recent;       // 0 <= need < hi - lo
  uint32_t prefix = 0;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int b = tid; b < 256; b += kSelectThreads) hist[b] = 0;
      __syncthreads();
      const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int p = lo + tid; p < hi; p += kSelectThreads) {
        const uint32_t key = weight_key(w[p]);
        if ((key & above) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // the bin that the need-th largest falls in
        uint32_t own[8], sum = 0;
#pragma unroll
        for (int b = 0; b < 8; ++b) {  // lane l holds bins 255-8l .. 248-8l
          own[b] = hist[255 - 8 * lane - b];
          sum += own[b];
        }
        uint32_t before = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t up = __shfl_up_sync(kFullMask, before, d);
          if (lane >= d) before += up;
        }
        before -= sum;
        const uint32_t want = static_cast<uint32_t>(need);
        if (before < want && want <= before + sum) {
          int b = 0;
          while (before + own[b] < want) before += own[b++];
          s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - b) << shift);
          s_need = need - static_cast<int>(before);
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
  }
  // prefix: the key of the last kept; `need` of those equal to it are kept
  const bool any = A.keep - A.sinks - A.recent > 0;
  int taken = 0, equal = 0;  // before this chunk
  for (int base = 0; base < len; base += kSelectThreads) {
    const int p = base + tid;
    float x = 0.f;
    bool more = false, same = false;
    if (p < len) {
      x = w[p];
      if (p < lo || p >= hi) {
        more = true;
      } else if (any) {
        const uint32_t key = weight_key(x);
        more = key > prefix;
        same = key == prefix;
      }
    }
    const unsigned bs = __ballot_sync(kFullMask, same);
    if (lane == 0) s_warp[0][warp] = __popc(bs);
    __syncthreads();
    int eq = equal, eq_all = equal;
    for (int k = 0; k < kSelectThreads / 32; ++k) {
      const int v = s_warp[0][k];
      if (k < warp) eq += v;
      eq_all += v;
    }
    eq += __popc(bs & ((1u << lane) - 1u));
    const bool keep = more || (same && eq < need);
    const unsigned bk = __ballot_sync(kFullMask, keep);
    if (lane == 0) s_warp[1][warp] = __popc(bk);
    __syncthreads();
    int at = taken, at_all = taken;
    for (int k = 0; k < kSelectThreads / 32; ++k) {
      const int v = s_warp[1][k];
      if (k < warp) at += v;
      at_all += v;
    }
    at += __popc(bk & ((1u << lane) - 1u));
    if (keep) {
      kept[at] = p;
      if (wo) wo[at] = x;
    }
    taken = at_all;
    equal = eq_all;
    __syncthreads();
  }
}

// Rows kept[j] -> j of one cache part, in place.  A block owns one slice of
// the row's bytes of one (sequence, head, part) and walks j upwards in
// chunks: a chunk is loaded whole before any of it is stored, and every
// source of a later chunk lies at or behind that chunk's first target
// (kept[j] >= j), so no row is overwritten before it is read.
constexpr int kMoveRows = 8;  // rows in flight a thread

template <typename V>
__device__ __forceinline__ void move_rows(const EvictParams& A, uint8_t* base, int i, int h,
                                          const int32_t* kept, int keep, int vecs, int col_bytes,
                                          int num, int den) {
  // byte address of element offset e: e * num / den
  const int per = kMoveThreads / vecs;  // rows side by side
  const int r = threadIdx.x / vecs, x = threadIdx.x - r * vecs;
  const int64_t head = h * A.q.stride_head;
  for (int j0 = 0; j0 < keep; j0 += per * kMoveRows) {
    V buf[kMoveRows];
    bool mv[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int j = j0 + u * per + r;
      mv[u] = false;
      if (r < per && j < keep) {
        const int p = kept[j];
        if (p > j) {
          const int page = page_of(A.q, i, p, true);
          if (page >= 0) {
            mv[u] = true;
            buf[u] = *reinterpret_cast<const V*>(
                base + (row_offset(A.q, page, p) + head) * num / den + col_bytes + x * sizeof(V));
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int j = j0 + u * per + r;
      if (mv[u]) {
        const int page = page_of(A.q, i, j, true);
        if (page >= 0)
          *reinterpret_cast<V*>(base + (row_offset(A.q, page, j) + head) * num / den + col_bytes +
                                x * sizeof(V)) = buf[u];
      }
    }
  }
}

// grid (parts, H, S): parts = 2 (K, V), or 4 with the MXFP8 scales.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams A) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int part = blockIdx.x, h = blockIdx.y, i = blockIdx.z;
  const SeqView s = seq_view(A.q, i, false);
  if (!s.ok || s.ctx <= A.keep) return;
  const int32_t* kept = A.kept + (static_cast<int64_t>(i) * A.H + h) * A.keep;
  if (part < 2) {
    uint8_t* base = part ? A.c.v : A.c.k;
    const int bytes = A.mx ? A.D : 2 * A.D;
    move_rows<uint4>(A, base, i, h, kept, A.keep, bytes / 16, 0, A.mx ? 1 : 2, 1);
  } else {
    uint8_t* base = part == 3 ? A.c.vs : A.c.ks;
    move_rows<uint8_t>(A, base, i, h, kept, A.keep, A.D / 32, 0, 1, 32);
  }
}

}  // namespace sconv
