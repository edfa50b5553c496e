// Eviction from the paged cache by accumulated attention weight (sm_100a).
//
// Per sequence and K/V head: keep the first `sinks` and the last `recent`
// positions and the (keep - sinks - recent) others of the largest weight,
// ties to the lowest position; the kept rows move to positions 0 .. keep-1 in
// their order.
//
// Both kernels give a (sequence, head) to a cluster of CTAs, one when there are
// enough of them to fill the GPU, up to eight for a single long sequence.
//
// Selection: the weight as an order-preserving 32-bit key, the k-th largest key
// found 8 bits at a time from histograms in shared memory, which the cluster's
// CTAs, a slice of the positions each, read from one another; then the positions
// in order, a warp a stretch: counted, scanned over warps and CTAs, written.  The
// keys stay in shared memory when a slice fits.  It reads 4 bytes a position and is
// bound by the latency of its seven steps.
//
// (30 us for 128 heads of 6072 positions, 37 for 8 of 131,071.)
//
// Movement: in place, so it goes up in rounds.  All of a round's rows are
// loaded by the cluster before any of them is stored; a later round's sources lie
// at or behind its own targets (kept[j] >= j), which no earlier round writes.  It is bound by the
// bytes when there are many heads (16 bf16 contexts to 4096 rows: 80 us, 5 TB/s read and
// written) and by a round's latency for a single context (32,768 MXFP8 rows: 46 us).
#pragma once
#include <cooperative_groups.h>

#include "paged.cuh"

namespace sconv {

namespace cg = cooperative_groups;

// Key whose unsigned order is the weight's: -0 equals +0, NaN above +inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// grid (CTAs of a cluster * H, S); dynamic shared memory: room for `room` keys.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams A, int room) {
  constexpr int kWarps = kSelectThreads / 32;
  grid_dependency_wait();
  allow_dependent_launch();
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  extern __shared__ __align__(16) uint32_t s_keys[];  // room + 128 words
  __shared__ uint32_t s_hist[2][256], s_all[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int2 s_count[kWarps];  // more, equal
  __shared__ int2 s_slice;
  const int h = blockIdx.x / ctas, i = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lead = h == 0 && rank == 0 && tid == 0;
  const SeqView s = seq_view(A.q, i, lead);
  if (!s.ok) return;  // the whole cluster
  const int len = s.ctx;
  if (lead) A.new_lens[i] = min(len, A.keep);
  const float* w = A.weights + i * A.w_seq + h * A.w_head;
  float* wo = A.weights_out ? A.weights_out + i * A.o_seq + h * A.o_head : nullptr;
  int32_t* kept = A.kept + (static_cast<int64_t>(i) * A.H + h) * A.keep;
  if (len <= A.keep) {
    for (int p = rank * kSelectThreads + tid; p < A.keep; p += ctas * kSelectThreads) {
      kept[p] = p < len ? p : -1;
      if (wo && p < len) wo[p] = w[p];
    }
    return;
  }
  // this CTA's slice of the positions, and a warp's stretch of it (multiples of 32)
  const int stretch = ((len / ctas + 1 + kWarps - 1) / kWarps + 31) & ~31;
  const int64_t slice = static_cast<int64_t>(stretch) * kWarps;
  auto at_most = [](int64_t x, int y) { return x < y ? static_cast<int>(x) : y; };
  const int a = at_most(static_cast<int64_t>(rank) * slice, len);
  const int e = at_most(static_cast<int64_t>(a) + slice, len);
  const int lo = A.sinks, hi = len - A.recent;  // candidates
  const bool held = e - a <= room;
  if (held) {
#pragma unroll 4
    for (int p = a + tid; p < e; p += kSelectThreads) s_keys[p - a] = weight_key(w[p]);
  }
  for (int b = tid; b < 512; b += kSelectThreads) (&s_hist[0][0])[b] = 0;
  __syncthreads();
  auto key_at = [&](int p) { return held ? s_keys[p - a] : weight_key(w[p]); };
  const bool any = A.keep - A.sinks - A.recent > 0;
  int need = A.keep - A.sinks - A.recent;  // 0 <= need < hi - lo
  uint32_t prefix = 0;
  if (any) {
    const int c0 = max(a, lo), c1 = min(e, hi);
    for (int step = 0; step < 4; ++step) {
      const int shift = 24 - 8 * step;
      uint32_t* hist = s_hist[step & 1];
      const uint32_t above = step == 0 ? 0u : 0xffffffffu << (shift + 8);
      // one key: equal bins (weights are often equal) are added once a warp
      auto tally = [&](uint32_t key, bool in) {
        const bool mine = in && (key & above) == prefix;
        if (!__any_sync(kFullMask, mine)) return;
        const uint32_t bin = mine ? (key >> shift) & 255u : 256u;
        const unsigned same = __match_any_sync(kFullMask, bin);
        if (mine && lane == __ffs(same) - 1) atomicAdd(&hist[bin], __popc(same));
      };
      if (held) {  // four keys a lane; the slice begins on a multiple of 1024
        const int n = c1 - a;
        for (int q = (c0 - a) / 128 * 128 + warp * 128; q < n; q += 4 * kSelectThreads) {
          const int x = q + 4 * lane;
          const uint4 k = *reinterpret_cast<const uint4*>(s_keys + x);
          tally(k.x, x >= c0 - a && x < n);
          tally(k.y, x + 1 >= c0 - a && x + 1 < n);
          tally(k.z, x + 2 >= c0 - a && x + 2 < n);
          tally(k.w, x + 3 >= c0 - a && x + 3 < n);
        }
      } else {
        for (int p = c0 + warp * 32; p < c1; p += kSelectThreads)
          tally(p + lane < c1 ? weight_key(w[p + lane]) : 0u, p + lane < c1);
      }
      cluster.sync();
      if (tid < 256) {
        uint32_t sum = 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)  // all in flight at once
          if (c < ctas) sum += cluster.map_shared_rank(hist, c)[tid];
        s_all[tid] = sum;
        s_hist[(step + 1) & 1][tid] = 0;  // last read before the sync above
      }
      __syncthreads();
      if (warp == 0) {  // the bin that the need-th largest falls in
        uint32_t own[8], sum = 0;
#pragma unroll
        for (int b = 0; b < 8; ++b) {  // lane l holds bins 255-8l .. 248-8l
          own[b] = s_all[255 - 8 * lane - b];
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
#pragma unroll
          for (int k = 0; k < 7; ++k)
            if (b == k && before + own[k] < want) {
              before += own[k];
              ++b;
            }
          s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - b) << shift);
          s_need = need - static_cast<int>(before);
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
  }
  // prefix: the key of the last kept; the first `need` of those equal to it are kept
  const int p0 = at_most(static_cast<int64_t>(a) + warp * stretch, e);
  const int p1 = at_most(static_cast<int64_t>(p0) + stretch, e);
  auto classify = [&](int p, bool& more, bool& same) {
    more = same = false;
    if (p >= p1) return;
    if (p < lo || p >= hi) {
      more = true;
    } else if (any) {
      const uint32_t key = key_at(p);
      more = key > prefix;
      same = key == prefix;
    }
  };
  int2 count = make_int2(0, 0);
#pragma unroll 4
  for (int p = p0; p < p1; p += 32) {
    bool more, same;
    classify(p + lane, more, same);
    count.x += more;
    count.y += same;
  }
  count.x = __reduce_add_sync(kFullMask, count.x);
  count.y = __reduce_add_sync(kFullMask, count.y);
  if (lane == 0) s_count[warp] = count;
  __syncthreads();
  int2 before = make_int2(0, 0);
  if (warp == 0) {
    int2 c = s_count[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(kFullMask, c.x, d), y = __shfl_up_sync(kFullMask, c.y, d);
      if (lane >= d) {
        c.x += x;
        c.y += y;
      }
    }
    if (lane == 31) s_slice = c;
    const int2 own = s_count[lane];
    s_count[lane] = make_int2(c.x - own.x, c.y - own.y);
  }
  cluster.sync();
  for (int c = 0; c < rank; ++c) {
    const int2 v = *cluster.map_shared_rank(&s_slice, c);
    before.x += v.x;
    before.y += v.y;
  }
  int more_at = before.x + s_count[warp].x, same_at = before.y + s_count[warp].y;
  for (int p = p0; p < p1; p += 32) {
    bool more, same;
    classify(p + lane, more, same);
    const unsigned bm = __ballot_sync(kFullMask, more), bs = __ballot_sync(kFullMask, same);
    const unsigned lower = (1u << lane) - 1u;
    const int rank_same = same_at + __popc(bs & lower);
    const int at = more_at + __popc(bm & lower) + min(rank_same, need);
    if (more || (same && rank_same < need)) {
      kept[at] = p + lane;
      if (wo) wo[at] = w[p + lane];
    }
    more_at += __popc(bm);
    same_at += __popc(bs);
  }
  cluster.sync();  // nobody leaves while its counts may be read
}

// A row's scale bytes, one access where they are aligned.
template <typename SC>
__device__ __forceinline__ SC load_scales(const uint8_t* p, bool packed) {
  if (packed) return *reinterpret_cast<const SC*>(p);
  SC v = 0;
#pragma unroll
  for (int b = 0; b < static_cast<int>(sizeof(SC)); ++b) v |= static_cast<SC>(p[b]) << (8 * b);
  return v;
}
template <typename SC>
__device__ __forceinline__ void store_scales(uint8_t* p, SC v, bool packed) {
  if (packed) {
    *reinterpret_cast<SC*>(p) = v;
    return;
  }
#pragma unroll
  for (int b = 0; b < static_cast<int>(sizeof(SC)); ++b) p[b] = static_cast<uint8_t>(v >> (8 * b));
}

// grid (CTAs of a cluster * 2 * H, S): K's or V's rows of one head, with their
// scales (MXFP8).  A thread has one 16-byte piece of kMoveRows rows a round.
// DB: bytes of a row; SC: its scales as one number (bf16: unused).
constexpr int kMoveRows = 8;

template <int DB, bool MX, typename SC>
__global__ void __launch_bounds__(kMoveThreads, 2) evict_move_kernel(const EvictParams A) {
  grid_dependency_wait();
  allow_dependent_launch();
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / ctas, h = unit >> 1, i = blockIdx.y;
  const SeqView s = seq_view(A.q, i, false);
  if (!s.ok || s.ctx <= A.keep) return;  // the whole cluster
  constexpr int kVecs = DB / 16, kSide = kMoveThreads / kVecs, kChunk = kSide * kMoveRows;
  const int r = threadIdx.x / kVecs, x = threadIdx.x % kVecs;
  const int32_t* kept = A.kept + (static_cast<int64_t>(i) * A.H + h) * A.keep;
  const int32_t* table = A.q.table + i * A.q.table_stride;
  const int64_t head = h * A.q.stride_head;
  uint8_t* base = ((unit & 1) ? A.c.v : A.c.k) + head * (MX ? 1 : 2) + x * 16;
  uint8_t* scales = MX ? ((unit & 1) ? A.c.vs : A.c.ks) + (head >> 5) : nullptr;
  const bool packed = A.c.scales_packed;
  // Where a round's rows are and go, looked up by a thread each while the
  // round before is under way (~0u: stays, or a page outside the cache).
  __shared__ uint32_t s_from[3][kChunk], s_to[3][kChunk];
  auto look_up = [&](int b, int j0) {
    for (int q = threadIdx.x; q < kChunk; q += kMoveThreads) {
      const int j = j0 + q;
      uint32_t f = ~0u, t = ~0u;
      if (j < A.keep) {
        const int p = __ldg(kept + j);
        if (p > j) {
          const int pf = __ldg(table + page_index(A.q, p)), pt = __ldg(table + page_index(A.q, j));
          if (static_cast<unsigned>(pf) < static_cast<unsigned>(A.q.num_pages) &&
              static_cast<unsigned>(pt) < static_cast<unsigned>(A.q.num_pages)) {
            f = row_off8(A.q, pf, p);
            t = row_off8(A.q, pt, j);
          } else {
            raise_flag(A.q.err, kFlagSlotRange);
          }
        }
      }
      s_from[b][q] = f;
      s_to[b][q] = t;
    }
  };
  int j0 = rank * kChunk;
  look_up(0, j0);
  __syncthreads();
  for (int b = 0; j0 - rank * kChunk < A.keep; j0 += ctas * kChunk) {
    const int next = b == 2 ? 0 : b + 1;
    uint4 buf[kMoveRows];
    SC sc[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const uint32_t f = s_from[b][u * kSide + r];
      if (f != ~0u) {
        buf[u] = *reinterpret_cast<const uint4*>(base + static_cast<uint64_t>(f) * (MX ? 8 : 16));
        if (MX && x == 0) sc[u] = load_scales<SC>(scales + (f >> 2), packed);
      }
    }
    look_up(next, j0 + ctas * kChunk);
    cluster.sync();
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const uint32_t t = s_to[b][u * kSide + r];
      if (t != ~0u) {
        *reinterpret_cast<uint4*>(base + static_cast<uint64_t>(t) * (MX ? 8 : 16)) = buf[u];
        if (MX && x == 0) store_scales<SC>(scales + (t >> 2), sc[u], packed);
      }
    }
    b = next;  // (of three: one that a slower thread may still read is not written)
  }
}

}  // namespace sconv
