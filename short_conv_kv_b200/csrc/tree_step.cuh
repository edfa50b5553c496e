// The ShortConv K/V step for a tree of drafted tokens, and the acceptance of
// one of its paths (sm_100a).
//
// Step: the conv window of a drafted token follows its parents, then the
// sequence's conv_state, instead of its packed predecessors; the state is
// only read.  Each output is the same chain of fused multiply-adds, head
// butterfly and rounding as in the prefill and decode kernels, so a tree that
// is a chain gives their bits.
//
// Acceptance: with path a_0 < a_1 < ... < a_{m-1} (the leaf's ancestors and
// the leaf), position ctx + a_r moves to ctx + r, and the conv_state takes
// the last W-1 rows of (state ++ the path's raw rows).
//
// Both move a few KB a token through HBM and are bound by its latency at
// small sizes: 4.9 and 5.1 us a call for a tree of 8, 33 us for the step of 256 MXFP8 trees, 15 for the
// acceptance of 512 paths.
#pragma once
#include "paged.cuh"

namespace sconv {

// A block has up to kStepTokens tokens.  First a warp a token finds the token's
// sequence, walks its parents and looks its slot up (some five dependent loads), then
// all threads compute, 8 channels of one token at a time; a warp's 32 groups are
// consecutive, so a head's D/8 lanes are aligned.  (With a token a block and the
// walk in every thread, 8192 tokens of 2 x 1024 channels took 53 us, so 33.)  Bound by
// latency, so four blocks an SM go before loads ahead: with the next token's rows in
// registers there are two, and it takes 40 us.
constexpr int kStepTokens = 8;

// (the raw rows and the state are only read)
__device__ __forceinline__ uint4 ld_plain(const uint16_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}

template <int W, int D, bool MX, bool LV>
__global__ void __launch_bounds__(256, W <= 4 ? 4 : 2) tree_step_kernel(const TreeStepParams A, int tokens) {
  grid_dependency_wait();
  allow_dependent_launch();
  const StepParams& P = A.s;
  __shared__ int s_row[kStepTokens][8];  // tap j's row: a token, or ~q for row q of the state
  __shared__ int64_t s_state[kStepTokens], s_off[kStepTokens];
  __shared__ int s_run[kStepTokens];
  const int half = P.NG >> 1;
  const int64_t srow = 2 * static_cast<int64_t>(P.C);
  const int64_t t0 = blockIdx.x * static_cast<int64_t>(tokens);
  const int here = static_cast<int>(min(static_cast<int64_t>(tokens), P.num_tokens - t0));
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  if (wp < here) {  // (a block has kStepTokens warps)
    const int64_t t = t0 + wp;
    const int64_t slot = __ldg(P.slots + t);
    const int first_up = __ldg(A.parents + t);
    const int i = warp_seq_of(P.cu_seqlens, P.num_seqs, t);
    const int64_t a = __ldg(P.cu_seqlens + i), e = __ldg(P.cu_seqlens + i + 1);
    int flags = 0;
    bool run = slot >= 0;
    if (run && slot >= P.num_slots) {
      flags |= kFlagSlotRange;
      run = false;
    }
    if (!(a >= 0 && a <= t && t < e && e <= P.num_tokens)) {
      // behind the last sequence (t >= e) is not an error
      if (t < e) flags |= kFlagCuSeqlens;
      run = false;
    }
    int64_t si = 0;
    int rot = 0;
    if (W > 1 && run) {
      si = P.state_indices ? static_cast<int64_t>(__ldg(P.state_indices + i)) : i;
      int64_t pos = 0;
      if (LV && P.state_pos) pos = __ldg(P.state_pos + i);
      if (si < 0 || si >= P.pool || pos < 0) {
        flags |= kFlagStateIndex;
        run = false;
      } else if (LV && P.state_pos) {
        rot = static_cast<int>(pos % (W > 1 ? W - 1 : 1));
      }
    }
    // tap j's row: the ancestor W-1-j levels up, or a state row
    int64_t node = t - a;
    int above = 0;  // state rows passed
#pragma unroll
    for (int j = W - 1; j >= 0; --j) {
      if (!run) break;
      if (node >= 0) {
        const int64_t up = j == W - 1 ? first_up : __ldg(A.parents + a + node);
        if (lane == 0) s_row[wp][j] = static_cast<int>(a + node);
        if (up < -1 || up >= node) {
          // unused (the token itself below -1: padding), or malformed
          if (up >= node || j != W - 1) flags |= kFlagTree;
          run = false;
        }
        node = up;
      } else {
        int q = W - 2 - above;
        if (LV) q = q + rot >= W - 1 ? q + rot - (W - 1) : q + rot;
        if (lane == 0) s_row[wp][j] = ~q;
        ++above;
      }
    }
    if (lane == 0) {
      if (flags) raise_flag(P.err, flags);
      int64_t off = 0;
      if (run) {
        const int64_t page = P.slot_linear ? 0 : slot / P.page_size;
        off = page * P.stride_page + (slot - page * P.page_size) * P.stride_slot;
      }
      s_off[wp] = off;
      s_state[wp] = si * (W - 1) * srow;
      s_run[wp] = run;
    }
  }
  __syncthreads();
  // A thread keeps its 8 channels, taps and gammas unpacked in registers, and takes
  // every side-th token (rows narrower than the block stand side by side).
  const int side = max(1, 256 / P.NG), mine = threadIdx.x / P.NG;
  for (int gb = 0; gb < P.NG; gb += 256) {
    const int gg = P.NG < 256 ? static_cast<int>(threadIdx.x) - mine * P.NG : gb + static_cast<int>(threadIdx.x);
    const bool inside = gg < P.NG && (P.NG >= 256 || mine < side);
    const int g = inside ? gg : 0;
    const bool isv = g >= half;
    const int c0 = (isv ? g - half : g) * 8;
    const int d0 = c0 % D, h = c0 / D;
    const uint16_t* x = (isv ? P.v : P.k) + c0;
    const uint16_t* st0 = P.state + (isv ? P.C : 0) + c0;
    const uint16_t* w = (isv ? P.w_v : P.w_k) + c0;
    float2 tw[W][4];
#pragma unroll
    for (int j = 0; j < W; ++j) unpack8(ld_ro(w + static_cast<int64_t>(j) * P.C), tw[j]);
    const float* gam = (isv ? P.gamma_v : P.gamma_k) + h * P.gamma_hs + d0;
    const float4 ga = __ldg(reinterpret_cast<const float4*>(gam));
    const float4 gc = __ldg(reinterpret_cast<const float4*>(gam) + 1);
    const float2 gm[4] = {make_float2(ga.x, ga.y), make_float2(ga.z, ga.w),
                          make_float2(gc.x, gc.y), make_float2(gc.z, gc.w)};
    const int step0 = P.NG < 256 ? mine : 0;
    // the rows of token k0 + step0, zeros where it does not run
    auto load = [&](uint4(&rows)[W], int k0) {
      const int k = min(k0 + step0, kStepTokens - 1);
      const bool run = inside && k < here && s_run[k];
      const uint16_t* st = st0 + s_state[k];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int r = run ? s_row[k][j] : 0;
        const uint16_t* from = r >= 0 ? x + r * P.row_stride : st + ~r * srow;
        rows[j] = run ? ld_plain(from) : make_uint4(0, 0, 0, 0);
      }
    };
#pragma unroll 1
    for (int k0 = 0; k0 < here; k0 += side) {
      const int k = min(k0 + step0, kStepTokens - 1);
      const bool run = inside && k < here && s_run[k];
      uint4 rows[W];
      load(rows, k0);
      float2 acc[4];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float2 rf[4];
        unpack8(rows[j], rf);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          acc[u] = j == 0 ? fmul2(tw[j][u], rf[u]) : ffma2(tw[j][u], rf[u], acc[u]);
      }
      float2 s2 = fmul2(acc[0], acc[0]);
      s2 = ffma2(acc[1], acc[1], s2);
      s2 = ffma2(acc[2], acc[2], s2);
      s2 = ffma2(acc[3], acc[3], s2);
      const float ss = group_sum<D / 8>(s2.x + s2.y);
      const float rn = rsqrt_approx(fmaf(ss, P.inv_d, P.eps));
      const int64_t off = s_off[k] + h * P.stride_head + d0;
      if constexpr (MX) {
        // every lane takes part: the block scale is a 4-lane reduction
        const float2 tt[4] = {fmul2(acc[0], gm[0]), fmul2(acc[1], gm[1]), fmul2(acc[2], gm[2]),
                              fmul2(acc[3], gm[3])};
        mx_store8(tt, rn, run, (isv ? P.v_data : P.k_data) + off,
                  (isv ? P.v_scale : P.k_scale) + (off >> 5));
      } else if (run) {
        const float2 rr = make_float2(rn, rn);
        uint4 o;
        o.x = pack_bf16x2(fmul2(fmul2(acc[0], rr), gm[0]));
        o.y = pack_bf16x2(fmul2(fmul2(acc[1], rr), gm[1]));
        o.z = pack_bf16x2(fmul2(fmul2(acc[2], rr), gm[2]));
        o.w = pack_bf16x2(fmul2(fmul2(acc[3], rr), gm[3]));
        *reinterpret_cast<uint4*>((isv ? P.v_cache : P.k_cache) + off) = o;
      }
    }
  }
}

// Move the path's rows of one cache part: `unit` bytes a vector, vectors of
// a head contiguous.  A thread owns one vector of the row and walks the path
// upwards, kBatch rows loaded before they are stored: the targets r .. r+7
// lie before every source a_s, s >= r + 8, so nothing unread is overwritten.
template <typename V>
__device__ __forceinline__ void accept_part(const AcceptParams& A, uint8_t* base, int elem_per_vec,
                                            int64_t div, const int64_t* from, const int64_t* to,
                                            int m, int first, int slot, int slots) {
  constexpr int kBatch = 8;
  const int per_head = A.D / elem_per_vec, all = A.H * per_head;
  for (int x = slot; x < all; x += slots) {
    const int h = x / per_head;
    const int64_t col = h * A.q.stride_head + static_cast<int64_t>(x - h * per_head) * elem_per_vec;
    for (int r0 = first; r0 < m; r0 += kBatch) {
      V buf[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (r0 + u < m && from[r0 + u] >= 0)
          buf[u] = *reinterpret_cast<const V*>(base + (from[r0 + u] + col) * 2 / div);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (r0 + u < m && from[r0 + u] >= 0)
          *reinterpret_cast<V*>(base + (to[r0 + u] + col) * 2 / div) = buf[u];
    }
  }
}

// grid (num_seqs, slices): the slices share a sequence's columns.
__global__ void __launch_bounds__(256) tree_accept_kernel(const AcceptParams A) {
  grid_dependency_wait();
  allow_dependent_launch();
  __shared__ int s_par[kMaxDraft], s_path[kMaxDraft];
  __shared__ int64_t s_from[kMaxDraft], s_to[kMaxDraft];
  __shared__ int s_m, s_first;
  const int i = blockIdx.x;
  const bool lead = blockIdx.y == 0;
  const SeqView s = seq_view(A.q, i, lead && threadIdx.x == 0);
  if (!s.ok) return;
  for (int j = threadIdx.x; j < s.n; j += blockDim.x) s_par[j] = __ldg(A.q.parents + s.a + j);
  __syncthreads();
  if (threadIdx.x == 0) {
    int m = 0, node = __ldg(A.leaves + i);
    bool bad = node >= s.n || node < -1;
    if (!bad)
      for (int j = node; j >= 0; ++m) {  // ends: each parent is below its child
        s_path[m] = j;
        const int up = s_par[j];
        if (up < -1 || up >= j) {
          bad = true;
          break;
        }
        j = up;
      }
    if (bad && lead) raise_flag(A.q.err, kFlagTree);
    s_m = bad ? 0 : m;
    s_first = kMaxDraft;
  }
  __syncthreads();
  const int m = s_m;
  if (lead && threadIdx.x == 0) A.new_lens[i] = s.ctx + m;
  if (m == 0) return;
  if (threadIdx.x < m) {
    const int r = threadIdx.x, j = s_path[m - 1 - r];
    int64_t from = -1, to = -1;
    if (j != r) {
      const int pf = page_of(A.q, i, s.ctx + j, true), pt = page_of(A.q, i, s.ctx + r, true);
      if (pf >= 0 && pt >= 0) {
        from = row_offset(A.q, pf, s.ctx + j);
        to = row_offset(A.q, pt, s.ctx + r);
      }
      atomicMin(&s_first, r);
    }
    s_from[r] = from;
    s_to[r] = to;
  }
  __syncthreads();
  const int slot = blockIdx.y * blockDim.x + threadIdx.x, slots = gridDim.y * blockDim.x;
  const int first = s_first;
  if (first < m) {
    if (A.mx) {
      accept_part<uint4>(A, A.c.k, 16, 2, s_from, s_to, m, first, slot, slots);
      accept_part<uint4>(A, A.c.v, 16, 2, s_from, s_to, m, first, slot, slots);
      accept_part<uint8_t>(A, A.c.ks, 32, 64, s_from, s_to, m, first, slot, slots);
      accept_part<uint8_t>(A, A.c.vs, 32, 64, s_from, s_to, m, first, slot, slots);
    } else {
      accept_part<uint4>(A, A.c.k, 8, 1, s_from, s_to, m, first, slot, slots);
      accept_part<uint4>(A, A.c.v, 8, 1, s_from, s_to, m, first, slot, slots);
    }
    if (A.weights) {  // a warp a head, 32 entries loaded before they are stored
      const int lane = threadIdx.x & 31;
      for (int h = slot >> 5; h < A.H; h += slots >> 5) {
        float* w = A.weights + i * A.w_seq + h * A.w_head + s.ctx;
        for (int r0 = first; r0 < m; r0 += 32) {
          const int r = r0 + lane;
          float x = 0.f;
          if (r < m) x = w[s_path[m - 1 - r]];
          __syncwarp();
          if (r < m) w[r] = x;
          __syncwarp();
        }
      }
    }
  }
  if (A.W == 1) return;
  // conv_state: row q of the new state is row m + q of (old state ++ path)
  const int64_t si = A.state_indices ? static_cast<int64_t>(__ldg(A.state_indices + i)) : i;
  int64_t pos = 0;
  if (A.state_pos) pos = __ldg(A.state_pos + i);
  if (si < 0 || si >= A.pool || pos < 0) {
    if (lead && threadIdx.x == 0) raise_flag(A.q.err, kFlagStateIndex);
    return;
  }
  const int C = A.H * A.D, keep = A.W - 1;
  for (int x = slot; x < 2 * C / 8; x += slots) {
    const int c = x * 8;
    uint16_t* st = A.state + si * keep * 2 * C + c;
    const uint16_t* raw = c < C ? A.k + c : A.v + (c - C);
    uint4 row[7];
#pragma unroll
    for (int q = 0; q < 7; ++q) {
      if (q >= keep) continue;
      const int at = m + q - keep;  // on the path, or before it
      if (at >= 0)
        row[q] = ld_ro(raw + (s.a + s_path[m - 1 - at]) * A.row_stride);
      else if (!A.state_pos)
        row[q] = *reinterpret_cast<const uint4*>(st + static_cast<int64_t>(m + q) * 2 * C);
    }
#pragma unroll
    for (int q = 0; q < 7; ++q) {
      if (q >= keep) continue;
      const int at = m + q - keep;
      if (A.state_pos) {  // ring: only the path's rows are written
        if (at >= 0)
          *reinterpret_cast<uint4*>(st + ((pos + at) % keep) * 2 * C) = row[q];
      } else {
        *reinterpret_cast<uint4*>(st + static_cast<int64_t>(q) * 2 * C) = row[q];
      }
    }
  }
}

}  // namespace sconv
