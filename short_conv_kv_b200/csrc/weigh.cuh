// Accumulated attention weights of the cache's rows (sm_100a): for every
// position p of sequence i and K/V head h
//     add = sum over used drafted tokens j that see p, and the head's query
//           heads, of exp(scale * q . k_p - lse)
//     weights[i, h, p] += add   (p < ctx),   = add   (a drafted token's row)
// with the lse that the attention left.  This kernel is for up to 16 query rows
// a K/V head (64 decode steps over 2355 tokens: 82 us, 3.9 TB/s, weigh_tc.cuh 124; 64 rows over 262,139
// MXFP8 tokens: 312 us against 137), and for head_dim 256, where a unit of weigh_tc.cuh's ring would take
// 64 KB.  S^T[key, row] = K Q^T: 16 keys a warp
// and step are the m16 of the matrix instruction, straight from global memory (as
// in attend_rows_kernel), the query rows its n8 from shared memory, so few
// rows cost no padding; a key's sum over the rows stays in one lane
// group and is added to memory once.  Every position belongs to one warp:
// no atomics, and the same call gives the same bits.
#pragma once
#include "attend.cuh"

namespace sconv {

template <int D>
constexpr int kWeighRowsQ = D == 256 ? 64 : 16;  // rows of Q in shared memory

template <int D, bool MX>
__global__ void __launch_bounds__(32 * kWeighWarps, D == 256 ? 2 : 4)
    weigh_kernel(const WeighParams W) {
  using L = RowsLayout<D, MX>;
  constexpr int THREADS = 32 * kWeighWarps, KV = L::kKVec, RC = kWeighRowsQ<D>;
  constexpr int kTile = 16 * kWeighWarps;
  grid_dependency_wait();
  allow_dependent_launch();
  const AttendParams& P = W.a;
  extern __shared__ __align__(16) uint8_t smem[];  // Q
  __shared__ uint32_t s_anc[kMaxDraft][kMaskWords];
  __shared__ int s_ptr[kMaxDraft];
  __shared__ __align__(16) float s_lse[RC];  // lse * log2(e); +inf for a row that counts nothing
  __shared__ int s_tok[RC];
  __shared__ int64_t s_scan[2 * (THREADS / 32)], s_found[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lr = lane >> 2, lc = lane & 3;
  int64_t cur, end, seq_first;
  int seq, extra = 0;
  find_range<THREADS>(P.s, P.g, P.H, kAllRows, kTile, nullptr, blockIdx.x, gridDim.x, s_scan,
                      s_found, cur, end, seq, seq_first, extra);
  if (cur >= end) return;
  int masked_seq = -1;
  SeqView sv = seq_view(P.s, seq, false);
  SeqTiles st = seq_tiles(sv, P.g, P.H, kAllRows, kTile);
  while (cur < end) {
    while (cur >= seq_first + st.all) {
      seq_first += st.all;
      ++seq;
      sv = seq_view(P.s, seq, false);
      st = seq_tiles(sv, P.g, P.H, kAllRows, kTile);
    }
    const int64_t rel = cur - seq_first;
    const int h = static_cast<int>(rel / st.kt);
    const int t0 = static_cast<int>(rel - static_cast<int64_t>(h) * st.kt);
    const int t1 = static_cast<int>(min(static_cast<int64_t>(st.kt), t0 + (end - cur)));
    const int all_rows = sv.n * P.g, total = sv.ctx + sv.n;
    const int key1 = min(total, t1 * kTile);
    if (masked_seq != seq) {
      ancestor_masks(P.s, sv, s_anc, s_ptr, t0 == 0 && h == 0);
      masked_seq = seq;
    }
    const uint8_t* kb = P.c.k + h * P.s.stride_head * (MX ? 1 : 2);
    const uint8_t* ksb = MX ? P.c.ks + (h * P.s.stride_head >> 5) : nullptr;
    const int32_t* table = P.s.table + seq * P.s.table_stride;
    float* wrow = W.weights + seq * W.w_seq + h * W.w_head;

    for (int row0 = 0; row0 < all_rows; row0 += RC) {
      const int rows = min(RC, all_rows - row0), ntiles = (rows + 7) >> 3;
      for (int x = tid; x < ntiles * 8 * (D / 8); x += THREADS) {
        const int r = x / (D / 8), d = (x - r * (D / 8)) * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows) {
          const int tok = (row0 + r) / P.g, hg = row0 + r - tok * P.g;
          if ((s_anc[tok][tok >> 5] >> (tok & 31)) & 1u)
            v = ld_ro(P.q + (sv.a + tok) * P.q_tok + (h * P.g + hg) * P.q_head + d);
        }
        *reinterpret_cast<uint4*>(smem + r * L::kQPitch + d * 2) = v;
      }
      for (int r = tid; r < ntiles * 8; r += THREADS) {
        float l = INFINITY;
        int tok = -1;
        if (r < rows) {
          tok = (row0 + r) / P.g;
          if ((s_anc[tok][tok >> 5] >> (tok & 31)) & 1u) {
            const float x = P.lse[(sv.a + tok) * P.HQ + h * P.g + row0 + r - tok * P.g];
            if (x != -INFINITY) l = x * kLog2e;
          } else {
            tok = -1;
          }
        }
        s_lse[r] = l;
        s_tok[r] = tok;
      }
      __syncthreads();

      uint4 kreg[2][KV];
      uint64_t ksc[2] = {0, 0};
      auto page_at = [&](int b) {
        return __ldg(table + page_index(P.s, min(b + (lane & 15), total - 1)));
      };
      auto off_at = [&](int b, int page) -> uint32_t {
        const int p = min(b + (lane & 15), total - 1);
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(P.s.num_pages)) {
          if (b < key1) raise_flag(P.s.err, kFlagSlotRange);
          page = 0;
        }
        return row_off8(P.s, page, p);
      };
      auto load_k = [&](uint32_t off8) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint64_t o8 = __shfl_sync(kFullMask, off8, t * 8 + lr);
          const uint8_t* p = kb + o8 * (MX ? 8 : 16) + lc * 16;
#pragma unroll
          for (int k = 0; k < KV; ++k) kreg[t][k] = ld_stream(p + k * 64);
          if constexpr (MX) ksc[t] = ld_scales<D>(ksb + (o8 >> 2), P.c.ks_packed);
        }
      };
      const int step = kTile;
      int base = t0 * kTile + warp * 16;
      uint32_t off_next = 0;
      if (base < key1) {
        load_k(off_at(base, page_at(base)));
        off_next = off_at(base + step, page_at(base + step));
      }
      for (; base < key1; base += step) {
        // the keys as bf16 fragments: kk[t] holds 8 dims of keys lr and lr + 8
        uint4 kk[2][D / 32];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < D / 32; ++t) {
            if constexpr (MX) {
              const uint4 raw = kreg[u][t >> 1];
              const uint32_t sc = e8m0_bf16x2(
                  static_cast<uint32_t>(ksc[u] >> (8 * ((t >> 1) * 2 + (lc >> 1)))) & 255u);
              e4m3x4_bf16((t & 1) ? raw.z : raw.x, sc, kk[u][t].x, kk[u][t].y);
              e4m3x4_bf16((t & 1) ? raw.w : raw.y, sc, kk[u][t].z, kk[u][t].w);
            } else {
              kk[u][t] = kreg[u][t];
            }
          }
        if (base + step < key1) {
          load_k(off_next);
          off_next = off_at(base + 2 * step, page_at(base + 2 * step));
        }
        const bool tail = base + 16 > sv.ctx;
        float add[2] = {0.f, 0.f};
#pragma unroll 2
        for (int nt = 0; nt < ntiles; ++nt) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
          const uint8_t* qp = smem + (nt * 8 + lr) * L::kQPitch;
#pragma unroll
          for (int t = 0; t < D / 32; ++t) {
            const uint4 q = *reinterpret_cast<const uint4*>(qp + q_dim<MX>(t, lc) * 2);
            mma_bf16(c, kk[0][t].x, kk[1][t].x, kk[0][t].y, kk[1][t].y, q.x, q.y);
            mma_bf16(c, kk[0][t].z, kk[1][t].z, kk[0][t].w, kk[1][t].w, q.z, q.w);
          }
          const float2 l = *reinterpret_cast<const float2*>(s_lse + nt * 8 + 2 * lc);
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float le = (e & 1) ? l.y : l.x;
            p[e] = le == INFINITY ? 0.f : ex2(fmaf(c[e], P.scale_log2, -le));
          }
          if (tail) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int a = base + lr + (e >> 1) * 8 - sv.ctx;
              const int tok = s_tok[nt * 8 + 2 * lc + (e & 1)];
              if (a >= 0 &&
                  !(tok >= 0 && a < sv.n && ((s_anc[tok][a >> 5] >> (a & 31)) & 1u)))
                p[e] = 0.f;
            }
          }
          add[0] += p[0] + p[1];
          add[1] += p[2] + p[3];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          add[u] += __shfl_xor_sync(kFullMask, add[u], 1);
          add[u] += __shfl_xor_sync(kFullMask, add[u], 2);
          const int p = base + lr + u * 8;
          if (lc == 0 && p < total)
            wrow[p] = (p < sv.ctx || row0 > 0) ? wrow[p] + add[u] : add[u];
        }
      }
      __syncthreads();
    }
    cur += t1 - t0;
  }
}

}  // namespace sconv
