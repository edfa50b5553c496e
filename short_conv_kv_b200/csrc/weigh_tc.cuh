// Accumulated attention weights (formulas: weigh.cuh) on the fifth-generation tensor
// cores, for head_dim 64 and 128.
//
// S[key, row] = K Q^T: 128 cache rows are the product's M, the query rows that count (used
// tokens, packed) its N, so ragged row counts cost little padding, and a thread
// owns a key: it adds up its row of S and updates one weight, with no exchange between
// threads and no atomics.  (Up to 16 rows go to weigh.cuh, which has both sides' times.)  Two warpgroups take the tiles in turn, each with its own S in
// tensor memory (256 columns); the products run two tiles ahead.  K comes through the ring of
// tc.cuh; more than 256 rows read it again.  Bound by the bytes of K with few rows, by
// the exponentials with many and, with MXFP8, by the decoding.  Measured: 64 rows over 262,139 MXFP8 tokens
// 137 us (2.1 TB/s of codes), as bf16 105 (5.3 TB/s).
#pragma once
#include "tc.cuh"

namespace sconv {

constexpr int kWeighRows = 256;  // rows of a pass

template <bool MX>
__host__ __device__ constexpr int weigh_tc_threads() {
  return 32 * (8 + (MX ? 8 : 4) + 4);
}

template <int D, bool MX>
__global__ void __launch_bounds__(weigh_tc_threads<MX>(), 1)
    weigh_tc_kernel(const WeighParams W, int q_rows, int ring_units) {
  constexpr int TN = 128, THREADS = weigh_tc_threads<MX>(), kSoft = 256;
  using F = FeedShape<D, TN, MX>;
  grid_dependency_wait();
  allow_dependent_launch();
  const AttendParams& P = W.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_anc[kMaxDraft][kMaskWords];
  __shared__ int s_ptr[kMaxDraft];
  __shared__ __align__(16) float s_lse[kWeighRows];  // lse * log2(e); +inf behind the rows
  __shared__ int s_row[kWeighRows];                  // rows that count
  __shared__ int s_warp[8];
  __shared__ int64_t s_scan[2 * (THREADS / 32)], s_found[2];
  __shared__ uint64_t s_full[8], s_empty[8], s_score[2], s_free[2], s_query, s_drain;
  __shared__ uint64_t s_raw_full[F::kRaw], s_raw_empty[F::kRaw];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort[3], s_rows;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_block = q_rows * 128;
  const uint32_t units = smem + ((q_rows * D * 2 + 1023) & ~1023);
  const uint32_t raw = units + ring_units * F::kUnit;
  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&s_full[i], F::kThreads);
      mbar_init(&s_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_score[i], 1);
      mbar_init(&s_free[i], 128);
    }
    if (MX)
      for (int i = 0; i < F::kRaw; ++i) {
        mbar_init(&s_raw_full[i], 32 * F::kFetchWarps);
        mbar_init(&s_raw_empty[i], F::kThreads);
      }
    mbar_init(&s_query, kSoft);
    mbar_init(&s_drain, 1);
    mbar_init_fence();
    s_abort[0] = s_abort[1] = s_abort[2] = 0;
  }
  if (warp == 0) tmem_alloc(&s_tmem, 512);
  tc_fence_before();
  int64_t cur, end, seq_first;
  int seq, extra = 0;
  find_range<THREADS>(P.s, P.g, P.H, kAllRows, TN, nullptr, blockIdx.x, gridDim.x, s_scan, s_found,
                      cur, end, seq, seq_first, extra);  // barriers inside
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  SeqView sv;
  SeqTiles st;
  int h = 0, t0 = 0, tiles = 0, total = 0, all_rows = 0;
  auto enter = [&] {
    sv = seq_view(P.s, seq, false);
    st = seq_tiles(sv, P.g, P.H, kAllRows, TN);
  };
  auto locate = [&] {
    while (cur >= seq_first + st.all) {
      seq_first += st.all;
      ++seq;
      enter();
    }
    const int64_t rel = cur - seq_first;
    h = static_cast<int>(rel / st.kt);
    t0 = static_cast<int>(rel - static_cast<int64_t>(h) * st.kt);
    tiles = static_cast<int>(min(static_cast<int64_t>(st.kt - t0), end - cur));
    total = sv.ctx + sv.n;
    all_rows = sv.n * P.g;
  };
  if (cur < end) enter();

  if (warp < 8) {
    // ------------------------------------------------------------ sums
    const int stream = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    uint32_t scores = 0;
    int masked_seq = -1;
    bool ok = true;
    auto meet = [&] { asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory"); };
    while (cur < end) {
      locate();
      if (masked_seq != seq) {
        ancestor_masks(P.s, sv, s_anc, s_ptr, t0 == 0 && h == 0, meet);
        masked_seq = seq;
      }
      float* wrow = W.weights + seq * W.w_seq + h * W.w_head;
      for (int row0 = 0; row0 < all_rows; row0 += q_rows) {
        // ---- the rows that count, packed in their order
        {
          const int row = row0 + tid;
          bool counts = false;
          float l = INFINITY;
          if (tid < q_rows && row < all_rows) {
            const int tok = row / P.g;
            if ((s_anc[tok][tok >> 5] >> (tok & 31)) & 1u) {
              l = P.lse[(sv.a + tok) * P.HQ + h * P.g + row - tok * P.g];
              counts = l != -INFINITY;
            }
          }
          const unsigned b = __ballot_sync(kFullMask, counts);
          if (lane == 0) s_warp[warp] = __popc(b);
          meet();
          int at = __popc(b & ((1u << lane) - 1u)), n = 0;
          for (int w = 0; w < 8; ++w) {
            if (w < warp) at += s_warp[w];
            n += s_warp[w];
          }
          if (counts) {
            s_lse[at] = l * kLog2e;
            s_row[at] = row;
          }
          if (tid >= n) s_lse[tid] = INFINITY;
          if (tid == 0) s_rows = n;
          meet();
        }
        const int n = s_rows;
        {
          constexpr int kStep = kSoft / (D / 8);
          const int c = tid % (D / 8);
          const uint16_t* qp =
              P.q + sv.a * P.q_tok + static_cast<int64_t>(h) * P.g * P.q_head + c * 8;
          const int fill = max(16, (n + 15) & ~15);  // rows of the product
          for (int r0 = tid / (D / 8); r0 < fill; r0 += 8 * kStep) {
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = r0 + i * kStep;
              v[i] = make_uint4(0, 0, 0, 0);
              if (rr < n) {
                const int row = s_row[rr], tk = row / P.g;
                v[i] = ld_ro(qp + tk * P.q_tok + (row - tk * P.g) * P.q_head);
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = r0 + i * kStep;
              if (rr < fill)
                sts16(smem + (c >> 3) * q_block + rr * 128 + (((c & 7) ^ (rr & 7)) << 4),
                      tc_order<MX>(v[i]));
            }
          }
        }
        async_proxy_fence();
        mbar_arrive(&s_query);
        const float2 sc = make_float2(P.scale_log2, P.scale_log2);
        for (int t = stream; t < tiles; t += 2) {
          const int p = (t0 + t) * TN + (warp & 3) * 32 + lane;
          const bool fresh = p >= sv.ctx && row0 == 0;  // a drafted row's first pass
          float old = 0.f;
          if (p < total && !fresh) old = wrow[p];
          if (ok) ok = tc_wait(&s_score[stream], scores & 1u, s_abort);
          ok = __all_sync(kFullMask, ok);
          ++scores;
          tc_fence_after();
          if (ok) {
            const uint32_t at = tmem + lanes + stream * kWeighRows;
            const bool tail = (t0 + t + 1) * TN > sv.ctx;
            float2 acc = make_float2(0.f, 0.f), acc2 = make_float2(0.f, 0.f);
            float x[32];
#pragma unroll 1
            for (int c = 0; c < n; c += 32) {
              tmem_ld32(x, at + c);
              tmem_landed(x);
              const bool part = c + 32 > n;
              if (part || tail) {
                const int a = p - sv.ctx;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  bool see = c + e < n;
                  if (see && a >= 0) {
                    const int tok = s_row[c + e] / P.g;
                    see = a < sv.n && ((s_anc[tok][a >> 5] >> (a & 31)) & 1u);
                  }
                  const float y = see ? ex2(fmaf(x[e], P.scale_log2, -s_lse[c + e])) : 0.f;
                  acc.x += y;
                }
              } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  const float4 l = *reinterpret_cast<const float4*>(s_lse + c + e);
                  float2 y = ffma2(make_float2(x[e], x[e + 1]), sc, make_float2(-l.x, -l.y));
                  float2 z = ffma2(make_float2(x[e + 2], x[e + 3]), sc, make_float2(-l.z, -l.w));
                  y.x = ex2(y.x);
                  y.y = ex2(y.y);
                  z.x = ex2(z.x);
                  z.y = ex2(z.y);
                  acc = __fadd2_rn(acc, y);
                  acc2 = __fadd2_rn(acc2, z);
                }
              }
            }
            if (p < total) wrow[p] = old + ((acc.x + acc.y) + (acc2.x + acc2.y));
          }
          tc_fence_before();
          mbar_arrive(&s_free[stream]);
        }
        meet();  // Q, its lse and the masks are free
      }
      cur += tiles;
    }
    if (!ok && lane == 0) raise_flag(P.s.err, kFlagTimeout);
  } else if (warp < 8 + F::kWarps) {
    // ------------------------------------------------------------ producers
    const int w = warp - 8;
    FeedRing R{units, s_full, s_empty, s_abort, ring_units};
    if constexpr (MX) {
      FeedRing Raw{raw, s_raw_full, s_raw_empty, s_abort, F::kRaw};
      while (cur < end) {
        locate();
        const int64_t head = h * P.s.stride_head >> 5;
        const int low = P.c.words ? reinterpret_cast<uintptr_t>(P.c.ks + head) & 3 : 0;
        const int64_t units_all = static_cast<int64_t>((all_rows + q_rows - 1) / q_rows) * tiles;
#pragma unroll 1
        for (int64_t u = 0; u < units_all; ++u)
          FeedMx<D, TN>::decode(R, Raw, w, lane, low, TN);
        cur += tiles;
      }
    } else {
      while (cur < end) {
        locate();
        const uint8_t* kb = P.c.k + h * P.s.stride_head * 2;
        const int32_t* table = P.s.table + seq * P.s.table_stride;
        const int key0 = t0 * TN + w * F::kKeysWarp + lane % F::kKeysWarp;
        const int64_t units_all = static_cast<int64_t>((all_rows + q_rows - 1) / q_rows) * tiles;
        int page = __ldg(table + page_index(P.s, min(key0, total - 1)));
        int t = 0;
#pragma unroll 1
        for (int64_t u = 0; u < units_all; ++u) {
          const uint32_t off = paged_off8(P.s, page, key0 + t * TN, total);
          t = t + 1 == tiles ? 0 : t + 1;
          page = __ldg(table + page_index(P.s, min(key0 + t * TN, total - 1)));
          FeedBf16<D, TN>::bring(R, w, lane, kb, off, TN);
        }
        cur += tiles;
      }
      cp_commit();
      cp_wait<0>();
    }
  } else if (warp == 8 + F::kWarps) {
    // ------------------------------------------------------------ products
    uint32_t queries = 0, used[2] = {0, 0};
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t count) {
      if (ok) ok = tc_wait(bar, count & 1u, s_abort);
      ok = __all_sync(kFullMask, ok);
    };
    const uint32_t keys = tc_desc(units, 16), query = tc_desc(smem, 16);
    while (cur < end && ok) {
      locate();
      for (int row0 = 0; row0 < all_rows && ok; row0 += q_rows) {
        wait(&s_query, queries++);
        const int n = *reinterpret_cast<volatile int*>(&s_rows);
        const uint32_t idesc = tc_idesc(128, max(16, (n + 15) & ~15), false);
        for (int t = 0; t < tiles && ok; ++t) {
          const int b = t & 1;
          wait(&s_full[slot], phase);
          async_proxy_fence();
          if (used[b]) wait(&s_free[b], used[b] - 1);  // the tile before in this buffer is summed
          ++used[b];
          tc_fence_after();
          const uint32_t k = keys + slot * (F::kUnit >> 4), to = tmem + b * kWeighRows;
          if (ok && elect_one()) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
              tc_mma(to, k + (((j >> 2) * (TN * 128) + (j & 3) * 32) >> 4),
                     query + (((j >> 2) * q_block + (j & 3) * 32) >> 4), idesc, j > 0);
            tc_commit(&s_score[b]);
            tc_commit(&s_empty[slot]);
          }
          __syncwarp();
          if (++slot == ring_units) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      cur += tiles;
    }
    if (elect_one()) tc_commit(&s_drain);
    __syncwarp();
    int dummy[1] = {0};
    if (!mbar_wait(&s_drain, 0, dummy, kDrainTimeoutNs)) ok = false;
    if (!ok && lane == 0) raise_flag(P.s.err, kFlagTimeout);
  } else if constexpr (MX) {
    // ------------------------------------------------------------ raw units
    using M = FeedMx<D, TN>;
    const int w = warp - (8 + F::kWarps + 1);
    FeedRing Raw{raw, s_raw_full, s_raw_empty, s_abort, F::kRaw};
    while (cur < end) {
      locate();
      const int64_t head = h * P.s.stride_head;
      const int32_t* table = P.s.table + seq * P.s.table_stride;
      const int key0 = t0 * TN + w * 8 + (lane >> 2);
      const int64_t units_all = static_cast<int64_t>((all_rows + q_rows - 1) / q_rows) * tiles;
      int page[M::kMine];
      auto pages = [&](int t) {
#pragma unroll
        for (int i = 0; i < M::kMine; ++i)
          page[i] = __ldg(table + page_index(P.s, min(key0 + t * TN + i * M::kStep, total - 1)));
      };
      pages(0);
      int t = 0;
#pragma unroll 1
      for (int64_t u = 0; u < units_all; ++u) {
        uint32_t off[M::kMine];
#pragma unroll
        for (int i = 0; i < M::kMine; ++i) {
          const uint32_t o = paged_off8(P.s, page[i], key0 + t * TN + i * M::kStep, total);
          off[i] = o == ~0u ? 0 : o;
        }
        const int left = total - (t0 + t) * TN;
        t = t + 1 == tiles ? 0 : t + 1;
        pages(t);
        M::fetch(Raw, w, lane, P.c.k + head, P.c.ks + (head >> 5), P.c.words, off, left);
      }
      cur += tiles;
    }
    cp_commit();
    cp_wait<0>();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, 512);
}

}  // namespace sconv
