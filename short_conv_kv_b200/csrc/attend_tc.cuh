// Attention of drafted-tree queries for many query rows, on the fifth-generation
// tensor cores.  Formulas, units, ranges and the join are those of attend.cuh.
//
// A unit is up to kStreams * 128 rows of one K/V head.  Two streams of
// softmax warps (128 rows each, a thread a row) take turns with the
// tensor cores, so that one computes exponentials while the other's products run:
//   pair       more than 128 rows: stream s has rows 128 s ..; both use every
//              K/V tile, which is brought (and, for MXFP8, decoded) once
//   alternate  up to 128 rows: stream s has the key tiles of parity s, with a
//              maximum, sum and output of its own, merged at the end
// (D = 256: one stream, and two score tiles that alternate.)
// S = Q K^T lands in tensor memory, the softmax warps read it, write the
// probabilities back over it as bf16, and O += P V takes them from there.  O
// stays in tensor memory and is rescaled only when a row's maximum has grown by
// more than 2^8.  Tensor memory holds just two S and two O tiles of 128
// columns, which is what sets two streams and 128 keys a tile.
#pragma once
#include "tc.cuh"

namespace sconv {

template <int D>
struct TcShape {
  static constexpr int kKeys = D == 256 ? 64 : 128;
  static constexpr int kStreams = D == 256 ? 1 : 2;
  static constexpr int kSoftWarps = 4 * kStreams;
  static constexpr uint32_t kOut = D == 256 ? 2 * kKeys : 256;  // first column of O
};
template <int D, bool MX>
__host__ __device__ constexpr int tc_threads() {
  return 32 * (TcShape<D>::kSoftWarps + Feed<D, TcShape<D>::kKeys, MX>::kWarps + 1);
}

// Bits a0 .. a0+31 of the row's view of the keys behind the context: a < 0
// (context) is seen, a draft where its bit is set.
__device__ __forceinline__ uint32_t seen32(const uint32_t* anc, int a0, bool used) {
  if (!used) return 0u;
  if (a0 <= -32) return ~0u;
  if (a0 < 0) return (anc[0] << -a0) | ((1u << -a0) - 1u);
  if (a0 >= kMaxDraft) return 0u;
  const int w = a0 >> 5, sh = a0 & 31;
  const uint32_t lo = anc[w], hi = w + 1 < kMaskWords ? anc[w + 1] : 0u;
  return __funnelshift_r(lo, hi, sh);
}

template <int D, bool MX>
__global__ void __launch_bounds__(tc_threads<D, MX>(), 1)
    attend_tc_kernel(const AttendParams P, int rows_unit, int ring_units) {
  using T = TcShape<D>;
  using F = Feed<D, T::kKeys, MX>;
  constexpr int TN = T::kKeys, NS = T::kStreams, THREADS = tc_threads<D, MX>();
  constexpr int kSoft = 32 * T::kSoftWarps;
  constexpr uint32_t kQTile = 128 * D * 2, kQBlock = 128 * 128;
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_anc[kMaxDraft][kMaskWords];
  __shared__ int s_ptr[kMaxDraft];
  __shared__ float2 s_ml[2][128];
  __shared__ int64_t s_scan[THREADS / 32], s_found[2];
  __shared__ uint64_t s_full[8], s_empty[8], s_score[2], s_prob[2], s_out[2], s_query, s_drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort[2];  // a wait ran out; a V row was cleaned
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t units = smem + (rows_unit > 128 || NS == 1 ? NS : 1) * kQTile;
  const uint32_t raw = units + ring_units * F::kUnit;

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&s_full[i], F::kThreads);
      mbar_init(&s_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_score[i], 1);
      mbar_init(&s_prob[i], 128);
      mbar_init(&s_out[i], 1);
    }
    mbar_init(&s_query, kSoft);
    mbar_init(&s_drain, 1);
    mbar_init_fence();
    s_abort[0] = s_abort[1] = 0;
  }
  if (warp == 0) tmem_alloc(&s_tmem, 512);
  tc_fence_before();
  int64_t cur, end, seq_first;
  int seq;
  find_range<THREADS>(P.s, P.g, P.H, rows_unit, TN, P.prefix, blockIdx.x, gridDim.x, s_scan,
                      s_found, cur, end, seq, seq_first);  // barriers inside
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // Every role walks the same segments.
  SeqView sv;
  SeqTiles st;
  int h = 0, row0 = 0, rows = 0, t0 = 0, tiles = 0, total = 0;
  bool pair = false;
  auto enter = [&] {
    sv = seq_view(P.s, seq, false);
    st = seq_tiles(sv, P.g, P.H, rows_unit, TN);
  };
  auto locate = [&] {
    while (cur >= seq_first + st.all) {  // the next sequence with tiles
      seq_first += st.all;
      ++seq;
      enter();
    }
    const int64_t rel = cur - seq_first;
    const int unit = static_cast<int>(rel / st.kt);
    t0 = static_cast<int>(rel - static_cast<int64_t>(unit) * st.kt);
    tiles = static_cast<int>(min(static_cast<int64_t>(st.kt - t0), end - cur));
    h = unit / st.mt;
    row0 = (unit - h * st.mt) * rows_unit;
    rows = min(rows_unit, sv.n * P.g - row0);
    total = sv.ctx + sv.n;
    pair = NS == 2 && rows > 128;
  };
  if (cur < end) enter();

  if (warp < T::kSoftWarps) {
    // ------------------------------------------------------------- softmax
    const int stream = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's lanes
    const int r = (warp & 3) * 32 + lane;                          // row of the stream's tile
    const float scale = fabsf(P.scale_log2);
    const uint32_t flip = P.scale_log2 < 0.f ? 0x80008000u : 0u;  // the sign goes to Q
    uint32_t seen_scores[2] = {0, 0}, seen_outs[2] = {0, 0};
    int segment = 0, masked_seq = -1;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t count) {  // until its phase `count` is complete
      if (ok) ok = mbar_wait(bar, count & 1u, s_abort, kTcTimeoutNs);
      ok = __all_sync(kFullMask, ok);
    };
    auto meet = [&] { asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory"); };
    while (cur < end) {
      locate();
      if (masked_seq != seq) {
        ancestor_masks(P.s, sv, s_anc, s_ptr, t0 == 0 && h == 0 && row0 == 0, meet);
        masked_seq = seq;
      }
      // ---- Q, rows of both streams
      for (int x = tid; x < rows * (D / 8); x += kSoft) {
        const int rr = x / (D / 8), c = x - rr * (D / 8);
        const int tok = (row0 + rr) / P.g, hg = row0 + rr - tok * P.g;
        uint4 v = ld_ro(P.q + (sv.a + tok) * P.q_tok + (h * P.g + hg) * P.q_head + c * 8);
        v.x ^= flip;
        v.y ^= flip;
        v.z ^= flip;
        v.w ^= flip;
        sts16(smem + (rr >> 7) * kQTile + (c >> 3) * kQBlock + (rr & 127) * 128 +
                  (((c & 7) ^ (rr & 7)) << 4),
              v);
      }
      async_proxy_fence();
      mbar_arrive(&s_query);

      const int mine = pair ? stream * 128 + r : r;  // row of the unit
      const int tok = mine < rows ? (row0 + mine) / P.g : 0;
      const bool used = mine < rows && ((s_anc[tok][tok >> 5] >> (tok & 31)) & 1u);
      const bool busy = (pair ? stream * 128 : 0) + (warp & 3) * 32 < rows;  // any row here
      float mx = -INFINITY, sum = 0.f;
      const int t_first = pair || NS == 1 ? 0 : stream, t_step = pair || NS == 1 ? 1 : 2;
      for (int t = t_first; t < tiles; t += t_step) {
        const int b = NS == 1 ? t & 1 : stream;
        wait(&s_score[b], seen_scores[b]++);
        tc_fence_after();
        if (busy && ok) {
          const uint32_t at = tmem + lanes + b * TN;
          const int a0 = (t0 + t) * TN - sv.ctx;
          const bool tail = a0 + TN > 0;
          float x[32];
          float m = -INFINITY;
#pragma unroll
          for (int c = 0; c < TN / 32; ++c) {
            tmem_ld32(x, at + c * 32);
            tmem_landed(x);
            if (tail) {
              const uint32_t vis = seen32(s_anc[tok], a0 + c * 32, used);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = (vis >> e) & 1u ? x[e] : -INFINITY;
            }
            float m0 = x[0], m1 = x[1];
#pragma unroll
            for (int e = 2; e < 32; e += 4) {
              m0 = fmaxf(m0, fmaxf(x[e], x[e + 1]));
              if (e + 2 < 32) m1 = fmaxf(m1, fmaxf(x[e + 2], x[e + 3]));
            }
            m = fmaxf(m, fmaxf(m0, m1));
          }
          m = m == -INFINITY ? m : m * scale;
          const bool grow = m > mx + 8.f;  // true at the first finite score
          if (__any_sync(kFullMask, grow)) {
            const float to = grow ? m : mx;
            const float w = merge_weight(mx, to);
            mx = to;
            sum *= w;
            if (t >= (NS == 1 ? 1 : t_first + t_step)) {
              // O holds the tiles before: complete with this S, or (one stream)
              // with the last product
              if (NS == 1) wait(&s_out[(t - 1) & 1], seen_outs[(t - 1) & 1] + ((t - 1) >> 1));
              tc_fence_after();
              const uint32_t o = tmem + lanes + T::kOut + (NS == 1 ? 0 : stream) * D;
              if (ok) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  tmem_ld32(x, o + c);
                  tmem_landed(x);
#pragma unroll
                  for (int e = 0; e < 32; ++e) x[e] *= w;
                  tmem_st32(o + c, x);
                }
              }
            }
          }
          const float base = mx == -INFINITY ? 0.f : mx;
          const float2 sc = make_float2(scale, scale), nb = make_float2(-base, -base);
          float2 acc = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < TN / 32; ++c) {
            tmem_ld32(x, at + c * 32);
            tmem_landed(x);
            uint32_t vis = ~0u;
            if (tail) vis = seen32(s_anc[tok], a0 + c * 32, used);
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 y = ffma2(make_float2(x[2 * e], x[2 * e + 1]), sc, nb);
              if (tail) {
                y.x = (vis >> (2 * e)) & 1u ? y.x : -INFINITY;
                y.y = (vis >> (2 * e + 1)) & 1u ? y.y : -INFINITY;
              }
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              acc = __fadd2_rn(acc, y);
              p[e] = pack_bf16x2(y);
            }
            tmem_st16(at + c * 16, p);
          }
          sum += acc.x + acc.y;
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&s_prob[b]);
      }
      // ---- the results: wait for the last products
      {
        const uint32_t n0 = pair ? tiles : (tiles + 1) >> 1, n1 = pair ? tiles : tiles >> 1;
        // this stream's first: its last product was issued behind all but the
        // other's last one, so neither wait can meet an older phase
        if (stream == 0) wait(&s_out[0], seen_outs[0] + n0 - 1);
        if ((!pair || stream == 1) && n1) wait(&s_out[1], seen_outs[1] + n1 - 1);
        if (stream == 1 && !pair) wait(&s_out[0], seen_outs[0] + n0 - 1);
        seen_outs[0] += n0;
        seen_outs[1] += n1;
        tc_fence_after();
      }
      float f0 = 1.f, f1 = 0.f;  // weights of the streams' outputs
      if (NS == 2 && !pair) {
        s_ml[stream][r] = make_float2(mx, sum);
        meet();
        const float2 a = s_ml[0][r], c = s_ml[1][r];
        mx = fmaxf(a.x, c.x);
        f0 = merge_weight(a.x, mx);
        f1 = merge_weight(c.x, mx);
        // (a side that saw nothing has weight 0, and 0 as its sum; NaN sums stay)
        sum = (a.y == 0.f ? 0.f : a.y * f0) + (c.y == 0.f ? 0.f : c.y * f1);
        if (a.x == -INFINITY && a.y != 0.f) sum = a.y;  // only NaN
        if (c.x == -INFINITY && c.y != 0.f) sum = c.y;
      }
      const bool whole = t0 == 0 && tiles == st.kt;
      if (busy && ok) {
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (segment ? 1 : 0);
        const int hq = h * P.g + row0 + mine - tok * P.g;
        const bool halves = NS == 2 && !pair;
        const int d0 = halves ? stream * (D / 2) : 0, d1 = halves ? d0 + D / 2 : D;
        const uint32_t o = tmem + lanes + T::kOut + (pair ? stream * D : 0);
        const float inv = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        const bool none = !used;
        const int key1 = min(total, (t0 + tiles) * TN);
        const bool bad = *reinterpret_cast<volatile int*>(&s_abort[1]);
#pragma unroll 1
        for (int d = d0; d < d1; d += 32) {
          float x[32];
          tmem_ld32(x, o + d);
          tmem_landed(x);
          if (halves) {
            if (tiles > 1) {
              float y[32];
              tmem_ld32(y, o + D + d);
              tmem_landed(y);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = fmaf(y[e], f1, x[e] * f0);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] *= f0;
            }
          }
          if (mine < rows) {
            if (bad)
              for (int e = 0; e < 32; ++e)
                x[e] = restore_nonfinite<MX>(P, seq, sv.ctx, sv.n, h, s_anc[tok], t0 * TN, key1,
                                             d + e, x[e]);
            if (whole) {
              uint16_t* to = P.out + (sv.a + tok) * P.o_tok + hq * P.o_head + d;
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint4 v;
                v.x = pack_bf16x2(make_float2(x[e] * inv, x[e + 1] * inv));
                v.y = pack_bf16x2(make_float2(x[e + 2] * inv, x[e + 3] * inv));
                v.z = pack_bf16x2(make_float2(x[e + 4] * inv, x[e + 5] * inv));
                v.w = pack_bf16x2(make_float2(x[e + 6] * inv, x[e + 7] * inv));
                if (none) v = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(to + e) = v;
              }
            } else {
              float* to = P.part_o + (slot * rows_unit + mine) * D + d;
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(to + e) =
                    none ? make_float4(0.f, 0.f, 0.f, 0.f)
                         : make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
          }
        }
        if (mine < rows && d0 == 0) {
          const float l = none ? 0.f : sum;
          if (!whole)
            P.part_ml[slot * rows_unit + mine] = make_float2(none ? -INFINITY : mx, l);
          else if (P.lse)
            P.lse[(sv.a + tok) * P.HQ + hq] = l == 0.f ? -INFINITY : (mx + log2f(l)) * kLn2;
        }
      }
      tc_fence_before();
      meet();  // Q, the masks, O and s_ml are free
      cur += tiles;
      ++segment;
    }
    if (!ok && lane == 0) raise_flag(P.s.err, kFlagTimeout);
  } else if (warp < T::kSoftWarps + F::kWarps) {
    // ------------------------------------------------------------ producers
    F feed;
    {
      FeedRing R;
      R.units = units;
      R.raw = raw + (tid - kSoft) * 16;
      R.full = s_full;
      R.empty = s_empty;
      R.abort = s_abort;
      R.count = ring_units;
      feed.init(R, tid - kSoft);
    }
    while (cur < end) {
      locate();
      const int64_t head = h * P.s.stride_head;
      const uint8_t* kb = P.c.k + head * (MX ? 1 : 2);
      const uint8_t* vb = P.c.v + head * (MX ? 1 : 2);
      const uint8_t* ksb = MX ? P.c.ks + (head >> 5) : nullptr;
      const uint8_t* vsb = MX ? P.c.vs + (head >> 5) : nullptr;
      const int32_t* table = P.s.table + seq * P.s.table_stride;
      const int key0 = t0 * TN + feed.my_key();
      auto page_at = [&](int t) { return __ldg(table + page_index(P.s, min(key0 + t * TN, total - 1))); };
      auto off_at = [&](int t, int page) -> uint32_t {
        const int p = key0 + t * TN;
        if (p >= total) return ~0u;
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(P.s.num_pages)) {
          raise_flag(P.s.err, kFlagSlotRange);
          page = 0;
        }
        return static_cast<uint32_t>(row_offset(P.s, page, p) >> 3);
      };
      auto clean_from = [&](int t) { return max(0, min(TN, sv.ctx - (t0 + t) * TN)); };
      uint32_t off0 = off_at(0, page_at(0));
      int page = page_at(1);
      feed.bring(kb, ksb, off0, TN);
      for (int t = 0; t < tiles; ++t) {
        const uint32_t off1 = off_at(t + 1, page);
        page = page_at(t + 2);
        if (!pair && t + 1 < tiles) feed.bring(kb, ksb, off1, TN);
        feed.bring(vb, vsb, off0, clean_from(t));
        if (pair && t + 1 < tiles) feed.bring(kb, ksb, off1, TN);
        off0 = off1;
      }
      cur += tiles;
    }
    feed.finish();
  } else if (lane == 0) {
    // ------------------------------------------------------------- products
    constexpr uint32_t kIdS = tc_idesc(128, TN, false), kIdO = tc_idesc(128, D, true);
    constexpr uint32_t kBlock = TN * 128;  // 64 columns of a unit
    uint32_t probs[2] = {0, 0}, queries = 0;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t count) {
      if (ok) ok = mbar_wait(bar, count & 1u, s_abort, kTcTimeoutNs);
    };
    auto next = [&] {
      if (++slot == ring_units) {
        slot = 0;
        phase ^= 1;
      }
    };
    auto score = [&](int b, int stream) {  // S[b] = Q K^T with the unit in `slot`
      if (!ok) return;
      const uint32_t q = smem + stream * kQTile, k = units + slot * F::kUnit;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        tc_mma(tmem + b * TN, tc_desc(q + (j >> 2) * kQBlock + (j & 3) * 32, 16),
               tc_desc(k + (j >> 2) * kBlock + (j & 3) * 32, 16), kIdS, j > 0);
      tc_commit(&s_score[b]);
    };
    auto output = [&](int b, int stream, bool first) {  // O += P V
      if (!ok) return;
      const uint32_t v = units + slot * F::kUnit;
#pragma unroll
      for (int j = 0; j < TN / 16; ++j)
        tc_mma_tmem(tmem + T::kOut + stream * D, tmem + b * TN + j * 8,
                    tc_desc(v + j * 2048, kBlock), kIdO, !first || j > 0);
      tc_commit(&s_out[b]);
    };
    auto free_unit = [&] {
      if (ok) tc_commit(&s_empty[slot]);
      next();
    };
    while (cur < end && ok) {
      locate();
      wait(&s_query, queries++);
      if (pair) {
        wait(&s_full[slot], phase);
        tc_fence_after();
        score(0, 0);
        score(1, 1);
        free_unit();
        for (int t = 0; t < tiles && ok; ++t) {
          const bool more = t + 1 < tiles;
          const int v_slot = slot;
          const uint32_t v_phase = phase;
          int k_slot = slot + 1;
          uint32_t k_phase = phase;
          if (k_slot == ring_units) {
            k_slot = 0;
            k_phase ^= 1;
          }
          for (int s = 0; s < 2; ++s) {
            wait(&s_prob[s], probs[s]++);
            slot = v_slot;
            if (s == 0) wait(&s_full[v_slot], v_phase);
            tc_fence_after();
            output(s, s, t == 0);
            if (s == 1 && ok) tc_commit(&s_empty[v_slot]);
            if (more) {
              slot = k_slot;
              if (s == 0) wait(&s_full[k_slot], k_phase);
              tc_fence_after();
              score(s, s);
              if (s == 1 && ok) tc_commit(&s_empty[k_slot]);
            }
          }
          slot = v_slot;
          phase = v_phase;
          next();
          if (more) next();
        }
      } else {
        for (int t = 0; t < 2 && t < tiles; ++t) {
          wait(&s_full[slot], phase);
          tc_fence_after();
          score(t, 0);
          free_unit();
        }
        for (int t = 0; t < tiles && ok; ++t) {
          const int b = t & 1;
          wait(&s_prob[b], probs[b]++);
          wait(&s_full[slot], phase);
          tc_fence_after();
          output(b, NS == 2 ? b : 0, t < NS);
          free_unit();
          if (t + 2 < tiles) {
            wait(&s_full[slot], phase);
            tc_fence_after();
            score(b, 0);
            free_unit();
          }
        }
      }
      cur += tiles;
    }
    // products still under way would write to freed tensor memory
    tc_commit(&s_drain);
    int dummy[1] = {0};
    if (!mbar_wait(&s_drain, 0, dummy, kDrainTimeoutNs)) ok = false;
    if (!ok) raise_flag(P.s.err, kFlagTimeout);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, 512);
}

}  // namespace sconv
