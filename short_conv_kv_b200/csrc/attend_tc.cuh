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
// Measured: 32 rows over 1,048,573 tokens 640 to 700 us in short runs (6.2 to 6.7 TB/s; bound by the bytes of K/V),
// 780 to 830 in long ones at the power limit, MXFP8 950 to 1000 (2.3 TB/s: the decoding); 32 ragged trees of 8 to 64
// rows 150 to 159 us (a unit's beginning and end); 384 to 512 rows over 12 to 20 thousand MXFP8 tokens 412 to 438 us
// (the decoding), as bf16 327 to 392.  (Ranges: several boxes.)
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
// Softmax warpgroups, producers, and a warpgroup of which one warp issues the
// products.  Two softmax warpgroups get more registers than an even share:
// with 16 warps of 128 launched, 2 * 184 + 2 * 72 = 4 * 128; with 20 warps
// of 96 (MXFP8), 2 * 136 + 2 * 64 + 80 = 5 * 96.
template <int D, bool MX>
__host__ __device__ constexpr int tc_threads() {
  return 32 * (TcShape<D>::kSoftWarps + FeedShape<D, TcShape<D>::kKeys, MX>::kWarps + 4);
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A unit's beginning and end (masks, queries, the first copies, the output), in tiles: a
// range with many short contexts gets fewer of their tiles (32 ragged ones: 179 us
// without, 169 with).
constexpr int kUnitExtra = 5;

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

// Scores (times log2(e)) from 2^24 on lie 1 or more apart.  The softmax passes subtract a rounded maximum from
// products that are not, which is then off by as much (from about 2^30 on the largest may come out as 0 or
// infinite), and handling that in the passes costs 3 to 10 % of every call.  So a row whose maximum says that
// it has met such scores is done again from the cache when its unit ends: rare, a thread a row, out of line, 0 to
// 1.5 % for the calls that do not need it.  (All of 32 rows over 1,048,573 tokens: 218 ms, MXFP8 392.)
__device__ __forceinline__ bool huge_score(float s) {
  return fabsf(s) >= 0x1p24f && fabsf(s) < INFINITY;
}
// Keys key0 .. key1-1 of the row with query q and view `anc`: its maximum and sum, and its sums of V's columns
// d0 .. d1-1 in acc[d0 ..].  Score products and maxima are both rounded.  The others' waits go by `steps`.
template <int D, bool MX>
__device__ __noinline__ float2 huge_row(const AttendParams& P, int seq, int ctx, int h, const uint32_t* anc,
                                        int key0, int key1, const uint16_t* q, float* acc, int d0, int d1,
                                        int* steps) {
  const uint8_t* kb = P.c.k + h * P.s.stride_head * (MX ? 1 : 2);
  const uint8_t* sb = MX ? P.c.ks + (h * P.s.stride_head >> 5) : nullptr;
  const float scale = P.scale_log2;
  float m = -INFINITY, l = 0.f, base = 0.f;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t off = paged_off8(P.s, page_of(P.s, seq, key0), key0, key1);
#pragma unroll 1
    for (int p = key0; p < key1; ++p) {
      const uint32_t here = off;
      if ((p & 255) == 0) atomicAdd(steps, 1);
      const int page = page_of(P.s, seq, min(p + 1, key1 - 1));  // the next row's
      if (p < ctx || ((anc[(p - ctx) >> 5] >> ((p - ctx) & 31)) & 1u)) {
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 2
        for (int d = 0; d < D; d += 16) {
          uint4 k[2];
          if constexpr (MX) {
            const uint4 w = *reinterpret_cast<const uint4*>(kb + static_cast<uint64_t>(here) * 8 + d);
            const uint32_t sc = e8m0_bf16x2(sb[(here >> 2) + (d >> 5)]);
            e4m3x4_bf16(w.x, sc, k[0].x, k[0].y);
            e4m3x4_bf16(w.y, sc, k[0].z, k[0].w);
            e4m3x4_bf16(w.z, sc, k[1].x, k[1].y);
            e4m3x4_bf16(w.w, sc, k[1].z, k[1].w);
          } else {
            const uint4* from = reinterpret_cast<const uint4*>(kb + static_cast<uint64_t>(here) * 16 + d * 2);
            k[0] = from[0];
            k[1] = from[1];
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float2 a[4], b[4];
            unpack8(k[u], a);
            unpack8(ld_ro(q + d + u * 8), b);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[u] = ffma2(a[e], b[e], sum[u]);
          }
        }
        const float s = __fmul_rn((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y), scale);
        if (pass == 0) {
          m = fmaxf(m, s);
        } else {
          const float w = ex2(__fsub_rn(s, base));
          l += w;
          const int64_t v = static_cast<int64_t>(here) * 8 + h * P.s.stride_head;
          if (w != 0.f)  // seldom
            for (int d = d0; d < d1; ++d) acc[d] = fmaf(w, cache_value<MX>(P.c.v, P.c.vs, v + d), acc[d]);
        }
      }
      off = row_off8(P.s, page, min(p + 1, key1 - 1));
    }
    if (pass == 0) {
      base = m == -INFINITY ? 0.f : m;
      for (int d = d0; d < d1; ++d) acc[d] = 0.f;
    }
  }
  return make_float2(m, l);
}

template <int D, bool MX>
__global__ void __launch_bounds__(tc_threads<D, MX>(), 1)
    attend_tc_kernel(const AttendParams P, int rows_unit, int ring_units) {
  using T = TcShape<D>;
  using F = FeedShape<D, T::kKeys, MX>;
  constexpr int TN = T::kKeys, NS = T::kStreams, THREADS = tc_threads<D, MX>();
  constexpr int kSoft = 32 * T::kSoftWarps;
  constexpr uint32_t kQTile = 128 * D * 2, kQBlock = 128 * 128;
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_anc[kMaxDraft][kMaskWords];
  __shared__ int s_ptr[kMaxDraft];
  __shared__ float2 s_ml[2][128];
  __shared__ int64_t s_scan[2 * (THREADS / 32)], s_found[2];
  __shared__ uint64_t s_full[8], s_empty[8], s_score[2], s_prob[2], s_out[2], s_query, s_drain;
  __shared__ uint64_t s_raw_full[F::kRaw], s_raw_empty[F::kRaw];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort[3];  // a wait ran out; a V row was cleaned; steps of huge_row()
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
  int seq, extra = kUnitExtra;
  find_range<THREADS>(P.s, P.g, P.H, rows_unit, TN, P.prefix, blockIdx.x, gridDim.x, s_scan,
                      s_found, cur, end, seq, seq_first, extra);  // barriers inside
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // Every role walks the same segments.
  SeqView sv;
  SeqTiles st;
  int h = 0, row0 = 0, rows = 0, t0 = 0, tiles = 0, total = 0;
  bool pair = false;
  auto enter = [&] {
    sv = seq_view(P.s, seq, false);
    st = seq_tiles(sv, P.g, P.H, rows_unit, TN, extra);
  };
  auto locate = [&]() -> bool {  // false behind the last one
    do {
      if (cur >= end) return false;
      while (cur >= seq_first + st.all) {  // the next sequence with tiles
        seq_first += st.all;
        ++seq;
        enter();
      }
      const int64_t rel = cur - seq_first;
      const int steps = st.kt + extra;
      const int unit = static_cast<int>(rel / steps);
      const int s0 = static_cast<int>(rel - static_cast<int64_t>(unit) * steps);
      const int s1 = static_cast<int>(min(static_cast<int64_t>(steps), s0 + (end - cur)));
      t0 = max(0, s0 - extra);
      tiles = max(0, s1 - extra) - t0;
      h = unit / st.mt;
      row0 = (unit - h * st.mt) * rows_unit;
      cur += s1 - s0;
    } while (tiles == 0);
    rows = min(rows_unit, sv.n * P.g - row0);
    total = sv.ctx + sv.n;
    pair = NS == 2 && rows > 128;
    return true;
  };
  if (cur < end) enter();

  if (warp < T::kSoftWarps) {
    // ------------------------------------------------------------- softmax
    if constexpr (NS == 2) more_registers<MX ? 136 : 184>();
    const int stream = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's lanes
    const int r = (warp & 3) * 32 + lane;                          // row of the stream's tile
    // (0 would make NaN of a masked -inf; 2^-100 of any sane score is 0 as well)
    const float scale = fmaxf(fabsf(P.scale_log2), 0x1p-100f);
    const uint32_t flip = P.scale_log2 < 0.f ? 0x80008000u : 0u;  // the sign goes to Q
    uint32_t seen_scores[2] = {0, 0}, seen_outs[2] = {0, 0};
    int segment = 0, masked_seq = -1;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t count) {  // until its phase `count` is complete
      if (ok) ok = tc_wait(bar, count & 1u, s_abort);
      ok = __all_sync(kFullMask, ok);
    };
    auto meet = [&] { asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory"); };
    while (locate()) {
      // ---- Q, rows of both streams
      // (a thread keeps its 8 columns; the loads of eight rows are in flight at once)
      {
        constexpr int kStep = kSoft / (D / 8);  // rows apart
        const int c = tid % (D / 8);
        const uint16_t* qp = P.q + sv.a * P.q_tok + static_cast<int64_t>(h) * P.g * P.q_head + c * 8;
        // rows of zeros up to a whole tile: what lay there would cost power, and so clocks
        // (32 rows over 1M tokens at the power limit, on one box: 820 us with it, 747 without)
        const int fill = pair ? 256 : 128;
        for (int r0 = tid / (D / 8); r0 < fill; r0 += 8 * kStep) {
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = r0 + i * kStep;
            v[i] = make_uint4(0, 0, 0, 0);
            if (rr < rows) {
              const int tk = (row0 + rr) / P.g;
              v[i] = ld_ro(qp + tk * P.q_tok + (row0 + rr - tk * P.g) * P.q_head);
              v[i].x ^= flip;
              v[i].y ^= flip;
              v[i].z ^= flip;
              v[i].w ^= flip;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = r0 + i * kStep;
            if (rr < fill)
              sts16(smem + (rr >> 7) * kQTile + (c >> 3) * kQBlock + (rr & 127) * 128 +
                        (((c & 7) ^ (rr & 7)) << 4),
                    tc_order<MX>(v[i]));
          }
        }
      }
      async_proxy_fence();
      mbar_arrive(&s_query);
      // the masks meanwhile: the first product does not need them
      if (masked_seq != seq) {
        ancestor_masks(P.s, sv, s_anc, s_ptr, t0 == 0 && h == 0 && row0 == 0, meet);
        masked_seq = seq;
      }

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
          if (tail) {  // masked scores become -inf where they lie
            float x[32];
#pragma unroll 1
            for (int c = 0; c < TN; c += 32) {
              if (a0 + c + 32 <= 0) continue;
              const uint32_t vis = seen32(s_anc[tok], a0 + c, used);
              tmem_ld32(x, at + c);
              tmem_landed(x);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = (vis >> e) & 1u ? x[e] : -INFINITY;
              tmem_st32(at + c, x);
            }
            tmem_wait_st();
          }
          // One pass with the maximum so far.  A tile whose own maximum is
          // more than 2^8 above it (a row's first tile among them) is done again with that:
          // the probabilities are stored behind the pass, so S is still there.
          uint32_t p[TN / 32][16];
          float2 acc;
#pragma unroll 1
          for (int pass = 0; pass < 3; ++pass) {
            const float base = mx == -INFINITY ? 0.f : mx;
            const float2 sc = make_float2(scale, scale), nb = make_float2(-base, -base);
            acc = make_float2(0.f, 0.f);
            float m0 = -INFINITY, m1 = -INFINITY;
            float x[2][32];
            tmem_ld32(x[0], at);
#pragma unroll
            for (int c = 0; c < TN / 32; ++c) {
              tmem_landed(x[c & 1]);
              if (c + 1 < TN / 32) tmem_ld32(x[(c + 1) & 1], at + (c + 1) * 32);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                float2 y = ffma2(make_float2(x[c & 1][e], x[c & 1][e + 1]), sc, nb);
                float2 z = ffma2(make_float2(x[c & 1][e + 2], x[c & 1][e + 3]), sc, nb);
                m0 = fmaxf(m0, fmaxf(y.x, y.y));
                m1 = fmaxf(m1, fmaxf(z.x, z.y));
                y.x = ex2(y.x);
                y.y = ex2(y.y);
                z.x = ex2(z.x);
                z.y = ex2(z.y);
                acc = __fadd2_rn(acc, __fadd2_rn(y, z));
                p[c][e / 2] = pack_bf16x2(y);
                p[c][e / 2 + 1] = pack_bf16x2(z);
                // (done here and now: postponed, twice the numbers would be live)
                asm volatile(""
                             : "+r"(p[c][e / 2]), "+r"(p[c][e / 2 + 1]), "+f"(acc.x), "+f"(acc.y),
                               "+f"(m0), "+f"(m1));
              }
            }
            const float top = fmaxf(m0, m1);
            const bool grow = top > (mx == -INFINITY ? -INFINITY : 8.f);
            if (!__any_sync(kFullMask, grow)) break;
            const float to = grow ? base + top : mx;
            const float w = merge_weight(mx, to);
            mx = to;
            sum *= w;
            if (t >= (NS == 1 ? 1 : t_first + t_step)) {
              // O holds the tiles before: complete with this S, or (one stream)
              // with the last product
              if (NS == 1) wait(&s_out[(t - 1) & 1], seen_outs[(t - 1) & 1] + ((t - 1) >> 1));
              tc_fence_after();
              const uint32_t o = tmem + lanes + T::kOut + (NS == 1 ? 0 : stream) * D;
              if (!ok) break;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                tmem_ld32(x[0], o + c);
                tmem_landed(x[0]);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[0][e] *= w;
                tmem_st32(o + c, x[0]);
              }
            }
          }
#pragma unroll
          for (int c = 0; c < TN / 32; ++c)
            tmem_st16(at + c * 16, p[c]);
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
          if constexpr (MX) {  // back from the units' order of columns
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float y = x[e + 1];
              x[e + 1] = x[e + 2];
              x[e + 2] = y;
            }
          }
          if (mine < rows) {
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
        if (*reinterpret_cast<volatile int*>(&s_abort[1]) && used)  // rare
          for (int d = d0; d < d1; ++d) {
            const float v = restore_nonfinite<MX>(P, seq, sv.ctx, sv.n, h, s_anc[tok], t0 * TN,
                                                  min(total, (t0 + tiles) * TN), d, 0.f);
            if (fabsf(v) < INFINITY) continue;
            if (whole) {
              uint16_t* to = P.out + (sv.a + tok) * P.o_tok + hq * P.o_head + d;
              const float o = __uint_as_float(static_cast<uint32_t>(*to) << 16);
              *to = static_cast<uint16_t>(pack_bf16x2(make_float2(o + v, 0.f)));
            } else {
              P.part_o[(slot * rows_unit + mine) * D + d] += v;
            }
          }
        if (huge_score(mx) && used) {
          float* acc = P.part_o + (slot * rows_unit + mine) * D;  // (its place, or free while the unit is whole)
          const float2 r = huge_row<D, MX>(P, seq, sv.ctx, h, s_anc[tok], t0 * TN, min(total, (t0 + tiles) * TN),
                                           P.q + (sv.a + tok) * P.q_tok + hq * P.q_head, acc, d0, d1, &s_abort[2]);
          mx = r.x;
          sum = r.y;
          if (whole)
            for (int d = d0; d < d1; ++d)
              P.out[(sv.a + tok) * P.o_tok + hq * P.o_head + d] = static_cast<uint16_t>(
                  pack_bf16x2(make_float2(sum == 0.f ? 0.f : acc[d] / sum, 0.f)));
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
      ++segment;
    }
    if (!ok && lane == 0) raise_flag(P.s.err, kFlagTimeout);
  } else if (warp < T::kSoftWarps + F::kWarps) {
    // ------------------------------------------------------------ producers
    if constexpr (NS == 2) fewer_registers<MX ? 64 : 72>();
    const int w = warp - T::kSoftWarps;
    FeedRing R{units, s_full, s_empty, s_abort, ring_units};
    if constexpr (MX) {
      FeedRing Raw{raw, s_raw_full, s_raw_empty, s_abort, F::kRaw};
      while (locate()) {
        const int64_t head = h * P.s.stride_head >> 5;
        const int k_low = P.c.words ? reinterpret_cast<uintptr_t>(P.c.ks + head) & 3 : 0;
        const int v_low = P.c.words ? reinterpret_cast<uintptr_t>(P.c.vs + head) & 3 : 0;
#pragma unroll 1
        for (int u = 0; u < 2 * tiles; ++u) {
          bool is_v;
          int t;
          unit_of(u, tiles, pair, is_v, t);
          const int clean = is_v ? max(0, min(TN, sv.ctx - (t0 + t) * TN)) : TN;
          FeedMx<D, TN>::decode(R, Raw, w, lane, is_v ? v_low : k_low, clean);
        }
      }
    } else {
      while (locate()) {
        const int64_t head = h * P.s.stride_head;
        const uint8_t *kb = P.c.k + head * 2, *vb = P.c.v + head * 2;
        const int32_t* table = P.s.table + seq * P.s.table_stride;
        const int key0 = t0 * TN + w * F::kKeysWarp + lane % F::kKeysWarp;
        int page = __ldg(table + page_index(P.s, min(key0, total - 1)));
        uint32_t off0 = ~0u, off1 = ~0u;  // of the tiles of either parity
#pragma unroll 1
        for (int u = 0; u < 2 * tiles; ++u) {
          bool is_v;
          int t, clean = TN;
          unit_of(u, tiles, pair, is_v, t);
          if (is_v) {
            clean = max(0, min(TN, sv.ctx - (t0 + t) * TN));
          } else {
            const int p = key0 + t * TN;
            const uint32_t o = paged_off8(P.s, page, p, total);
            if (t & 1) off1 = o;
            else off0 = o;
            page = __ldg(table + page_index(P.s, min(p + TN, total - 1)));  // of the next tile
          }
          FeedBf16<D, TN>::bring(R, w, lane, is_v ? vb : kb, t & 1 ? off1 : off0, clean);
        }
      }
      cp_commit();
      cp_wait<0>();
    }
  } else {
    // ------------------------------------------------------------- products
    if constexpr (NS == 2) fewer_registers<MX ? 80 : 72>();
    // (the whole warp goes along, so that addresses stay in uniform registers; one
    // lane issues)
    if (warp == T::kSoftWarps + F::kWarps) {
    constexpr uint32_t kIdS = tc_idesc(128, TN, false), kIdO = tc_idesc(128, D, true);
    constexpr uint32_t kBlock = TN * 128;  // 64 columns of a unit
    uint32_t probs[2] = {0, 0}, queries = 0;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t count) {
      if (ok) ok = tc_wait(bar, count & 1u, s_abort);
      ok = __all_sync(kFullMask, ok);
    };
    auto unit = [&](int at, uint32_t par) {  // until the unit is there
      wait(&s_full[at], par);
      async_proxy_fence();
      tc_fence_after();
    };
    auto next = [&] {
      if (++slot == ring_units) {
        slot = 0;
        phase ^= 1;
      }
    };
    const uint32_t query = tc_desc(smem, 16), keys = tc_desc(units, 16);
    const uint32_t values = tc_desc(units, kBlock);
    auto commit = [&](uint64_t* bar) {
      if (ok && elect_one()) tc_commit(bar);
      __syncwarp();
    };
    auto score = [&](int b, int stream) {  // S[b] = Q K^T with the unit in `slot`
      const uint32_t q = query + stream * (kQTile >> 4), k = keys + slot * (F::kUnit >> 4);
      const uint32_t to = tmem + b * TN;
      if (ok && elect_one()) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          tc_mma(to, q + (((j >> 2) * kQBlock + (j & 3) * 32) >> 4),
                 k + (((j >> 2) * kBlock + (j & 3) * 32) >> 4), kIdS, j > 0);
        tc_commit(&s_score[b]);
      }
      __syncwarp();
    };
    auto output = [&](int b, int stream, bool first) {  // O += P V
      const uint32_t v = values + slot * (F::kUnit >> 4);
      const uint32_t to = tmem + T::kOut + stream * D, p = tmem + b * TN;
      if (ok && elect_one()) {
        tc_mma_tmem(to, p, v, kIdO, !first);
#pragma unroll
        for (int j = 1; j < TN / 16; ++j) tc_mma_tmem(to, p + j * 8, v + j * 128, kIdO, 1);
        tc_commit(&s_out[b]);
      }
      __syncwarp();
    };
    auto free_unit = [&] {
      commit(&s_empty[slot]);
      next();
    };
    while (ok && locate()) {
      wait(&s_query, queries++);
      if (pair) {
        unit(slot, phase);
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
            if (s == 0) unit(v_slot, v_phase);
            tc_fence_after();
            output(s, s, t == 0);
            if (s == 1) commit(&s_empty[v_slot]);
            if (more) {
              slot = k_slot;
              if (s == 0) unit(k_slot, k_phase);
              tc_fence_after();
              score(s, s);
              if (s == 1) commit(&s_empty[k_slot]);
            }
          }
          slot = v_slot;
          phase = v_phase;
          next();
          if (more) next();
        }
      } else {
        for (int t = 0; t < 2 && t < tiles; ++t) {
          unit(slot, phase);
          score(t, 0);
          free_unit();
        }
        for (int t = 0; t < tiles && ok; ++t) {
          const int b = t & 1;
          wait(&s_prob[b], probs[b]++);
          unit(slot, phase);
          output(b, NS == 2 ? b : 0, t < NS);
          free_unit();
          if (t + 2 < tiles) {
            unit(slot, phase);
            score(b, 0);
            free_unit();
          }
        }
      }
    }
    // products still under way would write to freed tensor memory
    if (elect_one()) tc_commit(&s_drain);
    __syncwarp();
    int dummy[1] = {0};
    if (!mbar_wait(&s_drain, 0, dummy, kDrainTimeoutNs)) ok = false;
    if (!ok && lane == 0) raise_flag(P.s.err, kFlagTimeout);
    } else if constexpr (MX) {
      // ---- raw units
      using M = FeedMx<D, TN>;
      const int w = warp - (T::kSoftWarps + F::kWarps + 1);
      FeedRing Raw{raw, s_raw_full, s_raw_empty, s_abort, F::kRaw};
      while (locate()) {
        const int64_t head = h * P.s.stride_head;
        const int32_t* table = P.s.table + seq * P.s.table_stride;
        const int key0 = t0 * TN + w * 8 + (lane >> 2);
        int page[M::kMine];  // of the next tile
        uint32_t off0[M::kMine], off1[M::kMine];  // of the tiles of either parity
        auto pages = [&](int t) {
#pragma unroll
          for (int i = 0; i < M::kMine; ++i)
            page[i] = __ldg(table + page_index(P.s, min(key0 + t * TN + i * M::kStep, total - 1)));
        };
        auto offsets = [&](uint32_t(&off)[M::kMine], int t) {
#pragma unroll
          for (int i = 0; i < M::kMine; ++i) {
            const uint32_t o = paged_off8(P.s, page[i], key0 + t * TN + i * M::kStep, total);
            off[i] = o == ~0u ? 0 : o;
          }
        };
        pages(0);
#pragma unroll 1
        for (int u = 0; u < 2 * tiles; ++u) {
          bool v;
          int t;
          unit_of(u, tiles, pair, v, t);
          if (!v) {
            if (t & 1) offsets(off1, t);
            else offsets(off0, t);
            pages(t + 1);
          }
          uint32_t off[M::kMine];
#pragma unroll
          for (int i = 0; i < M::kMine; ++i) off[i] = t & 1 ? off1[i] : off0[i];
          M::fetch(Raw, w, lane, (v ? P.c.v : P.c.k) + head, (v ? P.c.vs : P.c.ks) + (head >> 5),
                   P.c.words, off, total - (t0 + t) * TN);
        }
      }
      cp_commit();
      cp_wait<0>();
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, 512);
}

}  // namespace sconv
