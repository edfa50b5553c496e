// Attention of drafted-tree queries over the paged K/V cache (sm_100a): what
// its kernels share, the kernel for few query rows, and the join of the
// splits.
//
// Per drafted token j of sequence i and query head hq (K/V head h = hq / g,
// g = query heads a K/V head):
//     s_p = scale * q . k_p      over p < ctx, and p = ctx + a for a in
//                                {j, j's ancestors}
//     out = sum_p softmax(s)_p v_p,   lse = ln sum_p exp s_p
// with out = 0, lse = -inf for an unused token, which sees nothing.
//
// Rows: the n * g (token, query head) pairs of a K/V head, row r = j*g + hq%g,
// in M-tiles of R rows.  A unit is one (sequence, K/V head, M-tile); its keys
// come in tiles of kTile.  All units' tiles in one line are cut into
// equal ranges, one a CTA, whatever the lengths: a batch of short sequences
// and a single long one both fill the SMs.  A unit that lies in one CTA is
// finished there; a cut one leaves partial (o, m, l) per CTA in the
// workspace, and the join kernel merges them in range order (no atomics: the
// same call gives the same bits).
//
// Softmax statistics, scores and sums are fp32; the only rounding to fewer bits
// are the probabilities, to bf16 for the second product (which is what the matrix
// instruction takes next to bf16 values; 2^-8 relative each at most, independent of one
// another), and the output.  Measured against 64 bits: 0.0023 relative, where the output's
// own rounding alone is 0.0017.
//
// Masked keys: their score is replaced by -inf before the maximum, and a drafted V row
// (that nobody or not everybody may see) is cleaned of NaN and infinities before the
// product (0 * inf would reach rows that do not see it); rows that do see
// such a value get it back afterwards (restore_nonfinite).  The context's rows,
// which every used token sees, stay as they are.
#pragma once
#include "paged.cuh"

namespace sconv {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(m - base) for running maxima, 0 for an empty side.
__device__ __forceinline__ float merge_weight(float m, float base) {
  return m == -INFINITY ? 0.f : ex2(m - base);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E4M3 codes in the low bytes of each half of x (as 00bb00bb) ... the four
// codes of a word as bf16 pairs lo (codes 0, 1) and hi (2, 3), times 2^s.
// A code's bits, sign at 15 and the rest shifted to 4..10, read as bf16 are the
// value * 2^-120 (exponent bias 7 against 127, subnormals included), so one
// exact multiplication by 2^120 and one by the scale give the value; both
// are powers of two.  Codes 0x7f and 0xff are NaN.
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t e8m0_bf16x2(uint32_t byte) {
  // 2^(byte - 127) as bf16: the byte is the exponent field (0: 2^-127, subnormal;
  // 255: NaN, as E8M0 has it)
  const uint32_t h = byte == 0 ? 0x0040u : byte == 255 ? 0x7fc0u : byte << 7;
  return h * 0x10001u;
}
__device__ __forceinline__ void e4m3x4_bf16(uint32_t w, uint32_t scale2, uint32_t& lo,
                                            uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0, 0x1404);  // bytes 0, 1 to bits 8..15 of each half
  const uint32_t b = __byte_perm(w, 0, 0x3424);
  lo = (a & 0x80008000u) | ((a >> 4) & 0x07f007f0u);
  hi = (b & 0x80008000u) | ((b >> 4) & 0x07f007f0u);
  const uint32_t two120 = 0x7b807b80u;
  lo = bf16x2_mul(bf16x2_mul(lo, two120), scale2);
  hi = bf16x2_mul(bf16x2_mul(hi, two120), scale2);
  // NaN codes: 0x7f + 1 carries into bit 7
  if (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) {
    if ((w & 0x7fu) == 0x7fu) lo |= 0x00007fc0u;
    if ((w & 0x7f00u) == 0x7f00u) lo |= 0x7fc00000u;
    if ((w & 0x7f0000u) == 0x7f0000u) hi |= 0x00007fc0u;
    if ((w & 0x7f000000u) == 0x7f000000u) hi |= 0x7fc00000u;
  }
}

// One cached value (rare paths).
template <bool MX>
__device__ __forceinline__ float cache_value(const uint8_t* base, const uint8_t* scales,
                                             int64_t elem) {
  if constexpr (MX) {
    uint32_t lo, hi;
    e4m3x4_bf16(base[elem], e8m0_bf16x2(scales[elem >> 5]), lo, hi);
    return __uint_as_float(lo << 16);
  } else {
    return __uint_as_float(
        static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(base)[elem]) << 16);
  }
}

// Tiles of one sequence: M-tiles, key tiles of one unit, and what all its units take of the
// line over the K/V heads, where `extra` steps stand for a unit's beginning and end.
struct SeqTiles {
  int mt;
  int kt;
  int64_t all;
};
__device__ __forceinline__ SeqTiles seq_tiles(const SeqView& s, int g, int H, int rows, int tile,
                                              int extra = 0) {
  SeqTiles t;
  t.mt = (s.n * g + rows - 1) / rows;
  t.kt = s.n ? static_cast<int>((static_cast<int64_t>(s.ctx) + s.n + tile - 1) / tile) : 0;
  t.all = t.kt ? static_cast<int64_t>(t.mt) * H * (t.kt + extra) : 0;
  return t;
}

// Where in the line of all tiles this CTA's range begins: the
// sequence that holds step `first`, and the steps before that sequence.  The first
// CTA writes the prefix that the join reads (if there is one; `extra` behind it), and raises
// the flags.  `extra` comes in as what a unit's beginning and end cost, in tiles, and goes out
// as 0 where a range is too short for it to matter: a range of more than `extra` steps
// has a tile, which the join counts on.  Every thread of the block takes part (THREADS
// of them); s_scan has 2 * THREADS/32 entries.
template <int THREADS>
__device__ __forceinline__ void find_range(const PagedSeqs& Q, int g, int H, int rows, int tile,
                                           int64_t* prefix, int part, int parts, int64_t* s_scan,
                                           int64_t* s_found, int64_t& first, int64_t& last,
                                           int& seq, int64_t& seq_first, int& extra) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = THREADS / 32;
  const int S = Q.num_seqs;
  const int per = (S + THREADS - 1) / THREADS;
  const int i0 = min(S, tid * per), i1 = min(S, i0 + per);
  const bool lead = part == 0;
  int64_t sum = 0, units = 0;
  for (int i = i0; i < i1; ++i) {
    const SeqTiles t = seq_tiles(seq_view(Q, i, lead), g, H, rows, tile);
    sum += t.all;
    units += t.kt ? static_cast<int64_t>(t.mt) * H : 0;
  }
  int64_t inc = sum, inu = units;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t up = __shfl_up_sync(kFullMask, inc, d), uu = __shfl_up_sync(kFullMask, inu, d);
    if (lane >= d) {
      inc += up;
      inu += uu;
    }
  }
  if (lane == 31) {
    s_scan[warp] = inc;
    s_scan[kWarps + warp] = inu;
  }
  if (tid == 0) {
    s_found[0] = -1;
    s_found[1] = 0;
  }
  __syncthreads();
  int64_t before = inc - sum, total = 0, units_before = inu - units, units_all = 0;
  for (int k = 0; k < kWarps; ++k) {
    if (k < warp) {
      before += s_scan[k];
      units_before += s_scan[kWarps + k];
    }
    total += s_scan[k];
    units_all += s_scan[kWarps + k];
  }
  if (total < 2ll * (extra + 1) * parts) extra = 0;
  before += extra * units_before;
  total += extra * units_all;
  sum += extra * units;
  // no empty range between two others: the join counts on it
  const int64_t used = min(static_cast<int64_t>(parts), max(total, static_cast<int64_t>(1)));
  first = min(part, static_cast<int>(used)) * total / used;
  last = min(part + 1, static_cast<int>(used)) * total / used;
  if (lead || (before <= first && first < before + sum)) {
    int64_t at = before;
    for (int i = i0; i < i1; ++i) {
      const int64_t all = seq_tiles(seq_view(Q, i, false), g, H, rows, tile, extra).all;
      if (lead && prefix) prefix[i] = at;
      if (at <= first && first < at + all) {
        s_found[0] = i;
        s_found[1] = at;
      }
      at += all;
    }
    if (lead && prefix && tid == THREADS - 1) {
      prefix[S] = total;
      prefix[S + 1] = extra;
    }
  }
  __syncthreads();
  seq = static_cast<int>(s_found[0]);
  seq_first = s_found[1];
}

// First tile of a range, and the range that holds a tile.
__device__ __forceinline__ int64_t range_start(int64_t part, int64_t total, int parts) {
  return part * total / parts;
}
__device__ __forceinline__ int range_of(int64_t tile, int64_t total, int parts) {
  return static_cast<int>(((tile + 1) * parts - 1) / total);
}

// Give the non-finite V values of drafted tokens that row `anc` sees back to
// its output element d (their probabilities are positive, so the sum takes the
// value itself).
template <bool MX>
__device__ __noinline__ float restore_nonfinite(const AttendParams& P, int seq, int ctx, int n,
                                                int h, const uint32_t* anc, int key0, int key1,
                                                int d, float o) {
  for (int j = max(0, key0 - ctx); j < n && ctx + j < key1; ++j)
    if ((anc[j >> 5] >> (j & 31)) & 1u) {
      const int64_t off =
          row_offset(P.s, page_of(P.s, seq, ctx + j), ctx + j) + h * P.s.stride_head + d;
      const float v = cache_value<MX>(P.c.v, P.c.vs, off);
      if (!(fabsf(v) < INFINITY)) o += v;
    }
  return o;
}

// ------------------------------------------------------------ few query rows
//
// R = 8 or 16 rows, 4 warps a CTA, 16 keys a warp and step, nothing staged in
// shared memory but Q: the operands of both products go from global memory
// straight into the registers in which the matrix instruction wants them.
//   S[row, key] = Q K^T   (m16 rows x n8 keys): a lane needs, of key row
//     lane/4, element pairs; which dims a k-step takes is free as long as Q
//     takes the same, so a lane loads 16 bytes (8 dims; 16 codes) a row and
//     four lanes cover 64 contiguous bytes of it.
//   O^T[d, row] = V^T P^T (m16 dims x n8 rows x k16 keys): P^T is S's own
//     register layout, and V's pairs of neighbouring keys are made from two
//     16-byte row pieces with one byte permutation each.
// The K/V bytes bound it: R rows cost 16 of the 512 issue slots that 16 keys'
// 8 KB take to arrive; what counts is bytes in flight, so the loads of the
// next step are issued as soon as the registers are free.  Measured: 64 heads' one row over 8192
// tokens 24 us with the join (latency: range, table, K/V, parts; the bytes take 5).

template <int D, bool MX>
struct RowsLayout {
  static constexpr int kKVec = MX ? D / 64 : D / 32;          // 16-byte K loads a key and lane
  static constexpr int kVBytes = MX && D == 64 ? 8 : 16;      // bytes of a V load
  static constexpr int kVDims = MX ? kVBytes : 8;             // dims of a V load
  static constexpr int kVVec = D / (8 * kVDims);              // V loads a key and lane
  static constexpr int kQPitch = 2 * D + 64;                  // bytes; rows land on other banks
};

// First dim of the 8 that Q's t-th 16-byte piece holds for lane column c.
template <bool MX>
__device__ __forceinline__ int q_dim(int t, int c) {
  return MX ? (t >> 1) * 64 + c * 16 + (t & 1) * 8 : t * 32 + c * 8;
}

// Eight bf16 values, NaN and infinities as 0.
__device__ __forceinline__ uint4 clean16(uint4 x, bool& found) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((w[e] & 0x7f80u) == 0x7f80u) {
      w[e] &= 0xffff0000u;
      found = true;
    }
    if ((w[e] & 0x7f800000u) == 0x7f800000u) {
      w[e] &= 0x0000ffffu;
      found = true;
    }
  }
  return x;
}

// Sixteen E4M3 codes of scale byte `s`, as 0 where they decode to NaN or an infinity.  A code with
// exponent field E stands for a value of at least 2^(E - 7) (E > 0), times 2^(s - 127): from
// E + s = 262 on that is 2^128, which no float holds; code 0x7f and scale 255 are NaN.
__device__ __forceinline__ uint4 clean_codes(uint4 x, uint32_t s, bool& found) {
  const uint32_t limit = s == 255u ? 0u : min(127u, (262u - s) * 8u);  // the first such code
  uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int b = 0; b < 32; b += 8)
      if (((w[e] >> b) & 0x7fu) >= limit) {
        w[e] &= ~(0xffu << b);
        found = true;
      }
  }
  return x;
}

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_stream8(const uint8_t* p) {
  uint4 v = make_uint4(0, 0, 0, 0);
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}
// The D/32 scale bytes of a row, the first in the low byte.
template <int D>
__device__ __forceinline__ uint64_t ld_scales(const uint8_t* p, int packed) {
  if (!packed) {
    uint64_t v = 0;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) v |= static_cast<uint64_t>(__ldg(p + b)) << (8 * b);
    return v;
  }
  if constexpr (D == 64) return __ldg(reinterpret_cast<const uint16_t*>(p));
  if constexpr (D == 128) return __ldg(reinterpret_cast<const uint32_t*>(p));
  return __ldg(reinterpret_cast<const unsigned long long*>(p));
}

template <int D, int NT, bool MX>
__global__ void __launch_bounds__(32 * kRowsWarps, D == 256 ? 2 : NT == 1 ? 4 : 3)
    attend_rows_kernel(const AttendParams P) {
  using L = RowsLayout<D, MX>;
  constexpr int R = 8 * NT, THREADS = 32 * kRowsWarps;
  constexpr int KV = L::kKVec, VV = L::kVVec, MTILES = D / 16;
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ __align__(16) uint8_t smem[];
  // Q (R rows), then at a segment's end the warps' results (fp32 [4][R][D + 4])
  float* s_o = reinterpret_cast<float*>(smem);
  __shared__ uint32_t s_anc[kMaxDraft][kMaskWords];
  __shared__ int s_ptr[kMaxDraft];
  __shared__ float2 s_ml[kRowsWarps][R];
  __shared__ int64_t s_scan[2 * (THREADS / 32)], s_found[2];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lr = lane >> 2, lc = lane & 3;  // row (or key) and column of a fragment

  int64_t cur, end, seq_first;
  int seq, extra = 0;
  find_range<THREADS>(P.s, P.g, P.H, R, kRowsTile, P.prefix, blockIdx.x, gridDim.x, s_scan,
                      s_found, cur, end, seq, seq_first, extra);
  if (tid == 0) s_bad = 0;
  if (cur >= end) return;
  int segment = 0, masked_seq = -1;
  SeqView sv = seq_view(P.s, seq, false);
  SeqTiles st = seq_tiles(sv, P.g, P.H, R, kRowsTile);
  while (cur < end) {
    while (cur >= seq_first + st.all) {  // the next sequence with tiles
      seq_first += st.all;
      ++seq;
      sv = seq_view(P.s, seq, false);
      st = seq_tiles(sv, P.g, P.H, R, kRowsTile);
    }
    const int64_t rel = cur - seq_first;
    const int unit = static_cast<int>(rel / st.kt);
    const int t0 = static_cast<int>(rel - static_cast<int64_t>(unit) * st.kt);
    const int t1 = static_cast<int>(min(static_cast<int64_t>(st.kt), t0 + (end - cur)));
    const int h = unit / st.mt, row0 = (unit - h * st.mt) * R;
    const int rows = min(R, sv.n * P.g - row0);
    const int total = sv.ctx + sv.n;
    const int key1 = min(total, t1 * kRowsTile);

    const uint8_t* kb = P.c.k + h * P.s.stride_head * (MX ? 1 : 2);
    const uint8_t* vb = P.c.v + h * P.s.stride_head * (MX ? 1 : 2);
    const uint8_t* ksb = MX ? P.c.ks + (h * P.s.stride_head >> 5) : nullptr;
    const uint8_t* vsb = MX ? P.c.vs + (h * P.s.stride_head >> 5) : nullptr;
    const int32_t* table = P.s.table + seq * P.s.table_stride;

    float o[MTILES][NT][4];
#pragma unroll
    for (int m = 0; m < MTILES; ++m)
#pragma unroll
      for (int r = 0; r < NT; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][r][e] = 0.f;
    float mx[NT], sum[NT];
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      mx[r] = -INFINITY;
      sum[r] = 0.f;
    }
    bool found = false;

    uint4 kreg[2][KV], vreg[4][VV];
    uint64_t ksc[2] = {0, 0};
    uint32_t vsc[4][VV];
    const int step = 16 * kRowsWarps;
    int base = t0 * kRowsTile + warp * 16;
    // row offset, in units of 8 elements, of key base + lane % 16
    auto page_at = [&](int b) {
      const int p = min(b + (lane & 15), total - 1);
      return __ldg(table + page_index(P.s, p));
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
    // keys of this lane in the second product: 2c, 2c+1, 2c+8, 2c+9
    auto load_v = [&](uint32_t off8) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint64_t o8 = __shfl_sync(kFullMask, off8, 2 * lc + (t & 1) + (t >> 1) * 8);
        const uint8_t* p = vb + o8 * (MX ? 8 : 16) + lr * L::kVBytes;
#pragma unroll
        for (int k = 0; k < VV; ++k) {
          vreg[t][k] = L::kVBytes == 8 ? ld_stream8(p) : ld_stream(p + k * 128);
          if constexpr (MX)
            vsc[t][k] = __ldg(vsb + (o8 >> 2) + ((k * 8 * L::kVDims + lr * L::kVDims) >> 5));
        }
      }
    };
    uint32_t off = 0, off_next = 0;
    int page_next = 0;
    if (base < key1) {
      off = off_at(base, page_at(base));
      page_next = page_at(base + step);
      load_k(off);
      load_v(off);
      off_next = off_at(base + step, page_next);
    }
    // ---- Q rows and ancestor masks
    if (masked_seq != seq) {
      ancestor_masks(P.s, sv, s_anc, s_ptr, t0 == 0 && unit == 0);
      masked_seq = seq;
    }
    for (int x = tid; x < R * (D / 8); x += THREADS) {
      const int r = x / (D / 8), d = (x - r * (D / 8)) * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int tok = (row0 + r) / P.g, hg = row0 + r - tok * P.g;
        v = ld_ro(P.q + (sv.a + tok) * P.q_tok + (h * P.g + hg) * P.q_head + d);
      }
      *reinterpret_cast<uint4*>(smem + r * L::kQPitch + d * 2) = v;
    }
    __syncthreads();
    // this lane's rows lr and lr + 8: their tokens (-1: unused, or beyond the unit)
    int tok_of[NT];
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const int row = lr + 8 * r;
      const int tok = row < rows ? (row0 + row) / P.g : -1;
      tok_of[r] = tok >= 0 && ((s_anc[tok][tok >> 5] >> (tok & 31)) & 1u) ? tok : -1;
    }

    for (; base < key1; base += step) {
      const bool more = base + step < key1;
      if (more) page_next = page_at(base + 2 * step);
      // ---- S = Q K^T
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        const uint8_t* qp = smem + lr * L::kQPitch + q_dim<MX>(t, lc) * 2;
        const uint4 qa = *reinterpret_cast<const uint4*>(qp);
        uint4 qb = make_uint4(0, 0, 0, 0);
        if constexpr (NT == 2) qb = *reinterpret_cast<const uint4*>(qp + 8 * L::kQPitch);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint4 kk;
          if constexpr (MX) {
            const uint4 raw = kreg[u][t >> 1];
            // dims (t/2)*64 + lc*16: block (t/2)*2 + lc/2
            const uint32_t sc =
                e8m0_bf16x2(static_cast<uint32_t>(ksc[u] >> (8 * ((t >> 1) * 2 + (lc >> 1)))) & 255u);
            e4m3x4_bf16((t & 1) ? raw.z : raw.x, sc, kk.x, kk.y);
            e4m3x4_bf16((t & 1) ? raw.w : raw.y, sc, kk.z, kk.w);
          } else {
            kk = kreg[u][t];
          }
          mma_bf16(s[u], qa.x, qb.x, qa.y, qb.y, kk.x, kk.y);
          mma_bf16(s[u], qa.z, qb.z, qa.w, qb.w, kk.z, kk.w);
        }
      }
      if (more) load_k(off_next);
      // ---- masks
      const bool tail = base + 16 > sv.ctx;
      uint32_t seen = 0xffffu;  // keys of this step that anybody sees
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] *= P.scale_log2;
      if (tail) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2 * NT; ++e) {
            const int p = base + t * 8 + 2 * lc + (e & 1);
            const int a = p - sv.ctx;
            bool vis = p < sv.ctx;
            if (!vis && p < total && tok_of[e >> 1] >= 0)
              vis = (s_anc[tok_of[e >> 1]][a >> 5] >> (a & 31)) & 1u;
            if (!vis) s[t][e] = -INFINITY;
          }
        const int p = base + (lane & 15), a = p - sv.ctx;
        const bool used =
            p < sv.ctx || (p < total && ((s_anc[a][a >> 5] >> (a & 31)) & 1u));
        seen = __ballot_sync(kFullMask, used);
      }
      // ---- running maximum and sum; the maximum moves only when it has
      // grown by more than 2^8, so o is seldom rescaled
      uint32_t pa[NT][2];
      float now[NT];
      bool grow = false;
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        float m = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
        m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 1));
        now[r] = fmaxf(m, __shfl_xor_sync(kFullMask, m, 2));
        grow |= now[r] > mx[r] + 8.f;
      }
      if (__any_sync(kFullMask, grow)) {
#pragma unroll
        for (int r = 0; r < NT; ++r) {
          const float to = fmaxf(mx[r], now[r]);
          const float w = merge_weight(mx[r], to);
          mx[r] = to;
          sum[r] *= w;
          // o's columns of this lane are rows 2c and 2c+1
          const float w0 = __shfl_sync(kFullMask, w, 8 * lc), w1 = __shfl_sync(kFullMask, w, 8 * lc + 4);
#pragma unroll
          for (int m = 0; m < MTILES; ++m) {
            o[m][r][0] *= w0;
            o[m][r][1] *= w1;
            o[m][r][2] *= w0;
            o[m][r][3] *= w1;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        const float b = mx[r] == -INFINITY ? 0.f : mx[r];
        const float p0 = ex2(s[0][2 * r] - b), p1 = ex2(s[0][2 * r + 1] - b);
        const float p2 = ex2(s[1][2 * r] - b), p3 = ex2(s[1][2 * r + 1] - b);
        sum[r] += (p0 + p1) + (p2 + p3);
        pa[r][0] = pack_bf16x2(make_float2(p0, p1));
        pa[r][1] = pack_bf16x2(make_float2(p2, p3));
      }
      if (tail) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int key = 2 * lc + (t & 1) + (t >> 1) * 8;
          if (base + key < sv.ctx) continue;  // the context, which all rows see: as it is
          const bool vis = (seen >> key) & 1u;
#pragma unroll
          for (int k = 0; k < VV; ++k) {
            if (!vis)
              vreg[t][k] = make_uint4(0, 0, 0, 0);
            else if constexpr (MX)
              vreg[t][k] = clean_codes(vreg[t][k], vsc[t][k], found);
            else
              vreg[t][k] = clean16(vreg[t][k], found);
            if constexpr (MX)
              if (!vis || vsc[t][k] == 255u) vsc[t][k] = 0;
          }
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int k = 0; k < VV; ++k) {
#pragma unroll
        for (int e = 0; e < L::kVDims / 2; ++e) {
          uint32_t w[4];
          if constexpr (MX) {
            // a word of codes gives two pairs: done once for both
            if ((e & 1) == 0) {
              uint32_t lo[4], hi[4];
#pragma unroll
              for (int t = 0; t < 4; ++t)
                e4m3x4_bf16(reinterpret_cast<const uint32_t*>(&vreg[t][k])[e >> 1],
                            e8m0_bf16x2(vsc[t][k]), lo[t], hi[t]);
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t* x = half ? hi : lo;
                const uint32_t a0 = __byte_perm(x[0], x[1], 0x5410), a1 = __byte_perm(x[0], x[1], 0x7632);
                const uint32_t a2 = __byte_perm(x[2], x[3], 0x5410), a3 = __byte_perm(x[2], x[3], 0x7632);
#pragma unroll
                for (int r = 0; r < NT; ++r)
                  mma_bf16(o[k * (L::kVDims / 2) + e + half][r], a0, a1, a2, a3, pa[r][0], pa[r][1]);
              }
            }
          } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = reinterpret_cast<const uint32_t*>(&vreg[t][k])[e];
            const uint32_t a0 = __byte_perm(w[0], w[1], 0x5410), a1 = __byte_perm(w[0], w[1], 0x7632);
            const uint32_t a2 = __byte_perm(w[2], w[3], 0x5410), a3 = __byte_perm(w[2], w[3], 0x7632);
#pragma unroll
            for (int r = 0; r < NT; ++r)
              mma_bf16(o[k * (L::kVDims / 2) + e][r], a0, a1, a2, a3, pa[r][0], pa[r][1]);
          }
        }
      }
      if (more) {
        load_v(off_next);
        off_next = off_at(base + 2 * step, page_next);
      }
    }

    // ---- join the warps
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      sum[r] += __shfl_xor_sync(kFullMask, sum[r], 1);
      sum[r] += __shfl_xor_sync(kFullMask, sum[r], 2);
      if (lc == 0) s_ml[warp][lr + 8 * r] = tok_of[r] >= 0 ? make_float2(mx[r], sum[r]) : make_float2(-INFINITY, 0.f);
    }
    if (found) s_bad = 1;
    __syncthreads();  // Q is no longer read
#pragma unroll
    for (int k = 0; k < VV; ++k)
#pragma unroll
      for (int e = 0; e < L::kVDims / 2; ++e) {
        const int d = k * 8 * L::kVDims + lr * L::kVDims + 2 * e;
#pragma unroll
        for (int r = 0; r < NT; ++r) {
          const float* c = o[k * (L::kVDims / 2) + e][r];
          float* to = s_o + (warp * R + 8 * r + 2 * lc) * (D + 4) + d;
          *reinterpret_cast<float2*>(to) = make_float2(c[0], c[2]);
          *reinterpret_cast<float2*>(to + D + 4) = make_float2(c[1], c[3]);
        }
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == st.kt;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (segment ? 1 : 0);
    for (int x = tid; x < R * (D / 4); x += THREADS) {
      const int r = x / (D / 4), d = (x - r * (D / 4)) * 4;
      if (r >= rows) continue;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) m = fmaxf(m, s_ml[w][r].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) {
        const float2 ml = s_ml[w][r];
        if (ml.x == -INFINITY && ml.y == 0.f) continue;  // saw nothing
        const float f = merge_weight(ml.x, m);
        const float4 v = *reinterpret_cast<const float4*>(s_o + (w * R + r) * (D + 4) + d);
        l += ml.y * f;
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
      }
      const int tok = (row0 + r) / P.g, hq = h * P.g + row0 + r - tok * P.g;
      if (s_bad) {
        float* a = &acc.x;
        for (int u = 0; u < 4; ++u)
          a[u] = restore_nonfinite<MX>(P, seq, sv.ctx, sv.n, h, s_anc[tok], t0 * kRowsTile, key1,
                                       d + u, a[u]);
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint2 v;
        v.x = pack_bf16x2(make_float2(acc.x * inv, acc.y * inv));
        v.y = pack_bf16x2(make_float2(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2*>(P.out + (sv.a + tok) * P.o_tok + hq * P.o_head + d) = v;
        if (d == 0 && P.lse)
          P.lse[(sv.a + tok) * P.HQ + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(P.part_o + (slot * R + r) * D + d) = acc;
        if (d == 0) P.part_ml[slot * R + r] = make_float2(m, l);
      }
    }
    __syncthreads();
    if (tid == 0) s_bad = 0;
    cur += t1 - t0;
    ++segment;
  }
}

// ------------------------------------------------------------------- the join
//
// Few rows (split): grid (num_seqs * M-tiles, H, rows), a block a row, its four warps a
// quarter of the parts each; there can be a part a CTA (8192 tokens, one
// row: 74; 33 us a call with a warp a row, 24 so).  More rows: grid (.., rows / 4), a warp a
// row, as its parts are few (32 ragged trees: 224 us with a block a row, 185 so).  A unit
// that one CTA finished is skipped.
template <int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const AttendParams P, int R, int tile,
                                                          int mtiles, int split) {
  grid_dependency_wait();
  allow_dependent_launch();
  constexpr int V = D / 32;  // dims a lane
  __shared__ float2 s_ml[4];
  __shared__ float s_o[4][D];
  const int seq = blockIdx.x / mtiles, mt = blockIdx.x - seq * mtiles, h = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = split ? blockIdx.z : blockIdx.z * 4 + warp;
  const int w0 = split ? warp : 0, ws = split ? 4 : 1;  // this warp's parts
  const SeqView sv = seq_view(P.s, seq, false);
  const SeqTiles st = seq_tiles(sv, P.g, P.H, R, tile);
  if (mt >= st.mt || r >= R || mt * R + r >= sv.n * P.g) return;
  const int64_t total = P.prefix[P.s.num_seqs];
  const int extra = static_cast<int>(P.prefix[P.s.num_seqs + 1]);
  // the unit's first step, and its first tile's
  const int64_t u0 = P.prefix[seq] + (static_cast<int64_t>(h) * st.mt + mt) * (st.kt + extra);
  const int64_t t0 = u0 + extra;
  const int parts = static_cast<int>(min(static_cast<int64_t>(P.parts), total));
  const int c0 = range_of(t0, total, parts), c1 = range_of(t0 + st.kt - 1, total, parts);
  if (c0 == c1) return;
  const int64_t first = 2 * static_cast<int64_t>(c0) + (range_start(c0, total, parts) >= u0 ? 0 : 1);
  auto at = [&](int c) { return (c == c0 ? first : 2 * static_cast<int64_t>(c)) * R + r; };
  // the maximum over this warp's parts, a lane a part
  float m = -INFINITY;
  for (int c = c0 + w0 + ws * lane; c <= c1; c += 32 * ws) m = fmaxf(m, P.part_ml[at(c)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, d));
  float acc[V], l = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll 8
  for (int c = c0 + w0; c <= c1; c += ws) {
    const int64_t a = at(c);
    const float2 ml = P.part_ml[a];
    const float f = merge_weight(ml.x, m);
    float v[V];
    if constexpr (V == 2) {
      const float2 x = *reinterpret_cast<const float2*>(P.part_o + a * D + lane * V);
      v[0] = x.x;
      v[1] = x.y;
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const float4 x = *reinterpret_cast<const float4*>(P.part_o + a * D + lane * V + e);
        v[e] = x.x;
        v[e + 1] = x.y;
        v[e + 2] = x.z;
        v[e + 3] = x.w;
      }
    }
    const bool none = ml.x == -INFINITY && ml.y == 0.f;
    l += none ? 0.f : ml.y * f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = none ? acc[e] : fmaf(v[e], f, acc[e]);
  }
  const int row = mt * R + r, tok = row / P.g, hq = h * P.g + row - tok * P.g;
  uint16_t* to = P.out + (sv.a + tok) * P.o_tok + hq * P.o_head;
  if (!split) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < V; e += 2)
      *reinterpret_cast<uint32_t*>(to + lane * V + e) =
          pack_bf16x2(make_float2(acc[e] * inv, acc[e + 1] * inv));
    if (lane == 0 && P.lse)
      P.lse[(sv.a + tok) * P.HQ + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    return;
  }
  if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
  for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = acc[e];
  __syncthreads();
  const float top = fmaxf(fmaxf(s_ml[0].x, s_ml[1].x), fmaxf(s_ml[2].x, s_ml[3].x));
  float sum = 0.f, f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool none = s_ml[k].x == -INFINITY && s_ml[k].y == 0.f;
    f[k] = none ? 0.f : merge_weight(s_ml[k].x, top);
    sum += none ? 0.f : s_ml[k].y * f[k];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int d = 2 * threadIdx.x; d < D; d += 256) {
    float o[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      o[e] = fmaf(s_o[3][d + e], f[3], fmaf(s_o[2][d + e], f[2],
                  fmaf(s_o[1][d + e], f[1], s_o[0][d + e] * f[0])));
    *reinterpret_cast<uint32_t*>(to + d) = pack_bf16x2(make_float2(o[0] * inv, o[1] * inv));
  }
  if (threadIdx.x == 0 && P.lse)
    P.lse[(sv.a + tok) * P.HQ + hq] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

}  // namespace sconv
