// Fifth-generation tensor cores (sm_100a): tensor memory, matrix
// instructions, descriptors, and the producer that feeds them with rows of
// the paged cache.
#pragma once
#include "attend.cuh"

namespace sconv {

constexpr uint64_t kTcTimeoutNs = 1000000000ull;

// mbar_wait() for the roles of these kernels: abort[2] counts work that may hold a warpgroup up for longer than
// the limit (rows that are done again, attend_tc.cuh); the limit runs from its last step, so a wait ends
// when that work has.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = global_ns();
  int step = 0;
  while (true) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (global_ns() - t0 > kTcTimeoutNs) {
      const int now = abort[2];
      if (now == step) {
        *abort = 1;
        return false;
      }
      step = now;
      t0 = global_ns();
    }
  }
}

// ------------------------------------------------------------ tensor memory

__device__ __forceinline__ void tmem_alloc(uint32_t* to, uint32_t cols) {  // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(to)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 columns of this warp's 32 lanes: thread l gets lane l.
__device__ __forceinline__ void tmem_ld32(float (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]),
        "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]),
        "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(at));
}
// The registers of a load are only defined behind tmem_wait_ld(); this ties
// their uses to it.
__device__ __forceinline__ void tmem_landed(float (&r)[32]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(r[i]));
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const float (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
      "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]),
      "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]), "f"(r[19]), "f"(r[20]), "f"(r[21]),
      "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]),
      "f"(r[29]), "f"(r[30]), "f"(r[31])
      : "memory");
}

// --------------------------------------------------------- matrix products

// Shared-memory operand in 128-byte swizzled atoms (8 rows of 128 bytes, 16-byte
// chunk c of row r at chunk c ^ (r & 7)), atoms 1024 bytes apart along the
// rows; `lead` is the distance of the next 64 columns where the columns are the
// product's M or N dimension (unused where they are its K dimension).
// The low half holds the address and `lead` (so the operand moves by adding 16-byte
// units to it), the high half is constant.
__device__ __forceinline__ uint32_t tc_desc(uint32_t addr, uint32_t lead) {
  return (addr >> 4) | ((lead >> 4) << 16);
}
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
// bf16 x bf16 -> fp32, M rows, N columns; b_rows: B's rows are its K dimension.
__host__ __device__ constexpr uint32_t tc_idesc(int M, int N, bool b_rows) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_rows ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 y, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh), "r"(accumulate)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}
// Arrive on `bar` when the products issued so far by this thread are complete.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// --------------------------------------------------------- async copies

// 16 bytes (or 16 zero bytes) to shared memory.
__device__ __forceinline__ void cp16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from),
               "r"(there ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// One of `bar`'s arrivals, made when this thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void async_proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts1(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Four E4M3 codes to bf16 pairs, bytes 0 and 2 to `even`, 1 and 3 to `odd`: the bits
// as in e4m3x4_bf16, and one multiplication: `both` is 2^120 times the scale, which
// needs a scale byte of 134 (2^7) at most.  NaN codes (0x7f, 0xff) come out
// finite; they leave bit 7 of a half of `nan.x`, or bit 11 of one of `nan.y`.
// The integer pipe bounds this (half the rate of the others), so what can be
// is a multiply-add: `sixteen` and `one` are registers to keep it so.
__device__ __forceinline__ void e4m3x4_bf16_fast(uint32_t w, uint32_t both, uint32_t sixteen,
                                                 uint32_t one, uint32_t& even, uint32_t& odd,
                                                 uint2& nan) {
  const uint32_t te = w & 0x007f007fu, to = (w >> 4) & 0x07f007f0u;
  const uint32_t se = w & 0x00800080u;
  uint32_t e, ne, no;
  asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(e) : "r"(se), "r"(sixteen), "r"(te));
  asm("mul.lo.u32 %0, %1, %2;" : "=r"(e) : "r"(e), "r"(sixteen));
  asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(ne) : "r"(te), "r"(one), "r"(0x00010001u));
  asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(no) : "r"(to), "r"(one), "r"(0x00100010u));
  nan.x |= ne;
  nan.y |= no;
  even = bf16x2_mul(e, both);
  odd = bf16x2_mul((w & 0x80008000u) | to, both);
}
// The order in which a decoded unit holds its columns (and Q then too): the
// middle two of every four are swapped.
template <bool MX>
__device__ __forceinline__ uint4 tc_order(const uint4& v) {
  if constexpr (!MX) return v;
  return make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                    __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
}

// Sixteen codes with any scale byte, NaN codes among them (rare).  With `clean`, NaN
// and infinities become 0; returns whether there were any.
__device__ __noinline__ bool e4m3x16_slow(uint4 w, uint32_t sb, bool clean, uint4* out) {
  const uint32_t sc = e8m0_bf16x2(sb);
  uint4 a, b;
  e4m3x4_bf16(w.x, sc, a.x, a.y);
  e4m3x4_bf16(w.y, sc, a.z, a.w);
  e4m3x4_bf16(w.z, sc, b.x, b.y);
  e4m3x4_bf16(w.w, sc, b.z, b.w);
  bool bad = false;
  if (clean) {
    a = clean16(a, bad);
    b = clean16(b, bad);
  }
  out[0] = tc_order<true>(a);
  out[1] = tc_order<true>(b);
  return bad;
}

// ------------------------------------------------------------ the producers
//
// A unit is a tile of KEYS cache rows of one K/V head, K's or V's, as bf16 in swizzled
// shared memory: [D / 64][KEYS][64], each block of 64 columns in 128-byte
// atoms.  Rows come through the block table, so they are gathered 16 bytes a
// copy (any page size, any strides).
//
// bf16: four warps bring KEYS / 4 rows each.  Copies land in place and arrive on the
// unit's barrier by themselves, so the ring is in flight but for the units in
// use.  (The thread that issues the products fences the proxies behind its wait.)
// MXFP8: three warps bring the codes and scale bytes to a raw ring of kRaw
// units, eight warps write them to the unit as bf16 (exact).  (With one kind of
// warp for both, the addresses and copies stood between a unit's decoding and the
// next one's: 3,200 cycles a unit, so 2,030.)
//
// One call site brings all units: several copies of this code, with the
// softmax's, fall out of the instruction cache.

struct FeedRing {
  uint32_t units;  // shared-memory address of the first unit
  uint64_t* full;
  uint64_t* empty;
  volatile int* abort;  // [1]: a V row was cleaned; [2]: as tc_wait() has it
  int count;            // units in the ring

  int slot = 0, phase = 0;  // the unit to fill next
  bool wrapped = false, ok = true;

  __device__ __forceinline__ void wait_empty() {
    if (wrapped && ok && !tc_wait(empty + slot, phase, abort)) ok = false;
  }
  __device__ __forceinline__ void advance() {
    if (++slot == count) {
      slot = 0;
      if (wrapped) phase ^= 1;
      wrapped = true;
    }
  }
};

// Threads that make a unit, those that fetch its raw bytes, and what they hold
// of shared memory besides.
template <int D, int KEYS, bool MX>
struct FeedShape {
  static constexpr int kWarps = MX ? 8 : 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kUnit = KEYS * D * 2;
  static constexpr int kKeysWarp = KEYS / kWarps;  // rows of a warp
  static constexpr int kBlocks = D / 64;
  // a warp's step: 4 (MXFP8) or 8 pieces of 16 bytes of 8 or 4 rows, one block
  static constexpr int kCols = MX ? 4 : 8;
  static constexpr int kRowsStep = 32 / kCols;
  static constexpr int kSteps = kKeysWarp / kRowsStep;
  static constexpr int kRaw = 3;          // units in the raw ring
  static constexpr int kFetchWarps = 3;
  static constexpr int kScaleRow = 16;    // bytes of a raw row's scales
  static constexpr int kRawUnit = MX ? KEYS * (D + kScaleRow) : 0;
  static constexpr int kRawBytes = kRaw * kRawUnit;
  static_assert(kKeysWarp % kRowsStep == 0, "");
};

template <int D, int KEYS>
struct FeedBf16 : FeedShape<D, KEYS, false> {
  using S = FeedShape<D, KEYS, false>;
  // One unit: off8 is the offset, in units of 8 elements, of the row of key
  // warp * kKeysWarp + lane % kKeysWarp, ~0u for a row of zeros; rows at or behind
  // `clean` lose NaN and infinities.
  static __device__ __forceinline__ void bring(FeedRing& R, int warp, int lane,
                                               const uint8_t* base, uint32_t off8, int clean) {
    R.wait_empty();
    const int chunk = lane % S::kCols;
    const uint8_t* col = base + chunk * 16;
    const int row0 = warp * S::kKeysWarp + lane / S::kCols;
    auto place = [&](int j, int b) {
      const int key = row0 + j * S::kRowsStep;
      return R.units + R.slot * S::kUnit + b * (KEYS * 128) + key * 128 +
             ((chunk ^ (key & 7)) << 4);
    };
#pragma unroll
    for (int j = 0; j < S::kSteps; ++j) {
      const uint32_t o = __shfl_sync(kFullMask, off8, j * S::kRowsStep + lane / S::kCols);
      const uint8_t* from = col + (o == ~0u ? 0 : static_cast<uint64_t>(o) * 16);
#pragma unroll
      for (int b = 0; b < S::kBlocks; ++b)
        if (R.ok) cp16(place(j, b), from + b * 128, o != ~0u);
    }
    if (clean >= KEYS) {
      cp_arrive(R.full + R.slot);
    } else {
      cp_commit();
      cp_wait<0>();
#pragma unroll 1
      for (int j = 0; j < S::kSteps; ++j) {
        if (row0 + j * S::kRowsStep < clean) continue;
#pragma unroll 1
        for (int b = 0; b < S::kBlocks; ++b) {
          bool bad = false;
          const uint4 v = clean16(lds16(place(j, b)), bad);
          if (bad) {
            sts16(place(j, b), v);
            R.abort[1] = 1;
          }
        }
      }
      async_proxy_fence();
      mbar_arrive(R.full + R.slot);
    }
    R.advance();
  }
};

// Raw unit: codes [D / 64][KEYS][64], then the scales, kScaleRow bytes a row from
// its first aligned word on.  The scale bytes begin `low` bytes into
// that word, the same for all rows (`words`), or at 0, copied one by one.
template <int D, int KEYS>
struct FeedMx : FeedShape<D, KEYS, true> {
  using S = FeedShape<D, KEYS, true>;
  static constexpr int kGroups = KEYS / 8;  // of eight rows
  static constexpr int kMine = (kGroups + S::kFetchWarps - 1) / S::kFetchWarps;
  static constexpr int kScales = KEYS * D;  // where a raw unit's scales begin

  // Fetching warp w's part of a raw unit: the rows of keys kStep * i + w * 8 + lane / 4
  // at offsets off[i] (units of 8 elements); zeros for keys from `left` on.
  static constexpr int kStep = 8 * S::kFetchWarps;
  static __device__ __forceinline__ void fetch(FeedRing& R, int w, int lane, const uint8_t* base,
                                               const uint8_t* scales, bool words,
                                               const uint32_t (&off)[kMine], int left) {
    R.wait_empty();
    const int c = lane & 3, key = w * 8 + (lane >> 2);
    const uint32_t unit = R.units + R.slot * S::kRawUnit;
    const uint32_t to = unit + w * 512 + lane * 16;
    const uint32_t st = unit + kScales + key * S::kScaleRow + c * 4;
    const uint8_t* from = base + c * 16;
    if (R.ok && words) {
      const int low = static_cast<int>(reinterpret_cast<uintptr_t>(scales) & 3u);
      const bool mine = c * 4 < low + D / 32;
      const uint8_t* sp = scales - low + c * 4;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        if (i == kMine - 1 && kGroups % S::kFetchWarps && w + S::kFetchWarps * i >= kGroups) break;
        const bool there = key + i * kStep < left;
        const uint8_t* f = from + static_cast<uint64_t>(off[i]) * 8;
#pragma unroll
        for (int b = 0; b < S::kBlocks; ++b)
          cp16(to + b * (KEYS * 64) + i * (S::kFetchWarps * 512), f + b * 64, there);
        if (mine) cp4(st + i * (kStep * S::kScaleRow), sp + (off[i] >> 2), there);
      }
      cp_arrive(R.full + R.slot);
    } else {
      if (R.ok) {
#pragma unroll 1
        for (int i = 0; i < kMine && w + S::kFetchWarps * i < kGroups; ++i) {
          uint32_t o = 0;
#pragma unroll
          for (int k = 0; k < kMine; ++k) o = k == i ? off[k] : o;
          const bool there = key + i * kStep < left;
          const uint8_t* f = from + static_cast<uint64_t>(o) * 8;
#pragma unroll 1
          for (int b = 0; b < S::kBlocks; ++b)
            cp16(to + b * (KEYS * 64) + i * (S::kFetchWarps * 512), f + b * 64, there);
          for (int b = c; b < D / 32; b += 4)
            sts1(st - c * 4 + i * (kStep * S::kScaleRow) + b,
                 there ? __ldg(scales + (o >> 2) + b) : 0u);
        }
      }
      cp_commit();
      cp_wait<0>();
      mbar_arrive(R.full + R.slot);
    }
    R.advance();
  }

  // The next raw unit to the next unit.
  static __device__ __forceinline__ void decode(FeedRing& R, FeedRing& Raw, int warp, int lane,
                                                int low, int clean) {
    if (Raw.ok && !tc_wait(Raw.full + Raw.slot, Raw.phase, Raw.abort)) Raw.ok = false;
    R.wait_empty();
    if (R.ok && Raw.ok) {
      const int chunk = (lane & 3) * 2, row0 = warp * S::kKeysWarp + (lane >> 2);
      uint32_t sixteen = 16u, one = 1u;
      asm volatile("" : "+r"(sixteen), "+r"(one));
      const uint32_t raw = Raw.units + Raw.slot * S::kRawUnit;
      auto place = [&](int j, int b, int c) {
        const int key = row0 + j * 8;
        return R.units + R.slot * S::kUnit + b * (KEYS * 128) + key * 128 + ((c ^ (key & 7)) << 4);
      };
      constexpr int kPieces = S::kSteps * S::kBlocks;
      uint4 w[kPieces];
      uint32_t sb[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int j = i / S::kBlocks, b = i % S::kBlocks;
        w[i] = lds16(raw + b * (KEYS * 64) + (row0 + j * 8) * 64 + (lane & 3) * 16);
        sb[i] = lds1(raw + kScales + (row0 + j * 8) * S::kScaleRow + low + b * 2 + ((lane & 3) >> 1));
      }
      uint2 nan = make_uint2(0u, 0u);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int j = i / S::kBlocks, b = i % S::kBlocks;
        const uint32_t both = (sb[i] + 120u) * 0x00800080u;
        uint4 x, y;
        e4m3x4_bf16_fast(w[i].x, both, sixteen, one, x.x, x.y, nan);
        e4m3x4_bf16_fast(w[i].y, both, sixteen, one, x.z, x.w, nan);
        e4m3x4_bf16_fast(w[i].z, both, sixteen, one, y.x, y.y, nan);
        e4m3x4_bf16_fast(w[i].w, both, sixteen, one, y.z, y.w, nan);
        top = max(top, sb[i]);
        sts16(place(j, b, chunk), x);
        sts16(place(j, b, chunk + 1), y);
      }
      if ((nan.x & 0x00800080u) || (nan.y & 0x08000800u) || top > 134u) {  // rare: once more
#pragma unroll 1
        for (int i = 0; i < kPieces; ++i) {
          const int j = i / S::kBlocks, b = i % S::kBlocks;
          const uint4 v = lds16(raw + b * (KEYS * 64) + (row0 + j * 8) * 64 + (lane & 3) * 16);
          const uint32_t s = lds1(raw + kScales + (row0 + j * 8) * S::kScaleRow + low + b * 2 + ((lane & 3) >> 1));
          uint4 x[2];
          if (e4m3x16_slow(v, s, row0 + j * 8 >= clean, x)) R.abort[1] = 1;
          sts16(place(j, b, chunk), x[0]);
          sts16(place(j, b, chunk + 1), x[1]);
        }
      }
    }
    async_proxy_fence();
    mbar_arrive(R.full + R.slot);
    R.advance();
    mbar_arrive(Raw.empty + Raw.slot);
    if (++Raw.slot == Raw.count) {
      Raw.slot = 0;
      Raw.phase ^= 1;
    }
  }
};

// Unit u of a segment of `tiles` key tiles, in the order in which the products need
// them: K0 V0 K1 V1 .. for a pair of streams, K0 K1 V0 K2 V1 .. otherwise.
__device__ __forceinline__ void unit_of(int u, int tiles, bool pair, bool& is_v, int& t) {
  const int w = !pair && u == 2 * tiles - 1 ? u + 1 : u;
  is_v = pair ? w & 1 : w > 0 && !(w & 1);
  t = pair ? w >> 1 : is_v ? (w >> 1) - 1 : (w + 1) >> 1;
}

}  // namespace sconv
