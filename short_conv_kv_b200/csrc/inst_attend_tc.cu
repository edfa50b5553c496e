// Instances of the tensor-memory kernels: attention for many query rows, and the
// attention weights.
#include "attend_tc.cuh"
#include "weigh_tc.cuh"
#include "tree_instances.h"

namespace sconv {

template <int D, bool MX>
AttendTc tc_of(int rows) {
  using T = TcShape<D>;
  using F = FeedShape<D, T::kKeys, MX>;
  AttendTc A;
  A.fn = &attend_tc_kernel<D, MX>;
  A.threads = tc_threads<D, MX>();
  A.rows = T::kStreams * 128;
  if (rows <= 128) A.rows = 128;
  A.tile = T::kKeys;
  // what Q and the raw pieces leave of 227 KB (less the static part and the
  // alignment), at most 8 units
  const int fixed = A.rows * D * 2 + F::kRawBytes + 1024;
  const int room = (227 * 1024 - 5632 - fixed) / F::kUnit;
  A.units = room > 8 ? 8 : room;
  A.smem = static_cast<size_t>(fixed) + static_cast<size_t>(A.units) * F::kUnit;
  return A;
}

template <int D, bool MX>
WeighTc weigh_tc_of(int rows) {
  using F = FeedShape<D, 128, MX>;
  WeighTc A;
  A.fn = &weigh_tc_kernel<D, MX>;
  A.threads = weigh_tc_threads<MX>();
  A.rows = rows >= kWeighRows ? kWeighRows : (rows + 15) / 16 * 16;
  const int fixed = (A.rows * D * 2 + 1023) / 1024 * 1024 + F::kRawBytes + 1024;
  const int room = (227 * 1024 - 7168 - fixed) / F::kUnit;
  A.units = room > 8 ? 8 : room;
  A.smem = static_cast<size_t>(fixed) + static_cast<size_t>(A.units) * F::kUnit;
  return A;
}

WeighTc pick_weigh_tc(int D, bool mx, int rows) {
  if (D == 64) return mx ? weigh_tc_of<64, true>(rows) : weigh_tc_of<64, false>(rows);
  return mx ? weigh_tc_of<128, true>(rows) : weigh_tc_of<128, false>(rows);
}

AttendTc pick_attend_tc(int D, bool mx, int rows) {
  switch (D) {
    case 64: return mx ? tc_of<64, true>(rows) : tc_of<64, false>(rows);
    case 128: return mx ? tc_of<128, true>(rows) : tc_of<128, false>(rows);
    default: return mx ? tc_of<256, true>(rows) : tc_of<256, false>(rows);
  }
}

}  // namespace sconv
