// Instances of the attention kernels for few query rows, the join and the
// attention weights.
#include "tree_instances.h"
#include "weigh.cuh"

namespace sconv {

AttendFn pick_attend_rows(int D, int nt, bool mx) {
#define SCONV_ROWS(DD)                                                                   \
  (nt == 1 ? (mx ? &attend_rows_kernel<DD, 1, true> : &attend_rows_kernel<DD, 1, false>) \
           : (mx ? &attend_rows_kernel<DD, 2, true> : &attend_rows_kernel<DD, 2, false>))
  switch (D) {
    case 64: return SCONV_ROWS(64);
    case 128: return SCONV_ROWS(128);
    case 256:
      if (nt == 1) return mx ? &attend_rows_kernel<256, 1, true> : &attend_rows_kernel<256, 1, false>;
      return nullptr;
    default: return nullptr;
  }
}

JoinFn pick_attend_join(int D) {
  return D == 64 ? &attend_join_kernel<64>
                 : D == 128 ? &attend_join_kernel<128> : D == 256 ? &attend_join_kernel<256> : nullptr;
}

WeighFn pick_weigh(int D, bool mx) {
  switch (D) {
    case 64: return mx ? &weigh_kernel<64, true> : &weigh_kernel<64, false>;
    case 128: return mx ? &weigh_kernel<128, true> : &weigh_kernel<128, false>;
    default: return mx ? &weigh_kernel<256, true> : &weigh_kernel<256, false>;
  }
}

}  // namespace sconv
