// The eviction kernels.
#include "tree_instances.h"
#include "evict.cuh"

namespace sconv {

const void* evict_select_fn() { return reinterpret_cast<const void*>(&evict_select_kernel); }

MoveFn pick_evict_move(int D, bool mx) {
  switch (D) {
    case 64: return mx ? &evict_move_kernel<64, true, uint16_t> : &evict_move_kernel<128, false, uint16_t>;
    case 128: return mx ? &evict_move_kernel<128, true, uint32_t> : &evict_move_kernel<256, false, uint16_t>;
    case 256: return mx ? &evict_move_kernel<256, true, uint64_t> : &evict_move_kernel<512, false, uint16_t>;
    default: return nullptr;
  }
}

}  // namespace sconv
