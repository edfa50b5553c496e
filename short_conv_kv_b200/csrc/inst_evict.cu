// The eviction kernels.
#include "tree_instances.h"
#include "evict.cuh"

namespace sconv {

void (*evict_select_fn())(EvictParams) { return &evict_select_kernel; }
void (*evict_move_fn())(EvictParams) { return &evict_move_kernel; }

}  // namespace sconv
