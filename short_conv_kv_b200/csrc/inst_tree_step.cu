// Instances of the drafted-tree step, and the acceptance kernel.
#include "instances.h"
#include "tree_instances.h"
#include "tree_step.cuh"

namespace sconv {

#define SCONV_TREE_FOR(WW, DD) (&tree_step_kernel<WW, DD, MX, LV>)

template <bool MX, bool LV>
TreeStepFn pick_tree_step_t(int W, int D) { SCONV_PICK_BY_W_D(SCONV_TREE_FOR) }

TreeStepFn pick_tree_step(int W, int D, bool mx, bool lv) {
  if (mx) return lv ? pick_tree_step_t<true, true>(W, D) : pick_tree_step_t<true, false>(W, D);
  return lv ? pick_tree_step_t<false, true>(W, D) : pick_tree_step_t<false, false>(W, D);
}

void (*accept_fn())(AcceptParams) { return &tree_accept_kernel; }

}  // namespace sconv
