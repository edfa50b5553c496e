// Kernel instances of the drafted-tree entry points, picked at run time
// (inst_tree_step.cu, inst_attend.cu, inst_evict.cu).
#pragma once
#include "tree_params.h"

namespace sconv {

using TreeStepFn = void (*)(TreeStepParams);
using AttendFn = void (*)(AttendParams);
using JoinFn = void (*)(AttendParams, int, int, int);
using WeighFn = void (*)(WeighParams);

// nullptr for an unsupported combination.
TreeStepFn pick_tree_step(int W, int D, bool mx, bool lv);
AttendFn pick_attend_rows(int D, int nt, bool mx);
JoinFn pick_attend_join(int D);
WeighFn pick_weigh(int D, bool mx);
void (*accept_fn())(AcceptParams);
void (*evict_select_fn())(EvictParams);
void (*evict_move_fn())(EvictParams);

// Dynamic shared memory of attend_rows_kernel: Q, then the warps' results.
inline size_t attend_rows_smem(int D, int nt) {
  return static_cast<size_t>(kRowsWarps) * 8 * nt * (D + 4) * 4;
}
inline size_t weigh_smem(int D) { return static_cast<size_t>(D == 256 ? 64 : 128) * (2 * D + 64); }

}  // namespace sconv
