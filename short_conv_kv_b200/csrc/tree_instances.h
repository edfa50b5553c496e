// Kernel instances of the drafted-tree entry points, picked at run time
// (inst_tree_step.cu, inst_attend.cu, inst_attend_tc.cu, inst_evict.cu).
#pragma once
#include "tree_params.h"

namespace sconv {

using TreeStepFn = void (*)(TreeStepParams, int);
using AttendFn = void (*)(AttendParams);
using JoinFn = void (*)(AttendParams, int, int, int, int);
using AttendTcFn = void (*)(AttendParams, int, int);
using MoveFn = void (*)(EvictParams);
using WeighFn = void (*)(WeighParams);

// nullptr for an unsupported combination.
TreeStepFn pick_tree_step(int W, int D, bool mx, bool lv);
AttendFn pick_attend_rows(int D, int nt, bool mx);
// attend_tc_kernel for up to `rows` query rows a K/V head: its threads, rows a unit,
// keys a tile, units in the ring and dynamic shared memory.
struct AttendTc {
  AttendTcFn fn;
  int threads;
  int rows;
  int tile;
  int units;
  size_t smem;
};
AttendTc pick_attend_tc(int D, bool mx, int rows);
JoinFn pick_attend_join(int D);
WeighFn pick_weigh(int D, bool mx);
// weigh_tc_kernel (head_dim 64, 128; more than 16 rows) for up to `rows` query rows a K/V head: its threads, rows
// a pass, units in the ring and dynamic shared memory.
struct WeighTc {
  void (*fn)(WeighParams, int, int);
  int threads;
  int rows;
  int units;
  size_t smem;
};
WeighTc pick_weigh_tc(int D, bool mx, int rows);
void (*accept_fn())(AcceptParams);
const void* evict_select_fn();  // (EvictParams, int room)
MoveFn pick_evict_move(int D, bool mx);

// Dynamic shared memory of attend_rows_kernel: Q, then the warps' results.
inline size_t attend_rows_smem(int D, int nt) {
  return static_cast<size_t>(kRowsWarps) * 8 * nt * (D + 4) * 4;
}
inline size_t weigh_smem(int D) { return static_cast<size_t>(D == 256 ? 64 : 16) * (2 * D + 64); }

}  // namespace sconv
