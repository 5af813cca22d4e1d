// The 8-bit instances of attention of drafted trees (see gdn_tree.cu).
#include "gdn_tree_tc.cuh"

namespace gdn {
cudaError_t launch_tree_f8(const TreeArgs& A, const TreePlan& plan, cudaStream_t st) { return tree_tc_type<__nv_fp8_e4m3>(A, plan, st); }
int tree_status_f8() { return take_gave_up(); }
cudaError_t tree_wait_out_f8(int32_t limit_us, cudaStream_t st) { return launch_wait_out(limit_us, st); }
}  // namespace gdn
