// The bf16 instances of attention of drafted trees (see gdn_tree.cu).
#include "gdn_tree_tc.cuh"

namespace gdn {
cudaError_t launch_tree_bf16(const TreeArgs& A, const TreePlan& plan, cudaStream_t st) { return tree_tc_type<__nv_bfloat16>(A, plan, st); }
int tree_status_bf16() { return take_gave_up(); }
cudaError_t tree_wait_out_bf16(int32_t limit_us, cudaStream_t st) { return launch_wait_out(limit_us, st); }
}  // namespace gdn
