// The bf16 instances of the paged attention kernels (see gdn_paged.cu).
#include "gdn_paged_mma.cuh"

namespace gdn {
cudaError_t launch_paged_bf16(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) { return launch_type<__nv_bfloat16>(A, plan, st); }
PagedShape paged_shape_bf16(int D) { return shape_type<__nv_bfloat16>(D); }
}  // namespace gdn
