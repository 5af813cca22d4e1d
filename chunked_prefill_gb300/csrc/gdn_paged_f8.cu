// The 8-bit instances of the paged attention kernels (see gdn_paged.cu).
#include "gdn_paged_mma.cuh"

namespace gdn {
cudaError_t launch_paged_f8(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) { return launch_type<__nv_fp8_e4m3>(A, plan, st); }
PagedShape paged_shape_f8(int D) { return shape_type<__nv_fp8_e4m3>(D); }
}  // namespace gdn
