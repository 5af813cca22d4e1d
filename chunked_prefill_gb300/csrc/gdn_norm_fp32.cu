// The fp32 instances of the RMS norm's kernels (see gdn_norm.cu).
#include "gdn_norm.cuh"

namespace gdn {
cudaError_t norm_fwd_fp32(const NormArgs& A, cudaStream_t st) { return fwd_type<float>(A, st); }
cudaError_t norm_bwd_fp32(const NormArgs& A, int& parts, cudaStream_t st) { return bwd_type<float>(A, parts, st); }
}  // namespace gdn
