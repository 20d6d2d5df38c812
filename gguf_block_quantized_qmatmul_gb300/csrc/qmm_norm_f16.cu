// qmm_norm_f16.cu -- norms around a block, f16
#include "qmm_norm.cuh"

namespace qmm {

cudaError_t launch_block_norm_f16(const NormParams& p, cudaStream_t s) { return norm_go<X_F16>(p, s); }

}  // namespace qmm
