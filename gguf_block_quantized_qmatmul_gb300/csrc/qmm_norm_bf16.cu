// qmm_norm_bf16.cu -- norms around a block, bf16
#include "qmm_norm.cuh"

namespace qmm {

cudaError_t launch_block_norm_bf16(const NormParams& p, cudaStream_t s) { return norm_go<X_BF16>(p, s); }

}  // namespace qmm
