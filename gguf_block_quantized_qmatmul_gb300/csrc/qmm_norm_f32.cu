// qmm_norm_f32.cu -- norms around a block, f32
#include "qmm_norm.cuh"

namespace qmm {

cudaError_t launch_block_norm_f32(const NormParams& p, cudaStream_t s) { return norm_go<X_F32>(p, s); }

}  // namespace qmm
