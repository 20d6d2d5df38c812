// qmm_moe_layer_f32.cu -- the mixture-of-experts layer with f32 activations
#include "qmm_moe_layer.cuh"

namespace qmm {

cudaError_t launch_moe_layer_f32(const MoePlan& pl, const MoeParams& p, int smem_max, cudaStream_t s) {
    return pl.token ? moe_layer_go<true, true, true>(pl, p, smem_max, s) : moe_layer_go<true, true, false>(pl, p, smem_max, s);
}

}  // namespace qmm
