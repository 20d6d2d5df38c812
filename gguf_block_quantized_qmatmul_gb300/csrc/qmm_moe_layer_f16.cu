// qmm_moe_layer_f16.cu -- the mixture-of-experts layer with f16 activations
#include "qmm_moe_layer.cuh"

namespace qmm {

cudaError_t launch_moe_layer_f16(const MoePlan& pl, const MoeParams& p, int smem_max, cudaStream_t s) {
    return pl.token ? moe_layer_go<false, false, true>(pl, p, smem_max, s) : moe_layer_go<false, false, false>(pl, p, smem_max, s);
}

}  // namespace qmm
