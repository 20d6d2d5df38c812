// qmm_moe_layer_bf16.cu -- the mixture-of-experts layer with bf16 activations
#include "qmm_moe_layer.cuh"

namespace qmm {

cudaError_t launch_moe_layer_bf16(const MoePlan& pl, const MoeParams& p, int smem_max, cudaStream_t s) {
    return pl.token ? moe_layer_go<true, false, true>(pl, p, smem_max, s) : moe_layer_go<true, false, false>(pl, p, smem_max, s);
}

}  // namespace qmm
