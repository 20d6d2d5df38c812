// qmm_moe_layer_bf16.cu -- the mixture-of-experts layer on bf16 warp MMAs
#include "qmm_moe_layer.cuh"

namespace qmm {

cudaError_t launch_moe_layer_bf16(const MoePlan& pl, const MoeParams& p, int smem_max, cudaStream_t s) {
    return pl.down.by_slot ? moe_layer_go<1, true, true>(pl, p, smem_max, s)
           : pl.nb == 1    ? moe_layer_go<1, true, false>(pl, p, smem_max, s)
                           : moe_layer_go<2, true, false>(pl, p, smem_max, s);
}

}  // namespace qmm
