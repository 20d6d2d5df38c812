// qmm_norm.cu -- host side of the norms around a block (qmm_norm.cuh)
#include "qmm_q8c.cuh"

namespace qmm {

cudaError_t launch_block_norm(const NormCall& c, cudaStream_t s) {
    NormParams p = {c, 0};
    const uintptr_t x = (uintptr_t)x_size(c.xt);
    auto low = [](const void* q, uintptr_t row) { return q ? reinterpret_cast<uintptr_t>(q) | row : 0; };
    const uintptr_t all = low(c.y, c.ldy * x) | low(c.r, c.ldr * x) | low(c.gate, c.ldg * x) | low(c.post, 0) | low(c.pre, 0) | low(c.r_out, c.ldro * x) |
                          (c.codes ? low(c.codes, c.ldh) * 2 : low(c.h, c.ldh * x));  // 8 codes are 8 bytes
    p.vec = all % 16 == 0;
    return c.xt == X_F32 ? launch_block_norm_f32(p, s) : c.xt == X_F16 ? launch_block_norm_f16(p, s) : launch_block_norm_bf16(p, s);
}

}  // namespace qmm
