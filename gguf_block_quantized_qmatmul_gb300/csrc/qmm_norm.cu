// qmm_norm.cu -- what stands between two blocks of a decoder in one pass: the
// block's output is normed, gated, scaled and added to the residual stream, and
// the sum is normed for the next block, as floats or as 8-bit codes with a
// scale per row (what the 8-bit product takes).
//
// Mathematics, in f32 from the inputs to one rounding of each output:
//   v = y / sqrt(mean(y^2) + eps) (o + w_post)     (without post: v = y)
//   r' = r + s gate v,   h = r' / sqrt(mean(r'^2) + eps) (o + w_pre)
//   codes: d = max|h| / 127, round(h (1 / d)), as qmm_q8c_quant.cu
// h is made of r' before its rounding.
//
// Bound by the bytes, each read and written once: a row stays in registers, 8
// values a thread and piece, through up to three reductions (two sums, a
// maximum).  Everything that a row needs is asked for before the first one.
// Few rows are bound by a launch, one trip to memory and the reductions.
#include "qmm_q8c.cuh"

namespace qmm {
namespace {

struct NormParams {
    NormCall c;
    int vec;  // every row, and every one of the 8-value pieces, starts on its natural boundary
};

__device__ __forceinline__ void load8(const void* row, int type, int k, int K, bool vec, float f[8]) {
    if (type == X_F32) qc_load8<X_F32>(row, k, K, vec, f);
    else if (type == X_F16) qc_load8<X_F16>(row, k, K, vec, f);
    else qc_load8<X_BF16>(row, k, K, vec, f);
}
template <int XT>
__device__ __forceinline__ void store8(void* row, int k, int K, bool vec, const float f[8]) {
    if (vec && k + 8 <= K) {
        if constexpr (XT == X_F32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + k);
            p[0] = make_float4(f[0], f[1], f[2], f[3]);
            p[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (XT == X_F16) {
                    const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&v);
                } else {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&v);
                }
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < K) x_store(row, XT, k + i, f[i]);
    }
}

template <int TPR>
__device__ __forceinline__ float sum_row(float v, float* red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[threadIdx.x & (TPR / 32 - 1)];
#pragma unroll
        for (int o = TPR / 64; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}
template <int TPR>
__device__ __forceinline__ uint32_t max_row(uint32_t v, uint32_t* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = __reduce_max_sync(0xffffffffu, red[threadIdx.x & (TPR / 32 - 1)]);
    }
    return v;
}

template <int XT, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) block_norm_kernel(const NormParams p) {
    __shared__ float red[3][32];  // an area per reduction
    grid_dep_launch();
    const NormCall& c = p.c;
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    const int lane = threadIdx.x % TPR, K = c.K;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    const bool vec = p.vec;
    grid_dep_wait();
    if (row >= c.T) return;  // whole warps
    const uint8_t* y = static_cast<const uint8_t*>(c.y) + row * c.ldy * x_size(XT);
    float v[NV][8], r[NV][8], gate[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) qc_load8<XT>(y, 8 * (lane + TPR * j), K, vec, v[j]);
    if (c.r) {
        const uint8_t* from = static_cast<const uint8_t*>(c.r) + row * c.ldr * x_size(XT);
#pragma unroll
        for (int j = 0; j < NV; ++j) qc_load8<XT>(from, 8 * (lane + TPR * j), K, vec, r[j]);
    }
    if (c.gate) {
        const uint8_t* from = static_cast<const uint8_t*>(c.gate) + row * c.ldg * x_size(XT);
#pragma unroll
        for (int j = 0; j < NV; ++j) qc_load8<XT>(from, 8 * (lane + TPR * j), K, vec, gate[j]);
    }
    const float mean = 1.0f / (float)K;
    if (c.post) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[j][e], v[j][e], ss);
        const float rs = 1.0f / sqrtf(fmaf(sum_row<TPR>(ss, red[0]), mean, c.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float w[8];
            load8(c.post, c.wt, 8 * (lane + TPR * j), K, vec, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * rs * (c.offset + w[e]);
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float a = v[j][e];
            if (c.gate) a *= gate[j][e];
            v[j][e] = c.r ? fmaf(c.scale, a, r[j][e]) : c.scale * a;
            ss = fmaf(v[j][e], v[j][e], ss);
        }
    if (c.r_out) {
        uint8_t* to = static_cast<uint8_t*>(c.r_out) + row * c.ldro * x_size(XT);
#pragma unroll
        for (int j = 0; j < NV; ++j) store8<XT>(to, 8 * (lane + TPR * j), K, vec, v[j]);
    }
    // past the row's end (k >= K) y, r and gate are 0, so the values are; a weight offset does not reach them
    const float rs = 1.0f / sqrtf(fmaf(sum_row<TPR>(ss, red[1]), mean, c.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float w[8];
        load8(c.pre, c.wt, 8 * (lane + TPR * j), K, vec, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * rs * (c.offset + w[e]);
    }
    if (!c.codes) {
        uint8_t* to = static_cast<uint8_t*>(c.h) + row * c.ldh * x_size(XT);
#pragma unroll
        for (int j = 0; j < NV; ++j) store8<XT>(to, 8 * (lane + TPR * j), K, vec, v[j]);
        return;
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (8 * (lane + TPR * j) + e < K) top = max(top, qc_abs_bits(v[j][e]));
    float d, id;
    qc_row_scale(max_row<TPR>(top, reinterpret_cast<uint32_t*>(red[2])), d, id);
    int8_t* to = c.codes + row * c.ldh;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int k = 8 * (lane + TPR * j);
        const uint2 u = qc_codes8(v[j], id);
        if (vec && k + 8 <= K) {
            *reinterpret_cast<uint2*>(to + k) = u;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < K) to[k + e] = (int8_t)((e < 4 ? u.x : u.y) >> (8 * (e & 3)));
        }
    }
    if (lane == 0) c.scales[row] = d;
}

template <int XT>
cudaError_t norm_go(const NormParams& p, cudaStream_t s) {
    const int K = p.c.K;
    const unsigned T = (unsigned)p.c.T;
    if (K <= 1024 && T >= 1024) return launch_pdl(block_norm_kernel<XT, 32, 4>, (T + 7) / 8, 256, 0, s, p);
    if (K <= 2048) return launch_pdl(block_norm_kernel<XT, 256, 1>, T, 256, 0, s, p);
    if (K <= 4096) return launch_pdl(block_norm_kernel<XT, 256, 2>, T, 256, 0, s, p);
    if (K <= 8192) return launch_pdl(block_norm_kernel<XT, 1024, 1>, T, 1024, 0, s, p);
    return launch_pdl(block_norm_kernel<XT, 1024, 4>, T, 1024, 0, s, p);
}

}  // namespace

cudaError_t launch_block_norm(const NormCall& c, cudaStream_t s) {
    NormParams p = {c, 0};
    const uintptr_t x = (uintptr_t)x_size(c.xt);
    auto low = [](const void* q, uintptr_t row) { return q ? reinterpret_cast<uintptr_t>(q) | row : 0; };
    const uintptr_t all = low(c.y, c.ldy * x) | low(c.r, c.ldr * x) | low(c.gate, c.ldg * x) | low(c.post, 0) | low(c.pre, 0) | low(c.r_out, c.ldro * x) |
                          (c.codes ? low(c.codes, c.ldh) * 2 : low(c.h, c.ldh * x));  // 8 codes are 8 bytes
    p.vec = all % 16 == 0;
    return c.xt == X_F32 ? norm_go<X_F32>(p, s) : c.xt == X_F16 ? norm_go<X_F16>(p, s) : norm_go<X_BF16>(p, s);
}

}  // namespace qmm
