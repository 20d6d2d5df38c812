// qmm_q8c_layout.cu -- 8-bit channel-scaled weights: plain tensors to the
// laid-out form (qmm_q8c.cuh) and back to f32.
#include "qmm_q8c.cuh"

namespace qmm {
namespace {

// A block lays one row block out, a thread 16 codes at a time; bound by the codes' bytes, read and
// written once (14336 x 4096: 59 MB each way).
__global__ void __launch_bounds__(256) q8c_pack_kernel(const int8_t* __restrict__ codes, long long ldc, const float* __restrict__ scales,
                                                       const QcWeights w, uint8_t* out, int vec) {
    __shared__ uint32_t sq[16];
    if (threadIdx.x < 16) sq[threadIdx.x] = 0u;
    __syncthreads();
    const int rb = blockIdx.x, n16 = w.KS * 128;  // 16-byte pieces of a row block: KS x 2 tiles x 2 halves x 32 lanes
    uint8_t* to = out + qc_row_block(w, rb);
    const int step = qc_step(w, rb);
    for (int i = threadIdx.x; i < n16; i += 256) {
        const int lane = i & 31, row = (lane >> 2) + 8 * (i >> 5 & 1), n = rb * 16 + row, k = (i >> 6) * 64 + (lane & 3) * 16;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (n < w.N) {
            const int8_t* p = codes + (long long)n * ldc + k;
            if (vec && k + 16 <= w.K) {
                v = *reinterpret_cast<const uint4*>(p);
            } else {
                uint32_t u[4] = {};
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (k + j < w.K) u[j >> 2] |= (uint32_t)(uint8_t)p[j] << (8 * (j & 3));
                v = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
        reinterpret_cast<uint4*>(to + (long long)(i >> 7) * step)[i & 127] = v;
        int s = dp4a(v.x, v.x, 0);
        s = dp4a(v.y, v.y, s);
        s = dp4a(v.z, v.z, s);
        s = dp4a(v.w, v.w, s);
        atomicAdd(&sq[row], (uint32_t)s);
    }
    __syncthreads();
    if (threadIdx.x < 16) {
        const int n = rb * 16 + threadIdx.x;
        reinterpret_cast<float*>(out + w.scale_off)[n] = n < w.N ? scales[n] : 0.0f;
        atomicMax(reinterpret_cast<uint32_t*>(out + w.norm_off), sq[threadIdx.x]);
    }
}

__global__ void __launch_bounds__(256) q8c_dequantize_kernel(const QcWeights w, float* out) {
    const int rb = blockIdx.x, n16 = w.KS * 128;
    const uint8_t* from = w.data + qc_row_block(w, rb);
    const int step = qc_step(w, rb);
    const float* scales = reinterpret_cast<const float*>(w.data + w.scale_off) + rb * 16;
    for (int i = threadIdx.x; i < n16; i += 256) {
        const int lane = i & 31, row = (lane >> 2) + 8 * (i >> 5 & 1), n = rb * 16 + row, k = (i >> 6) * 64 + (lane & 3) * 16;
        if (n >= w.N) continue;
        const uint4 v = reinterpret_cast<const uint4*>(from + (long long)(i >> 7) * step)[i & 127];
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        const float s = scales[row];
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (k + j < w.K) out[(long long)n * w.K + k + j] = (float)(int8_t)(u[j >> 2] >> (8 * (j & 3))) * s;
    }
}

}  // namespace

cudaError_t launch_q8c_pack(const int8_t* codes, long long ldc, const float* scales, const QcWeights& w, void* out, cudaStream_t s) {
    uint8_t* o = static_cast<uint8_t*>(out);
    const cudaError_t e = cudaMemsetAsync(o + w.norm_off, 0, 16, s);
    if (e != cudaSuccess) return e;
    const int vec = (reinterpret_cast<uintptr_t>(codes) | (uintptr_t)ldc) % 16 == 0;
    q8c_pack_kernel<<<(unsigned)w.RB, 256, 0, s>>>(codes, ldc, scales, w, o, vec);
    return cudaGetLastError();
}

cudaError_t launch_q8c_dequantize(const QcWeights& w, float* out, cudaStream_t s) {
    q8c_dequantize_kernel<<<(unsigned)w.RB, 256, 0, s>>>(w, out);
    return cudaGetLastError();
}

}  // namespace qmm
