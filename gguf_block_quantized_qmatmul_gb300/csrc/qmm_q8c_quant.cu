// qmm_q8c_quant.cu -- rows of activations to 8-bit codes with one scale each:
// for the caller, and as the first launch of a product.
//
// Mathematics.  d = max|x| / 127, code = round(x (1 / d)), halves away from
// zero, in f32 with every operation rounded on its own: codes are a function
// of the row alone (qmm_device.cuh, q8_scale and q8_code).
//
// Bound by the bytes (a row is read twice, the second time out of the cache)
// and, for few rows, by a launch and two trips to memory.  A warp per row where
// there are many short ones, else 256 or 1024 threads.
#include "qmm_q8c.cuh"

namespace qmm {
namespace {

enum : int { X_CODES = 3 };  // int8 codes, with their scales

struct PrepParams {
    QcRows a;
    int K;
    QcPrep p;
    int vec;  // rows start on 16 bytes
};

// Lanes 2 t + h (of 8) hold words j = 4 h .. 4 h + 3 of K 16 t + 2 j, + 1; returns words 4 i .. 4 i + 3 of the
// tile's f16 order, i = 4 h + t: the word for (j, t) stands at 4 j + t.
__device__ __forceinline__ uint4 qc_tile_transpose(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, int lane) {
    const bool b0 = lane & 2, b1 = lane & 4;
    uint32_t s0 = __shfl_xor_sync(0xffffffffu, b0 ? w0 : w1, 2), s1 = __shfl_xor_sync(0xffffffffu, b0 ? w2 : w3, 2);
    const uint32_t x0 = b0 ? s0 : w0, x1 = b0 ? w1 : s0, y0 = b0 ? s1 : w2, y1 = b0 ? w3 : s1;
    s0 = __shfl_xor_sync(0xffffffffu, b1 ? x0 : y0, 4);
    s1 = __shfl_xor_sync(0xffffffffu, b1 ? x1 : y1, 4);
    return b1 ? make_uint4(s0, s1, y0, y1) : make_uint4(x0, x1, s0, s1);
}

template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (TPR > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = __reduce_max_sync(0xffffffffu, red[threadIdx.x & (TPR / 32 - 1)]);
    }
    return v;
}
template <int TPR>
__device__ __forceinline__ uint32_t row_sum(uint32_t v, uint32_t* red) {
    v = __reduce_add_sync(0xffffffffu, v);
    if constexpr (TPR > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = (threadIdx.x & 31) < TPR / 32 ? red[threadIdx.x & 31] : 0u;
        v = __reduce_add_sync(0xffffffffu, v);
    }
    return v;
}

template <int XT, int TPR, bool F16>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) q8c_prep_kernel(const PrepParams q) {
    __shared__ uint32_t red[32];
    grid_dep_launch();
    grid_dep_wait();
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    const int lane = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    if (row >= q.a.M) return;  // whole warps
    const int n = (int)(q.p.pitch / 8);  // pieces of 8 values; the pitch is a multiple of 64 (f16: 128)
    const uint8_t* x = static_cast<const uint8_t*>(q.a.x) + row * q.a.ld * (XT == X_CODES ? 1 : x_size(XT));
    float d = 0.0f, id = 0.0f;
    if constexpr (XT == X_CODES) {
        d = q.a.scales[row];
    } else {
        uint32_t top = 0;
        for (int i = lane; 8 * i < q.K; i += 4 * TPR) {
            float f[4][8];
#pragma unroll
            for (int j = 0; j < 4; ++j) qc_load8<XT>(x, 8 * (i + j * TPR), q.K, q.vec, f[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, qc_abs_bits(f[j][e]));
        }
        qc_row_scale(row_max<TPR>(top, red), d, id);
    }
    uint32_t sq = 0;
    for (int i0 = 0; i0 < n; i0 += TPR) {  // whole warps, for the exchange; the last ones in part
        const int i = i0 + lane;
        if (i - (lane & 31) >= n) break;
        uint2 u = make_uint2(0u, 0u);
        if constexpr (XT == X_CODES) {
            const int k = 8 * i;
            if (q.vec && k + 8 <= q.K) {
                u = *reinterpret_cast<const uint2*>(x + k);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t b = k + e < q.K ? (uint32_t)x[k + e] << (8 * (e & 3)) : 0u;
                    if (e < 4) u.x |= b;
                    else u.y |= b;
                }
            }
        } else if (i < n) {
            float f[8];
            qc_load8<XT>(x, 8 * i, q.K, q.vec, f);
            u = qc_codes8(f, id);
        }
        if constexpr (F16) {
            sq = (uint32_t)dp4a(u.x, u.x, dp4a(u.y, u.y, (int)sq));
            uint32_t w[4];
            qc_half4(u.x, w[0], w[1]);
            qc_half4(u.y, w[2], w[3]);
            const uint4 v = qc_tile_transpose(w[0], w[1], w[2], w[3], lane);
            if (i < n) {
                const int t = i >> 1 & 3, h = i & 1;
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(q.p.codes) + row * q.p.pitch)[(i & ~7) + 4 * h + t] = v;
            }
        } else if (i < n) {
            int8_t* to = static_cast<int8_t*>(q.p.codes) + row * q.p.pitch + 8 * i;
            *reinterpret_cast<uint2*>(to) = u;
        }
    }
    if (F16) sq = row_sum<TPR>(sq, red);
    if (lane == 0) {
        q.p.scales[row] = d;
        if (F16) q.p.norms[row] = sq;
    }
}

// rows for the caller: any pitch
template <int XT>
__global__ void __launch_bounds__(256) q8c_quantize_kernel(const QcRows a, int K, int8_t* codes, long long ldc, float* scales, int vec, int vec_out) {
    __shared__ uint32_t red[32];
    grid_dep_launch();
    grid_dep_wait();
    const long long row = blockIdx.x;
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + row * a.ld * x_size(XT);
    uint32_t top = 0;
    for (int k = 8 * threadIdx.x; k < K; k += 4 * 2048) {
        float f[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) qc_load8<XT>(x, k + 2048 * j, K, vec, f[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, qc_abs_bits(f[j][e]));
    }
    float d, id;
    qc_row_scale(row_max<256>(top, red), d, id);
    int8_t* to = codes + row * ldc;
    for (int k = 8 * threadIdx.x; k < K; k += 2048) {
        float f[8];
        qc_load8<XT>(x, k, K, vec, f);
        const uint2 u = qc_codes8(f, id);
        if (vec_out && k + 8 <= K) {
            *reinterpret_cast<uint2*>(to + k) = u;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < K) to[k + e] = (int8_t)((e < 4 ? u.x : u.y) >> (8 * (e & 3)));
        }
    }
    if (threadIdx.x == 0) scales[row] = d;
}

bool rows_aligned(const QcRows& a, int size) { return (reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.ld * size)) % 16 == 0; }

template <int XT, bool F16>
cudaError_t prep_go(const PrepParams& q, cudaStream_t s) {
    // A product's time with a warp / 256 / 1024 threads a row, us: 512 x 1536 x 576 9.0 / 9.2 / 12.8, 4096 x 1536 x 576
    // 20 / 26 / 65; 512 x 1536 x 2048 16.8 / 13.7 / 17.4; 16 x 4096 x 4096 - / 11.4 / 10.9, 1024 x 4096 x 4096 - / 33 /
    // 42; 16 x 4096 x 8192 - / 16.0 / 14.0, 256 x 1536 x 8192 - / 20.6 / 21.5; 64 x 1536 x 14336 - / 19.0 / 16.4.
    if (q.K <= 1024 && q.a.M >= 512) return launch_pdl(q8c_prep_kernel<XT, 32, F16>, (unsigned)((q.a.M + 7) / 8), 256, 0, s, q);
    if (q.K < 4096 || q.a.M > q.K / 64) return launch_pdl(q8c_prep_kernel<XT, 256, F16>, (unsigned)q.a.M, 256, 0, s, q);
    return launch_pdl(q8c_prep_kernel<XT, 1024, F16>, (unsigned)q.a.M, 1024, 0, s, q);
}

}  // namespace

cudaError_t launch_q8c_prep(const QcRows& a, int K, const QcPrep& p, bool f16, cudaStream_t s) {
    PrepParams q = {a, K, p, 0};
    const int xt = a.scales ? (int)X_CODES : a.xt;
    q.vec = rows_aligned(a, xt == X_CODES ? 1 : x_size(xt));
    if (f16)
        return xt == X_F32 ? prep_go<X_F32, true>(q, s) : xt == X_F16 ? prep_go<X_F16, true>(q, s) : xt == X_BF16 ? prep_go<X_BF16, true>(q, s) : prep_go<X_CODES, true>(q, s);
    return xt == X_F32 ? prep_go<X_F32, false>(q, s) : xt == X_F16 ? prep_go<X_F16, false>(q, s) : xt == X_BF16 ? prep_go<X_BF16, false>(q, s) : prep_go<X_CODES, false>(q, s);
}

cudaError_t launch_q8c_quantize(const QcRows& a, int K, int8_t* codes, long long ldc, float* scales, cudaStream_t s) {
    const int vec = rows_aligned(a, x_size(a.xt)), vec_out = (reinterpret_cast<uintptr_t>(codes) | (uintptr_t)ldc) % 8 == 0;
    auto* k = a.xt == X_F32 ? q8c_quantize_kernel<X_F32> : a.xt == X_F16 ? q8c_quantize_kernel<X_F16> : q8c_quantize_kernel<X_BF16>;
    return launch_pdl(k, (unsigned)a.M, 256, 0, s, a, K, codes, ldc, scales, vec, vec_out);
}

}  // namespace qmm
