// qmm_q4g_layout.cu -- laying out 4-bit weights with group scales, once, when
// a program loads them; and reading them back as f32.
#include "qmm_q4g_internal.h"

namespace qmm {
namespace {

// codes two to a byte (even k in the low nibble), scales f16 or bf16 and zero
// points per group of gsrc inputs
struct RowSource {
    const uint8_t* codes;  // [E][N][K / 2]
    const void* scales;    // [E][N][K / gsrc]
    const uint8_t* zeros;  // [E][N][K / gsrc], or NULL: 8
    int bf16, gsrc;
    // the codes of row (e N + n), k and k + 1 (k even)
    __device__ uint32_t pair(long long row, int K, int k) const { return codes[row * (K / 2) + k / 2]; }
    __device__ void group(long long row, int K, int k, float& s, uint32_t& z) const {
        const long long i = row * (K / gsrc) + k / gsrc;
        s = x_load(scales, bf16 ? X_BF16 : X_F16, i);
        z = zeros ? zeros[i] & 15u : 8u;
    }
};

// GGUF Q4_0 blocks: f16 d, then code j in the low nibble of byte j and code
// j + 16 in its high nibble; w = d (code - 8)
struct Q40Source {
    const uint8_t* wq;
    __device__ uint32_t pair(long long row, int K, int k) const {
        const uint8_t* b = wq + (row * (K / 32) + k / 32) * 18 + 2;
        const int j = k % 32, sh = j < 16 ? 0 : 4;
        return ((b[j & 15] >> sh) & 15u) | (((b[(j + 1) & 15] >> sh) & 15u) << 4);
    }
    __device__ void group(long long row, int K, int k, float& s, uint32_t& z) const {
        s = h2f(*reinterpret_cast<const uint16_t*>(wq + (row * (K / 32) + k / 32) * 18));
        z = 8u;
    }
};

// one warp per segment
template <class Source>
__global__ void __launch_bounds__(256) q4g_pack_kernel(Source src, QgWeights w, uint8_t* __restrict__ out) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long per = (long long)w.RB * w.KS, total = per * w.E;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (long long)gridDim.x * 8) {
        const int e = (int)(i / per), rb = (int)(i % per / w.KS), seg = (int)(i % w.KS);
        const int n0 = qg_row(w, rb, g), n1 = qg_row(w, rb, g + 8);
        const long long r0 = (long long)e * w.N + n0, r1 = (long long)e * w.N + n1;
        uint8_t* o = out + e * w.expert_stride + (long long)(rb * (long long)w.KS + seg) * qg_seg_bytes(w.ng);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t word[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = seg * kQgSegK + 64 * h + 16 * s + 2 * t;
                uint32_t v = 0;
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    const int kk = k + 8 * (i4 >> 1);
                    const bool on = kk < w.K && ((i4 & 1) ? n1 >= 0 : n0 >= 0);
                    const uint32_t b = on ? src.pair((i4 & 1) ? r1 : r0, w.K, kk) : 0u;
                    v |= (b & 15u) << (4 * i4) | (b >> 4) << (16 + 4 * i4);
                }
                word[s] = v;
            }
            reinterpret_cast<uint4*>(o + h * kQgTile)[lane] = make_uint4(word[0], word[1], word[2], word[3]);
        }
        for (int j = lane; j < 16 * w.ng; j += 32) {  // [g][group][2]
            const int gg = j / (2 * w.ng), gi = j / 2 % w.ng, hi = j & 1;
            const int n = qg_row(w, rb, gg + 8 * hi), k = seg * kQgSegK + gi * (kQgSegK / w.ng);
            float s = 0.0f;
            uint32_t z = 0;
            if (n >= 0 && k < w.K) src.group((long long)e * w.N + n, w.K, k, s, z);
            reinterpret_cast<uint32_t*>(o + 2 * kQgTile)[j] = (__float_as_uint(s) & ~15u) | z;
        }
    }
}

// the row powers of two: one warp per row
__global__ void __launch_bounds__(256) q4g_iscale_kernel(QgWeights w, uint8_t* __restrict__ out) {
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)w.E * w.RB * 16;
    float* is = reinterpret_cast<float*>(out + w.iscale_off);
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < rows; i += (long long)gridDim.x * 8) {
        const int e = (int)(i / (w.RB * 16)), rb = (int)(i / 16 % w.RB), r = (int)(i & 15);
        const uint8_t* base = out + e * w.expert_stride + (long long)rb * w.KS * qg_seg_bytes(w.ng);
        float m = 0.0f;
        for (int j = lane; j < w.KS * w.ng; j += 32) {
            const uint32_t* sw = reinterpret_cast<const uint32_t*>(base + (long long)(j / w.ng) * qg_seg_bytes(w.ng) + 2 * kQgTile);
            m = fmaxf(m, fabsf(qg_scale(sw[((r & 7) * w.ng + j % w.ng) * 2 + (r >> 3)])));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) is[i] = tc_row_iscale(15.0f * m);
    }
}

__global__ void __launch_bounds__(256) q4g_dequantize_kernel(QgWeights w, float* __restrict__ out) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long per = (long long)w.RB * w.KS, total = per * w.E;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (long long)gridDim.x * 8) {
        const int e = (int)(i / per), rb = (int)(i % per / w.KS), seg = (int)(i % w.KS);
        const uint8_t* b = w.data + e * w.expert_stride + (long long)(rb * (long long)w.KS + seg) * qg_seg_bytes(w.ng);
        const uint32_t* sw = reinterpret_cast<const uint32_t*>(b + 2 * kQgTile);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 q = reinterpret_cast<const uint4*>(b + h * kQgTile)[lane];
            const uint32_t word[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    const int kl = 64 * h + 16 * s + 2 * t + 8 * (i4 >> 1), k = seg * kQgSegK + kl;
                    const int n = qg_row(w, rb, g + 8 * (i4 & 1));
                    if (n < 0 || k >= w.K) continue;
                    const uint32_t v = sw[(g * w.ng + kl / (kQgSegK / w.ng)) * 2 + (i4 & 1)];
                    const float sc = qg_scale(v);
                    const int z = (int)(v & 15u);
                    float2 f;  // an 11-bit scale times at most 4 bits: exact
                    f.x = sc * (float)((int)((word[s] >> (4 * i4)) & 15u) - z);
                    f.y = sc * (float)((int)((word[s] >> (16 + 4 * i4)) & 15u) - z);
                    *reinterpret_cast<float2*>(out + ((long long)e * w.N + n) * w.K + k) = f;
                }
        }
    }
}

unsigned blocks_for(long long warps) {
    const long long b = (warps + 7) / 8;
    return (unsigned)(b < 4864 ? b : 4864);
}

template <class Source>
cudaError_t pack(const Source& src, const QgWeights& w, void* out, cudaStream_t s) {
    q4g_pack_kernel<<<blocks_for((long long)w.E * w.RB * w.KS), 256, 0, s>>>(src, w, static_cast<uint8_t*>(out));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    q4g_iscale_kernel<<<blocks_for((long long)w.E * w.RB * 16), 256, 0, s>>>(w, static_cast<uint8_t*>(out));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q4g_pack(const uint8_t* codes, const void* scales, int bf16, const uint8_t* zeros, int gsrc, const QgWeights& w,
                            void* out, cudaStream_t s) {
    return pack(RowSource{codes, scales, zeros, bf16, gsrc}, w, out, s);
}

cudaError_t launch_q4g_pack_q4_0(const uint8_t* wq, const QgWeights& w, void* out, cudaStream_t s) {
    return pack(Q40Source{wq}, w, out, s);
}

cudaError_t launch_q4g_dequantize(const QgWeights& w, float* out, cudaStream_t s) {
    q4g_dequantize_kernel<<<blocks_for((long long)w.E * w.RB * w.KS), 256, 0, s>>>(w, out);
    return cudaGetLastError();
}

}  // namespace qmm
